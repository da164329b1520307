// Softmax attention of a few new tokens per request over a paged cache
// (gfx950): at most 64 rows (tokens times heads of a group) per (request,
// group).  Semantics: include/kda_attn.h.
//
// Bound by HBM: keys and values are read once, for all heads of their group.
// The steps of 64 (128) keys of all units (request b, group g) lie on one line,
//   unit b G + g starts at G sum_{b' < b} steps(b') + g steps(b),
// which is cut into equal pieces, one per workgroup, so that every compute unit
// reads the same amount whatever the requests' lengths are; a workgroup finds
// its piece from the lengths by itself.  It may hold the end of one unit, some
// whole ones and the start of another.  A unit that one workgroup holds alone
// is finished there, the others are joined by a second launch from the parts'
// sums, in the order of the keys.
//   Within a workgroup a wave has 16 (32) keys of each step in LDS of its own,
// two steps deep, which come from memory without passing through registers: no
// barriers, only counts of loads.  S^T = K Q^T leaves lane l with row l & 15 and
// keys 4 (l >> 4) + i, the place of P^T as an operand of O^T = V^T P^T.  The
// waves' sums are joined when the unit or the piece ends.
//   One token of each of 64 requests, 32 heads of 128 on 8, bf16: 233 us where
// they hold 2048 to 8192 tokens (1.34 GB, 5.7 TB/s), 363 with 8192 each (2.15 GB,
// 5.9; a copy of 1 GiB: 5.2); 4, 6 and 8 tokens of 64 requests of 4096, 64 heads
// of 128 on 8: 195, 203 and 228 us (with four tiles of 16 rows 31 registers are
// in memory).
#include "kda_attn_mma.h"

namespace kda {

constexpr int SP_THREADS = 256, SP_WAVES = 4;

template <typename InT, int D>
struct StepTile {
    static constexpr int ROWB = D * (int)sizeof(InT), UNITS = ROWB / 16, GROUP = 16 * ROWB;   // a row, 16 rows
    static constexpr int NG = GROUP < 4096 ? 2 : 1;              // groups of 16 keys per wave and step
    static constexpr int LOADS = GROUP / 1024, RPL = 1024 / ROWB;
    static constexpr int STEP = 64 * NG;                         // keys
    static constexpr int BUF = 2 * NG * GROUP;                   // keys and values of a wave's step
    static constexpr int PER_UNIT = BUF > 8192 ? 1 : 2;          // workgroups that a compute unit's LDS holds
    static constexpr bool F32 = sizeof(InT) == 4;
};
__device__ __forceinline__ int step_swap(int units, int row) { return row & (units < 16 ? units - 1 : 15); }

// Steps of request n's keys (0: it has no rows).
__device__ __forceinline__ int32_t step_count(const AttnParams& p, int n, int step) {
    if (p.cu) {
        const AttnRange r = attn_range(p.cu, p.rows, p.T, n);
        if (r.end == r.start) return 0;
    }
    return (attn_length(p, n) + step - 1) / step;
}
// Sum of x over the workgroup's threads before this one, and over all.
__device__ __forceinline__ int64_t step_before(int32_t x, int64_t* s, int64_t& total) {
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    int64_t up = x;
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) {
        const int64_t y = __shfl_up(up, d);
        if (lane >= d) up += y;
    }
    __syncthreads();
    if (lane == 63) s[wave] = up;
    __syncthreads();
    int64_t base = 0;
    total = 0;
#pragma unroll
    for (int w = 0; w < SP_WAVES; ++w) {
        if (w < wave) base += s[w];
        total += s[w];
    }
    total = uniform(total);
    return base + up - x;
}
__device__ __forceinline__ int64_t step_quota(int64_t total, int32_t workgroups) {
    return total > 0 ? (total + workgroups - 1) / workgroups : 1;
}

// Row r of request b's new tokens.
struct StepRow {
    int64_t at;       // token row
    int32_t head, sees;
    bool valid;
};
__device__ __forceinline__ StepRow step_row(const AttnParams& p, const AttnRange& q, int32_t len, int g, int r) {
    const int32_t tokens = (int32_t)(q.end - q.start);
    StepRow x;
    x.valid = r < tokens * p.hpg;
    const int32_t t = x.valid ? r / p.hpg : 0;
    x.head = g * p.hpg + (x.valid ? r - t * p.hpg : 0);
    x.at = q.start + t;
    x.sees = x.valid ? len - tokens + t + 1 : 0;
    return x;
}

// Workspace: first and last workgroup of each unit, then the parts (see AttnParams).
__device__ __forceinline__ int32_t* step_info(const AttnParams& p) { return reinterpret_cast<int32_t*>(p.part); }
template <int D, int RT>
__device__ __forceinline__ float* step_part(const AttnParams& p, int64_t slot, int row) {
    return p.part + (((int64_t)p.n_seqs * p.G * 2 + 3) & ~(int64_t)3) + (slot * (RT * 16) + row) * (D + 4);
}

template <typename InT, int D, int RT>
__global__ __launch_bounds__(SP_THREADS, (StepTile<InT, D>::PER_UNIT)) void attn_step_kernel(AttnParams p) {
    typedef StepTile<InT, D> Tile;
    constexpr int NG = Tile::NG, LOADS = Tile::LOADS, GROUP = Tile::GROUP, ROWB = Tile::ROWB, UNITS = Tile::UNITS;
    constexpr bool F32 = Tile::F32;
    constexpr int S = F32 ? D / 16 : D / 32, O = D / 16, PITCH = D + 4;
    __shared__ __attribute__((aligned(1024))) char lds[SP_WAVES * 2 * Tile::BUF];
    __shared__ float ml[SP_WAVES][16][2];
    __shared__ int64_t sums[SP_WAVES];
    __shared__ int64_t found[2];   // first request of the piece, steps before it
    static_assert(SP_WAVES * 16 * PITCH * 4 <= (int)sizeof(lds), "");
    const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int col = lane & 15, grp = lane >> 4;

    // this workgroup's piece of the line; the first 256 requests stay in registers
    const int32_t mine = tid < p.n_seqs ? step_count(p, tid, Tile::STEP) : 0;
    int64_t all;
    const int64_t mine_before = step_before(mine, sums, all);
    int64_t total = all;
    for (int b0 = SP_THREADS; b0 < p.n_seqs; b0 += SP_THREADS) {
        int64_t more;
        step_before(b0 + tid < p.n_seqs ? step_count(p, b0 + tid, Tile::STEP) : 0, sums, more);
        total += more;
    }
    total *= p.G;
    const int64_t quota = step_quota(total, p.workgroups);
    const int64_t begin = blockIdx.x * quota, end = begin + quota < total ? begin + quota : total;
    if (begin >= end) return;
    auto find = [&](int b, int32_t x, int64_t before) {
        if (x > 0 && begin >= before * p.G && begin < (before + x) * p.G) {
            found[0] = b;
            found[1] = before;
        }
    };
    find(tid, mine, mine_before);
    for (int b0 = SP_THREADS; b0 < p.n_seqs && begin >= all * p.G; b0 += SP_THREADS) {
        const int32_t x = b0 + tid < p.n_seqs ? step_count(p, b0 + tid, Tile::STEP) : 0;
        int64_t more;
        const int64_t before = all + step_before(x, sums, more);
        find(b0 + tid, x, before);
        all += more;
    }
    __syncthreads();
    int b = (int)uniform(found[0]);
    int64_t unit0 = uniform(found[1]) * p.G;   // first step of request b
    const float scale = p.scale < 0.f ? -p.scale : p.scale > 0.f ? p.scale : 1.f;
    const float sign = p.scale < 0.f ? -1.f : p.scale > 0.f ? 1.f : 0.f;
    const float c = scale * kLog2e;

    const uint32_t lds0 = (uint32_t)(uintptr_t)(__attribute__((address_space(3))) char*)lds + wave * 2 * Tile::BUF;
    char* own = lds + wave * 2 * Tile::BUF;
    uint32_t off[LOADS];
#pragma unroll
    for (int i = 0; i < LOADS; ++i) {
        const int r = i * Tile::RPL + lane / UNITS;
        off[i] = (uint32_t)(r * ROWB + ((lane % UNITS) ^ step_swap(UNITS, r)) * 16);
    }

    int64_t at = begin;
    while (at < end) {
        int32_t steps = step_count(p, b, Tile::STEP);
        while (at >= unit0 + (int64_t)steps * p.G) {   // the next request that has any
            unit0 += (int64_t)steps * p.G;
            steps = step_count(p, ++b, Tile::STEP);
        }
        const int g = (int)((at - unit0) / steps);
        const int64_t base = unit0 + (int64_t)g * steps;
        const int32_t j0 = (int32_t)(at - base), j1 = (int32_t)(end - base < steps ? end - base : steps);
        const int32_t len = attn_length(p, b);
        const AttnRange qr = attn_range(p.cu, p.rows, p.T, b);
        const AttnKeys<InT, true> keys(p, b, 0, g);

        // page of (step, group) pbase + lane, 64 of them
        int32_t pages = 0, pbase = j0;
        auto pages_from = [&](int32_t step) {
            const int64_t key = (int64_t)(step + lane / NG) * Tile::STEP + 16 * (wave * NG + lane % NG);
            pages = key < len ? keys.pages[key >> keys.shift] : -1;
            pbase = step;
        };
        pages_from(j0);

        // queries as operands: lane l has row l & 15
        float qf[RT][F32 ? S : 1][4];
        bf16x8 qb[RT][F32 ? 1 : S];
        int32_t sees[RT];
#pragma unroll
        for (int rt = 0; rt < RT; ++rt) {
            const StepRow x = step_row(p, qr, len, g, 16 * rt + col);
            sees[rt] = x.sees;
            const InT* qrow = (const InT*)p.q + x.at * p.q_stride + (int64_t)x.head * D;
#pragma unroll
            for (int s = 0; s < S; ++s) {
                if constexpr (F32) {
                    load4(qrow + 16 * s + 4 * grp, qf[rt][s]);
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        qf[rt][s][e] = x.valid ? qf[rt][s][e] * sign : 0.f;
                    }
                } else {
                    u32x4 w = *reinterpret_cast<const u32x4*>(qrow + 32 * s + 8 * grp);
#pragma unroll
                    for (int e = 0; e < 4; ++e) w[e] = x.valid && sign != 0.f ? w[e] ^ (sign < 0.f ? 0x80008000u : 0u) : 0u;
                    qb[rt][s] = __builtin_bit_cast(bf16x8, w);
                }
            }
        }
#pragma unroll
        for (int rt = 0; rt < RT; ++rt)
#pragma unroll
            for (int s = 0; s < S; ++s) {
                if constexpr (F32) {
#pragma unroll
                    for (int e = 0; e < 4; ++e) asm volatile("" : "+v"(qf[rt][s][e]));
                } else {
                    arrive(qb[rt][s]);
                }
            }
        asm volatile("" : "+v"(pages));   // (arrive here, too)
        const int32_t sees_least = (int32_t)(len - (qr.end - qr.start)) + 1;

        auto request = [&](int32_t step, int buf, bool (&ok)[NG]) {
            if (step - pbase >= 64 / NG) {
                pages_from(step);
                asm volatile("" : "+v"(pages));
            }
#pragma unroll
            for (int n = 0; n < NG; ++n) {
                const int32_t key = step * Tile::STEP + 16 * (wave * NG + n);
                const int32_t page = __builtin_amdgcn_readlane(pages, (step - pbase) * NG + n);
                ok[n] = key < len && page >= 0 && page < keys.n_pages;
                const int64_t from = ok[n] ? (int64_t)page * keys.k_stride + (int64_t)(key & ((1 << keys.shift) - 1)) * D : 0;
                const int32_t left = len - key < 16 ? len - key : 16;
                const auto krs = make_rsrc(keys.k + from, ok[n] ? left * ROWB : 0);
                const auto vrs = make_rsrc(keys.v + from, ok[n] ? left * ROWB : 0);
                const uint32_t to = lds0 + buf * Tile::BUF + n * GROUP;
                load_to_lds(krs, off, to);
                load_to_lds(vrs, off, to + NG * GROUP);
            }
        };

        f32x4 o[RT][O];
        float m[RT], l[RT];
#pragma unroll
        for (int rt = 0; rt < RT; ++rt) {
            m[rt] = kAttnLowest;
            l[rt] = 0.f;
#pragma unroll
            for (int i = 0; i < O; ++i) o[rt][i] = f32x4{0.f, 0.f, 0.f, 0.f};
        }
        bool ok[NG], next_ok[NG];
        request(j0, 0, next_ok);
        for (int32_t j = j0; j < j1; ++j) {
            const int buf = (j - j0) & 1;
#pragma unroll
            for (int n = 0; n < NG; ++n) ok[n] = next_ok[n];
            if (j + 1 < j1) {
                asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");   // (the other half has been read)
                request(j + 1, buf ^ 1, next_ok);
                asm volatile("s_waitcnt vmcnt(%0)" ::"n"(2 * NG * LOADS) : "memory");
            } else {
                asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
            }
#pragma unroll
            for (int n = 0; n < NG; ++n) {
                const int32_t key0 = j * Tile::STEP + 16 * (wave * NG + n);
                if (!ok[n]) continue;
                const char* ks = own + buf * Tile::BUF + n * GROUP;
                const char* vs = ks + NG * GROUP;
                f32x4 x[RT];
#pragma unroll
                for (int rt = 0; rt < RT; ++rt) x[rt] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
                for (int s = 0; s < S; ++s) {
                    const char* from = ks + col * ROWB + (((4 * s + grp) ^ step_swap(UNITS, col)) * 16);
                    if constexpr (F32) {
                        float a[4];
                        load4(reinterpret_cast<const float*>(from), a);
#pragma unroll
                        for (int rt = 0; rt < RT; ++rt) mma_k16<true, PLAIN>(x[rt], a, qf[rt][s]);
                    } else {
                        const bf16x8 a = *reinterpret_cast<const bf16x8*>(from);
#pragma unroll
                        for (int rt = 0; rt < RT; ++rt) x[rt] = mfma32(a, qb[rt][s], x[rt]);
                    }
                }
                bool grown = false;
                float top[RT];
#pragma unroll
                for (int rt = 0; rt < RT; ++rt) {
                    if (key0 + 16 > sees_least) {
#pragma unroll
                        for (int i = 0; i < 4; ++i) x[rt][i] = key0 + 4 * grp + i < sees[rt] ? x[rt][i] : -INFINITY;
                    }
                    top[rt] = fmaxf(fmaxf(fmaxf(x[rt][0], x[rt][1]), fmaxf(x[rt][2], x[rt][3])) * c, kAttnLowest);
                    grown = grown || top[rt] > m[rt] + 8.f;
                }
                if (__any(grown)) {
#pragma unroll
                    for (int rt = 0; rt < RT; ++rt) {
                        const float to = fmaxf(m[rt], groups_max(top[rt])), fade = attn_exp2(m[rt] - to);
                        m[rt] = to;
                        l[rt] *= fade;
#pragma unroll
                        for (int i = 0; i < O; ++i) o[rt][i] *= fade;
                    }
                }
                float w[RT][4];
#pragma unroll
                for (int rt = 0; rt < RT; ++rt)
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        w[rt][i] = attn_exp2(fmaf(x[rt][i], c, -m[rt]));
                        l[rt] += w[rt][i];
                    }
#pragma unroll
                for (int i = 0; i < O; ++i) {
                    if constexpr (F32) {
                        float a[4];
#pragma unroll
                        for (int e = 0; e < 4; ++e) {
                            const int r = 4 * grp + e;
                            a[e] = *reinterpret_cast<const float*>(vs + r * ROWB + (((4 * i + (col >> 2)) ^ step_swap(UNITS, r)) * 16) + 4 * (col & 3));
                        }
#pragma unroll
                        for (int rt = 0; rt < RT; ++rt) mma_k16<true, PLAIN>(o[rt][i], a, w[rt]);
                    } else {
                        const int r = 4 * grp + (col >> 2);
                        const s16x4 a = __builtin_amdgcn_ds_read_tr16_b64_v4i16((__attribute__((address_space(3))) s16x4*)(
                            vs + r * ROWB + (((2 * i + ((col & 3) >> 1)) ^ step_swap(UNITS, r)) * 16) + 8 * (col & 1)));
#pragma unroll
                        for (int rt = 0; rt < RT; ++rt) o[rt][i] = mfma16(__builtin_bit_cast(bf16x4, a), round4(w[rt]), o[rt][i]);
                    }
                }
            }
        }

        // the waves' sums, 16 rows at a time
        const bool whole = j0 == 0 && j1 == steps;
        const int64_t unit = (int64_t)b * p.G + g;
        const int n_rows = (int)(qr.end - qr.start) * p.hpg;
        float* joint = reinterpret_cast<float*>(lds);
        if (tid == 0) {   // whose parts the second launch joins: the first workgroup (-1: nothing is left to do) and the last
            int32_t* info = step_info(p) + 2 * unit;
            if (j0 == 0) info[0] = whole ? -1 : (int32_t)blockIdx.x;
            if (j1 == steps) info[1] = (int32_t)blockIdx.x;
        }
#pragma unroll
        for (int rt = 0; rt < RT; ++rt) {
            if (16 * rt >= n_rows) break;
            const float sum = groups_sum(l[rt]);
            __syncthreads();
#pragma unroll
            for (int i = 0; i < O; ++i)
                *reinterpret_cast<f32x4*>(joint + (wave * 16 + col) * PITCH + 16 * i + 4 * grp) = o[rt][i];
            if (grp == 0) {
                ml[wave][col][0] = sum;
                ml[wave][col][1] = m[rt];
            }
            __syncthreads();
            const int r = tid >> 4, d = (tid & 15) * 4;
            float top = kAttnLowest, w[SP_WAVES], sl = 0.f;
#pragma unroll
            for (int v = 0; v < SP_WAVES; ++v) top = fmaxf(top, ml[v][r][1]);
#pragma unroll
            for (int v = 0; v < SP_WAVES; ++v) {
                w[v] = attn_exp2(ml[v][r][1] - top);
                sl += w[v] * ml[v][r][0];
            }
            const StepRow x = step_row(p, qr, len, g, 16 * rt + r);
            const float inv = !whole ? 1.f : attn_inverse(sl);
            float* part = step_part<D, RT>(p, blockIdx.x + unit, 16 * rt + r);
#pragma unroll
            for (int k = 0; k < D / 64; ++k) {
                float y[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
                for (int v = 0; v < SP_WAVES; ++v) {
                    const f32x4 z = *reinterpret_cast<const f32x4*>(joint + (v * 16 + r) * PITCH + 64 * k + d);
#pragma unroll
                    for (int e = 0; e < 4; ++e) y[e] += w[v] * z[e];
                }
#pragma unroll
                for (int e = 0; e < 4; ++e) y[e] *= inv;
                if (x.valid) {
                    if (whole) store4((InT*)p.o + (x.at * p.H + x.head) * D + 64 * k + d, y);
                    else store4(part + 64 * k + d, y);
                }
            }
            if (x.valid && d == 0) {
                if (!whole) {
                    part[D] = sl;
                    part[D + 1] = top;
                } else if (p.lse) {
                    p.lse[x.at * p.H + x.head] = attn_lse(top, sl);
                }
            }
        }
        __syncthreads();   // (the LDS is the tiles' again)
        at = base + j1;
    }
}

// Row r of request b's new tokens once more, by one wave (attn_row_again).
template <typename InT, int D>
__device__ __forceinline__ bool step_again(const AttnParams& p, int b, int g, int64_t at, int head, const AttnRange& qr, int r,
                                           bool anyway) {
    const int lane = threadIdx.x & 63;
    const int32_t len = attn_length(p, b), sees = step_row(p, qr, len, g, r).sees;
    float y[D / 64], m, l;
    if (!attn_row_again<InT, D, true>(p, b, 0, g, at, head, 0, sees, len, y, m, l, anyway)) return false;
    const float inv = attn_inverse(l);
#pragma unroll
    for (int e = 0; e < D / 64; ++e) ((InT*)p.o)[(at * p.H + head) * D + 64 * e + lane] = (InT)(y[e] * inv);
    if (p.lse && lane == 0) p.lse[at * p.H + head] = attn_lse(m, l);
    return true;
}

// A row of a unit that several workgroups hold: o = sum_s e^{m_s - m} o_s / sum_s e^{m_s - m} l_s;
// of one that nobody holds (a request without tokens); and any that is not finite because of a key that it does not see,
// or of the joining's own products with zero.  WAVES waves share a
// row's parts, lane i first takes the sums and maxima of parts i, i + 64, ...
template <typename InT, int D, int RT, int WAVES>
__global__ __launch_bounds__(WAVES > 4 ? 64 * WAVES : 256) void attn_step_join_kernel(AttnParams p, int32_t max_rows) {
    constexpr int E = D / 64, ROWS = WAVES > 4 ? 1 : 4 / WAVES;
    __shared__ float ml[ROWS * WAVES][2], joint[WAVES > 1 ? WAVES : 1][D];
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const uint32_t per = (uint32_t)(max_rows + ROWS - 1) / ROWS;
    const int64_t unit = blockIdx.x / per;
    const int r = (int)(blockIdx.x % per) * ROWS + wave / WAVES, share = wave % WAVES;
    const int b = (int)(unit / p.G), g = (int)(unit % p.G);
    const AttnRange qr = attn_range(p.cu, p.rows, p.T, b);
    const StepRow x = step_row(p, qr, 0, g, r);
    const int32_t steps = step_count(p, b, StepTile<InT, D>::STEP);
    int32_t w0 = 0, w1 = -1;
    if (steps > 0) {
        w0 = step_info(p)[2 * unit];
        w1 = step_info(p)[2 * unit + 1];
    }
    if (!x.valid) return;   // (the whole workgroup where its waves share a row)
    InT* orow = (InT*)p.o + (x.at * p.H + x.head) * D;
    float odd = 0.f;   // NaN if a value is not finite
    if (w0 < 0) {
        if (share == 0 && x.at + 1 < qr.end) {   // (the last token sees every key)
#pragma unroll
            for (int e = 0; e < E; ++e) odd = fmaf(to_f32(orow[64 * e + lane]), 0.f, odd);
            if (__any(odd != 0.f)) step_again<InT, D>(p, b, g, x.at, x.head, qr, r, false);
        }
        return;
    }
    const int32_t n = w1 - w0 + 1;
    float m = kAttnLowest, l = 0.f, o[E] = {};
    for (int32_t i0 = 64 * share; i0 < n; i0 += 64 * WAVES) {
        const bool in = i0 + lane < n;
        const float* mine = step_part<D, RT>(p, w0 + (in ? i0 + lane : 0) + unit, r);
        const float pl = in ? mine[D] : 0.f, pm = in ? mine[D + 1] : kAttnLowest;
        float top = pm;
#pragma unroll
        for (int d = 1; d < 64; d <<= 1) top = fmaxf(top, __shfl_xor(top, d));
        const float to = fmaxf(m, top), fade = attn_exp2(m - to), weight = attn_exp2(pm - to);
        m = to;
        l = l * fade + wave_sum_dpp(weight * pl);
#pragma unroll
        for (int e = 0; e < E; ++e) o[e] *= fade;
        const int32_t here = n - i0 < 64 ? n - i0 : 64;
        const float* from = step_part<D, RT>(p, w0 + i0 + unit, r);
        for (int32_t i = 0; i < here; i += 8) {   // (eight requests at once; behind the last part, its values with weight 0)
            float y[8][E];
#pragma unroll
            for (int k = 0; k < 8; ++k)
#pragma unroll
                for (int e = 0; e < E; ++e)
                    y[k][e] = from[(i + k < here ? i + k : here - 1) * (int64_t)(RT * 16) * (D + 4) + 64 * e + lane];
#pragma unroll
            for (int k = 0; k < 8; ++k) {
                const float w = i + k < here ? __int_as_float(__builtin_amdgcn_readlane(__float_as_int(weight), i + k)) : 0.f;
#pragma unroll
                for (int e = 0; e < E; ++e) o[e] += w * y[k][e];
            }
        }
    }
    if constexpr (WAVES > 1) {
#pragma unroll
        for (int e = 0; e < E; ++e) joint[share][64 * e + lane] = o[e];
        if (lane == 0) {
            ml[share][0] = l;
            ml[share][1] = m;
        }
        __syncthreads();
        if (wave != 0) return;
        m = kAttnLowest;
        l = 0.f;
#pragma unroll
        for (int e = 0; e < E; ++e) o[e] = 0.f;
#pragma unroll
        for (int v = 0; v < WAVES; ++v) m = fmaxf(m, ml[v][1]);
#pragma unroll
        for (int v = 0; v < WAVES; ++v) {
            const float f = attn_exp2(ml[v][1] - m);
            l += f * ml[v][0];
#pragma unroll
            for (int e = 0; e < E; ++e) o[e] += f * joint[v][64 * e + lane];
        }
    }
#pragma unroll
    for (int e = 0; e < E; ++e) odd = fmaf(o[e], 0.f, odd);
    if (__any(odd != 0.f) && l - l == 0.f && step_again<InT, D>(p, b, g, x.at, x.head, qr, r, true)) return;
    const float inv = attn_inverse(l);
#pragma unroll
    for (int e = 0; e < E; ++e) orow[64 * e + lane] = (InT)(o[e] * inv);
    if (p.lse && lane == 0) p.lse[x.at * p.H + x.head] = attn_lse(m, l);
}

// Waves for a row's parts: by how many parts a unit has, at the most.
template <typename InT, int D, int RT, int WAVES>
static void run_join(const AttnParams& p, int32_t max_rows, hipStream_t stream) {
    constexpr int ROWS = WAVES > 4 ? 1 : 4 / WAVES;
    const int64_t groups = (int64_t)p.n_seqs * p.G * ((max_rows + ROWS - 1) / ROWS);
    attn_step_join_kernel<InT, D, RT, WAVES><<<dim3((uint32_t)groups), WAVES > 4 ? 64 * WAVES : 256, 0, stream>>>(p, max_rows);
}
template <typename InT, int D, int RT>
static void run_step(const AttnParams& p, int32_t max_rows, hipStream_t stream) {
    attn_step_kernel<InT, D, RT><<<dim3((uint32_t)p.workgroups), SP_THREADS, 0, stream>>>(p);
    const int64_t parts = p.workgroups / ((int64_t)p.n_seqs * p.G);
    if (parts < 12) run_join<InT, D, RT, 1>(p, max_rows, stream);
    else if (parts < 64) run_join<InT, D, RT, 4>(p, max_rows, stream);
    else run_join<InT, D, RT, 16>(p, max_rows, stream);
}
template <typename InT, int D>
static void run_rows(const AttnParams& p, int32_t max_rows, hipStream_t stream) {
    switch (step_row_tiles(max_rows)) {
        case 1: return run_step<InT, D, 1>(p, max_rows, stream);
        case 2: return run_step<InT, D, 2>(p, max_rows, stream);
        case 3: return run_step<InT, D, 3>(p, max_rows, stream);
        default: return run_step<InT, D, 4>(p, max_rows, stream);
    }
}
hipError_t launch_attn_step(const AttnParams& p, bool bf16_in, int32_t max_rows, hipStream_t stream) {
    if (bf16_in) p.D == 64 ? run_rows<__bf16, 64>(p, max_rows, stream) : run_rows<__bf16, 128>(p, max_rows, stream);
    else p.D == 64 ? run_rows<float, 64>(p, max_rows, stream) : run_rows<float, 128>(p, max_rows, stream);
    return hipGetLastError();
}

}  // namespace kda
