// Softmax attention with bf16 inputs, of whole sequences and of chunks of new
// tokens over a paged cache (gfx950).  Semantics: include/kda_attn.h.
//
// One pass over the keys with each row's running maximum m and sum l.  A
// workgroup has 128 rows of one (sequence, group), 32 per wave, and takes 64
// keys at a time: while one tile is computed with, the next one's values and
// the keys of the one behind it come from memory straight into the other half
// of LDS (no registers in between).
//   S^T = K Q^T leaves lane l with row l & 31 and keys 8 b + 4 (l >> 5) + i: the
// place of P^T as an operand of O^T = V^T P^T, whose other operand the
// transposing LDS reads give for any order of keys.  So the weights stay in
// registers, and a row's maximum and sum are one lane's values and one
// exchange with lane l ^ 32.
//   m moves only when a row's maximum has grown by more than 2^8 over it: the
// weights are then up to 2^8 instead of 1, which costs no precision (l and o
// are float32, a bf16 weight has the same relative error), and the products
// with e^{m - m'} are left out of nearly all tiles.
//   Per tile and wave 32 products (1024 cycles of the matrix cores) stand beside
// 32 exponentials and about 110 other vector instructions (about 1000 cycles),
// so both have to run at once: the products of the next tile's scores beside
// this tile's exponentials, those with the values beside the sums and the next
// tile's maximum, and another wave's beside all of them (two waves per SIMD,
// which 240 registers and 64 KB of LDS leave room for).  8192 causal tokens, 32
// heads of 128 on 8: 495 to 525 us on different machines (1.05 to 1.11 PFLOP/s);
// 2 x 4096: 261 to 272 (3% less than with a tile's scores, weights and sums one
// after the other).
#include "kda_attn_mma.h"

namespace kda {

constexpr int FW_THREADS = 256, FW_BLOCK = kAttnBlockBf16, FW_KEYS = 64;

template <int D>
struct FwdShared {
    static constexpr int TILE = FW_KEYS * 2 * D;   // bytes
    char tiles[4 * TILE];                          // keys, keys, values, values
    int32_t there[4][4];                           // of each 16 keys of four tiles: their page exists
};

// Steps of 64 keys that a block's rows see, and the position of its first token.
template <bool PAGED>
__device__ __forceinline__ int32_t fwd_steps(const AttnParams& p, const AttnBlock& b, int32_t& len, int32_t& most) {
    len = PAGED ? attn_length(p, b.n) : b.tokens;
    most = b.j < 0 ? 0 : p.causal ? len - b.tokens + (b.r1 - 1) / p.hpg + 1 : len;
    return most > 0 ? (most + FW_KEYS - 1) / FW_KEYS : 0;
}

// The rows of this wave that `odds` names once more (attn_row_again), over what has been written of them.
template <int D, bool PAGED>
__device__ __forceinline__ void fwd_again(const AttnBlock& b, int g, uint32_t odds, int32_t t0, int32_t t1, float* part) {
    const AttnParams& p = attn_params_again();
    if (!p.causal) return;
    const int lane = thread_again() & 63, wave = thread_again() >> 6;
    int32_t len, most;
    fwd_steps<PAGED>(p, b, len, most);
    const int32_t k1 = t1 * FW_KEYS < most ? t1 * FW_KEYS : most;
    asm volatile("s_waitcnt vmcnt(0)" ::: "memory");   // (written)
    for (; odds; odds &= odds - 1) {
        const int r = __builtin_ctz(odds), row = b.r0 + wave * 32 + r, t = row / p.hpg, head = g * p.hpg + row - t * p.hpg;
        float y[D / 64], m, l;
        if (!attn_row_again<__bf16, D, PAGED>(p, b.n, b.start, g, b.start + t, head, t0 * FW_KEYS, len - b.tokens + t + 1, k1, y,
                                              m, l))
            continue;
        const float inv = attn_inverse(l);
        float* to = part + (wave * 32 + r) * (D + 4);
#pragma unroll
        for (int e = 0; e < D / 64; ++e) {
            if (part) to[64 * e + lane] = y[e];
            else ((__bf16*)p.o)[((b.start + t) * p.H + head) * D + 64 * e + lane] = (__bf16)(y[e] * inv);
        }
        if (part && lane == 0) {
            to[D] = l;
            to[D + 1] = m;
        }
    }
}

// A block's rows over the steps [t0, t1) of its keys: into o and lse, or with
// `part` its sums, FW_BLOCK rows of D sums, the sum of weights, m and two unused floats.
template <int D, bool PAGED>
__device__ __forceinline__ void fwd_block(const AttnParams& p, FwdShared<D>& sh, const AttnBlock& b, int g, int32_t len,
                                          int32_t most, int32_t t0, int32_t t1, float* part) {
    constexpr int ROWB = 2 * D, UNITS = D / 8, TILE = FW_KEYS * ROWB;
    constexpr int LOADS = D / 32, RPL = 1024 / ROWB;                    // loads per wave and tile, rows of each
    constexpr int S = D / 16, O = D / 32;
    char* lds = sh.tiles;
    auto& there = sh.there;
    const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int col = lane & 31, half = lane >> 5;
    const int32_t first = len - b.tokens;                    // position of the first query token
    const int row = b.r0 + wave * 32 + col;
    const bool valid = row < b.r1;
    const int32_t t = valid ? row / p.hpg : (b.r1 - 1) / p.hpg;
    const int head = g * p.hpg + (valid ? row - t * p.hpg : 0);
    const int32_t sees = p.causal ? first + t + 1 : len;     // keys [0, sees)
    // rows come in order of their tokens; a wave without any only fetches its share of the tiles
    const int32_t sees_least = __builtin_amdgcn_readfirstlane(sees);
    const int32_t sees_most = b.r0 + wave * 32 < b.r1 ? __builtin_amdgcn_readlane(sees, 31) : 0;

    // scores are scale * q . k with scale > 0: its sign goes to q
    const float scale = p.scale < 0.f ? -p.scale : p.scale > 0.f ? p.scale : 1.f;
    const uint32_t keep = p.scale == 0.f ? 0u : ~0u, flip = p.scale < 0.f ? 0x80008000u : 0u;
    bf16x8 q[S];
    const __bf16* qrow = (const __bf16*)p.q + (b.start + t) * p.q_stride + (int64_t)head * D + 8 * half;
#pragma unroll
    for (int s = 0; s < S; ++s) {
        u32x4 w = *reinterpret_cast<const u32x4*>(qrow + 16 * s);
#pragma unroll
        for (int i = 0; i < 4; ++i) w[i] = (w[i] & keep) ^ flip;
        q[s] = __builtin_bit_cast(bf16x8, w);
    }
#pragma unroll
    for (int s = 0; s < S; ++s) arrive(q[s]);
    const float c = scale * kLog2e;

    // this wave's 16 rows of each tile
    const AttnKeys<__bf16, PAGED> keys(p, b.n, b.start, g);
    const int64_t kstep = PAGED ? D : keys.k_stride, vstep = PAGED ? D : keys.v_stride;
    uint32_t koff[LOADS], voff[LOADS];
#pragma unroll
    for (int i = 0; i < LOADS; ++i) {
        const int r = i * RPL + lane / UNITS, u = (lane % UNITS) ^ tile_swap<D>(r);
        koff[i] = (uint32_t)(r * (int)kstep * 2 + u * 16);
        voff[i] = (uint32_t)(r * (int)vstep * 2 + u * 16);
    }
    const uint32_t lds0 = (uint32_t)(uintptr_t)(__attribute__((address_space(3))) char*)lds;
    auto page_of = [&](int32_t tile) -> int32_t {
        if constexpr (PAGED) {
            const int32_t key = tile * FW_KEYS + 16 * wave;
            return key < most ? keys.pages[key >> keys.shift] : -1;
        }
        return 0;
    };
    // A tile's keys are requested two steps before its weights are formed, its
    // values one step before.
    struct Source {
        const __bf16* at;
        bool ok;
    };
    auto source = [&](const __bf16* base, int64_t step, int32_t tile, int32_t page) -> Source {
        const int32_t key = tile * FW_KEYS + 16 * wave;
        bool ok = key < most;
        int64_t at;
        if constexpr (PAGED) {
            ok = ok && page >= 0 && page < keys.n_pages;
            at = (int64_t)page * keys.k_stride + (int64_t)(key & ((1 << keys.shift) - 1)) * D;
        } else {
            at = (int64_t)key * step;
        }
        const __bf16* p0 = base + (ok ? at : 0);
        if constexpr (PAGED) p0 = in_scalars(p0);
        return Source{p0, ok};
    };
    auto request = [&](const Source& s, int64_t step, const uint32_t (&off)[LOADS], int32_t tile, int half_of) {
        const int32_t left = most - (tile * FW_KEYS + 16 * wave);
        const auto rs = make_rsrc(s.at, s.ok ? (((left < 16 ? left : 16) - 1) * (int)step + D) * 2 : 0);
        load_to_lds(rs, off, lds0 + half_of * TILE + wave * 16 * ROWB);
    };
    int32_t page_v = 0, page_raw = t0 < t1 ? page_of(t0) : 0;   // of the last keys requested; of the next ones
    auto request_keys = [&](int32_t tile, int buf) {
        page_v = PAGED ? __builtin_amdgcn_readfirstlane(page_raw) : 0;
        const Source s = source(keys.k, kstep, tile, page_v);
        if (PAGED && lane == 0) there[tile & 3][wave] = s.ok;
        request(s, kstep, koff, tile, buf);
        if (PAGED && tile + 1 < t1) page_raw = page_of(tile + 1);   // (arrives with the tile)
    };
    auto request_values = [&](int32_t tile, int buf) { request(source(keys.v, vstep, tile, page_v), vstep, voff, tile, 2 + buf); };

    // where this lane reads its operands
    const int kat = lane_rows<D>(lane);
    const int2 vat = lane_cols<D>(lane);

    f32x16 o[O];
#pragma unroll
    for (int i = 0; i < O; ++i) o[i] = zero16();
    float m = kAttnLowest, l = 0.f;

    f32x16 x[2], y[2];   // scores of this tile, of the next one
    float top = 0.f;     // the largest of x, of what nobody may see too
    auto largest = [&](const f32x16 (&x)[2]) {
        float top = x[0][0];
#pragma unroll
        for (int e = 1; e < 32; ++e) top = fmaxf(top, x[e >> 4][e & 15]);
        return top;
    };
    if (t0 < t1) {
        request_keys(t0, 0);
        tiles_barrier();
        request_values(t0, 0);
        if (t0 + 1 < t1) request_keys(t0 + 1, 1);
        x[0] = x[1] = zero16();
#pragma unroll
        for (int s = 0; s < S; ++s)
#pragma unroll
            for (int kt = 0; kt < 2; ++kt) x[kt] = mfma32x32(read_rows(lds + kt * 32 * ROWB, kat ^ (32 * s)), q[s], x[kt]);
        top = largest(x);
    }
    auto step = [&](f32x16 (&x)[2], f32x16 (&y)[2], int32_t tile, int buf) {
        tiles_barrier();
        if (tile + 1 < t1) request_values(tile + 1, buf ^ 1);
        if (tile + 2 < t1) request_keys(tile + 2, buf);
        const int32_t key0 = tile * FW_KEYS;
        if (key0 >= sees_most) return;
        const char* ks = lds + (buf ^ 1) * TILE;   // the next tile's
        const char* vs = lds + 2 * TILE + buf * TILE;
        bf16x8 kf[2][2], vf[2][O];   // operands of this product and of the next one
#pragma unroll
        for (int kt = 0; kt < 2; ++kt) kf[0][kt] = read_rows(ks + kt * 32 * ROWB, kat);
        bool whole = key0 + FW_KEYS <= sees_least;
        const int ring = tile & 3;
        if constexpr (PAGED) whole = whole && (there[ring][0] & there[ring][1] & there[ring][2] & there[ring][3]);
        if (!__builtin_amdgcn_readfirstlane(whole)) {
#pragma unroll
            for (int kt = 0; kt < 2; ++kt)
#pragma unroll
                for (int e = 0; e < 16; ++e) {
                    const int key = 32 * kt + 8 * (e >> 2) + 4 * half + (e & 3);
                    const bool seen = key0 + key < sees && (!PAGED || there[ring][2 * kt + (e >> 3)]);
                    x[kt][e] = seen ? x[kt][e] : -INFINITY;
                }
            top = largest(x);
        }
        top = fmaxf(top * c, kAttnLowest);
        if (__any(top > m + 8.f)) {
            const float to = fmaxf(m, fmaxf(top, swap_halves(top))), fade = attn_exp2(m - to);
            m = to;
            l *= fade;
#pragma unroll
            for (int i = 0; i < O; ++i)
#pragma unroll
                for (int e = 0; e < 16; ++e) o[i][e] *= fade;
        }
        // This tile's weights, beside the next one's scores on the matrix cores.  Behind the last tile those are of
        // whatever the memory holds, and nobody reads them: a branch around them cost 4% more than they do.
        y[0] = y[1] = zero16();
#pragma unroll
        for (int s = 0; s < S; ++s) {
            if (s + 1 < S) {
#pragma unroll
                for (int kt = 0; kt < 2; ++kt) kf[(s + 1) & 1][kt] = read_rows(ks + kt * 32 * ROWB, kat ^ (32 * (s + 1)));
            } else {
#pragma unroll
                for (int i = 0; i < O; ++i) vf[0][i] = read_cols(vs, vat, i);
            }
            __builtin_amdgcn_sched_barrier(0);
#pragma unroll
            for (int kt = 0; kt < 2; ++kt) y[kt] = mfma32x32(kf[s & 1][kt], q[s], y[kt]);
#pragma unroll
            for (int e = 32 / S * s; e < 32 / S * (s + 1); ++e) x[e >> 4][e & 15] = attn_exp2(fmaf(x[e >> 4][e & 15], c, -m));
            __builtin_amdgcn_sched_barrier(0);
        }
        // The values' products, beside the sums of the weights and the largest of the next scores.
        float sum[4] = {0.f, 0.f, 0.f, 0.f};
        top = y[0][0];
#pragma unroll
        for (int s = 0; s < 4; ++s) {
            if (s < 3) {
#pragma unroll
                for (int i = 0; i < O; ++i) vf[(s + 1) & 1][i] = read_cols(vs + (s + 1) * 16 * ROWB, vat, i);
            }
            __builtin_amdgcn_sched_barrier(0);
            const bf16x8 pw = as_operand(x[s >> 1], s & 1);
#pragma unroll
            for (int i = 0; i < O; ++i) o[i] = mfma32x32(vf[s & 1][i], pw, o[i]);
#pragma unroll
            for (int e = 8 * s; e < 8 * s + 8; ++e) {
                sum[e & 3] += x[e >> 4][e & 15];
                top = fmaxf(top, y[e >> 4][e & 15]);
            }
            __builtin_amdgcn_sched_barrier(0);
        }
        l += (sum[0] + sum[1]) + (sum[2] + sum[3]);
    };
    for (int32_t tile = t0; tile < t1; tile += 2) {
        step(x, y, tile, 0);
        if (tile + 1 < t1) step(y, x, tile + 1, 1);
    }
    l += swap_halves(l);
    float odd = 0.f;   // NaN if a sum is not finite
#pragma unroll
    for (int i = 0; i < O; ++i)
#pragma unroll
        for (int e = 0; e < 16; ++e) odd = fmaf(o[i][e], 0.f, odd);
    const uint64_t odds = __ballot(valid && odd != 0.f && l - l == 0.f);
    if (valid && part) {
        float* to = part + (row - b.r0) * (D + 4);
#pragma unroll
        for (int i = 0; i < O; ++i)
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                const float y[4] = {o[i][4 * k], o[i][4 * k + 1], o[i][4 * k + 2], o[i][4 * k + 3]};
                store4(to + 32 * i + 8 * k + 4 * half, y);
            }
        if (half == 0) {
            to[D] = l;
            to[D + 1] = m;
        }
    } else if (valid) {
        const float inv = attn_inverse(l);
        __bf16* orow = (__bf16*)p.o + ((b.start + t) * p.H + head) * (int64_t)D;
#pragma unroll
        for (int i = 0; i < O; ++i)
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                const float y[4] = {o[i][4 * k] * inv, o[i][4 * k + 1] * inv, o[i][4 * k + 2] * inv, o[i][4 * k + 3] * inv};
                store4(orow + 32 * i + 8 * k + 4 * half, y);
            }
        if (p.lse && half == 0) p.lse[(b.start + t) * p.H + head] = attn_lse(m, l);
    }
    if (odds) fwd_again<D, PAGED>(b, g, (uint32_t)(odds | odds >> 32), t0, t1, part);
}

template <int D, bool PAGED>
__global__ __launch_bounds__(FW_THREADS, 2) void attn_fwd_bf16_kernel(AttnParams p) {
    __shared__ __attribute__((aligned(1024))) FwdShared<D> sh;
    const AttnPlace pl = attn_place(attn_turned(blockIdx.x, gridDim.x, p.G), p.slots, p.G);
    const AttnBlock b = attn_block(p, p.slots - 1 - pl.item, p.hpg, FW_BLOCK);   // (later blocks see more keys)
    if (b.j < 0) return;
    int32_t len, most;
    const int32_t steps = fwd_steps<PAGED>(p, b, len, most);
    fwd_block<D, PAGED>(p, sh, b, pl.g, len, most, 0, steps, nullptr);
}

// Few blocks: short ones are taken whole, in turn (the lengths that decide are
// on the device only).  Over long requests the steps of all of them, in the
// order of the groups, then of the blocks, lie on one line that is cut into as
// many equal pieces as workgroups run at once.  Each workgroup finds its piece, which may
// hold the end of one block, some whole ones and the start of another; blocks
// that are cut are joined by a second launch.  Neighbouring pieces go to one
// XCD, for their common keys and values.
//   (1024 new tokens in all of two requests of 8k to 32k tokens, 32 heads of 128
// on 8: 0.81 to 0.87 PFLOP/s with the append and the joining, 309 us for 251
// GFLOP and 433 for 379.  When an input took 435, the same number of parts for
// every block took 774 us with 512 workgroups or more in all, 467 with 1024, 430
// with 2048; but 256 tokens over 32k 165, 179 and 216, 163 here.)
struct FwdLine {
    int64_t per_group, quota;   // steps
};
__device__ __forceinline__ int64_t line_piece(uint32_t w, int32_t n) { return n % 8 == 0 ? (int64_t)(w % 8) * (n / 8) + w / 8 : w; }
__device__ __forceinline__ int32_t* line_info(const AttnParams& p) { return reinterpret_cast<int32_t*>(p.part); }
// Part of a piece's first block (goes on from the piece before) or of its last one (starts in it).
template <int D>
__device__ __forceinline__ float* line_part(const AttnParams& p, int64_t piece, bool starts) {
    return p.part + ((2 * p.slots * p.G + 3) & ~(int64_t)3) + (2 * piece + starts) * (FW_BLOCK * (D + 4));
}

template <int D>
__global__ __launch_bounds__(FW_THREADS, 2) void attn_fwd_line_kernel(AttnParams p) {
    __shared__ __attribute__((aligned(1024))) FwdShared<D> sh;
    __shared__ int64_t sums[FW_THREADS / 64], found[2];
    __shared__ int32_t most_steps[FW_THREADS / 64], counts[FW_THREADS / 64];
    const int tid = threadIdx.x, lane = tid & 63;
    int32_t len, most;
    // steps before this thread's slots, of one group
    const int64_t each = (p.slots + FW_THREADS - 1) / FW_THREADS, s0 = tid * each, s1 = s0 + each < p.slots ? s0 + each : p.slots;
    int64_t mine = 0;
    int32_t longest = 0, count = 0;   // (count: blocks that have any)
    for (int64_t s = s0; s < s1; ++s) {
        const int32_t x = fwd_steps<true>(p, attn_block(p, s, p.hpg, FW_BLOCK), len, most);
        mine += x;
        longest = x > longest ? x : longest;
        count += x > 0;
    }
    int64_t up = mine;
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) {
        const int64_t y = __shfl_up(up, d);
        if (lane >= d) up += y;
        const int32_t z = __shfl_xor(longest, d);
        longest = z > longest ? z : longest;
        count += __shfl_xor(count, d);
    }
    if (lane == 63) {
        counts[tid >> 6] = count;
        sums[tid >> 6] = up;
        most_steps[tid >> 6] = longest;
    }
    __syncthreads();
    int64_t before = up - mine, total = 0;
    count = 0;
#pragma unroll
    for (int w = 0; w < FW_THREADS / 64; ++w) {
        if (w < (tid >> 6)) before += sums[w];
        total += sums[w];
        longest = most_steps[w] > longest ? most_steps[w] : longest;
        count += counts[w];
    }
    total = uniform(total);
    const int64_t units = p.slots * p.G, quota = (total * p.G + p.workgroups - 1) / p.workgroups;
    // Whole blocks where that takes no longer, in steps of two workgroups on one compute unit (2.1 us; half a round of
    // blocks takes half of that): rounds of average blocks, uneven by an eighth, or the longest one; cutting costs 30 us
    // for more starts and the parts, and 0.04 per block to join.  One request's first 1024 / 2048 / 4096 tokens, 32 heads
    // of 128 on 8: 35, 63 and 171 us whole, 57, 102 and 232 cut; 512 new tokens of each of 8 over 4096: 266 and 305; one
    // of each of 64 over 4096, packed (a round and a few blocks): 293 and 198.
    const int64_t rest = units % p.workgroups, halves = units / p.workgroups * 2 + (rest > p.workgroups / 2 ? 2 : rest > 0);
    int64_t by_blocks = count > 0 ? total * halves * 9 / (16 * (int64_t)count) : 0;
    const int64_t one = units <= p.workgroups / 2 ? longest / 2 : longest;
    by_blocks = by_blocks > one ? by_blocks : one;
    const bool cut = uniform(by_blocks) > quota + 14 + units / 50;
    const int64_t piece = line_piece(blockIdx.x, p.workgroups), begin = piece * quota;
    const int64_t end = begin + quota < total * p.G ? begin + quota : total * p.G;
    if (cut && begin >= end) return;
    int g = cut ? (int)(begin / total) : 0;
    const int64_t within = begin - g * total;
    if (cut && within >= before && within < before + mine) {
        int64_t at = before;
        for (int64_t s = s0; s < s1; ++s) {
            const int32_t x = fwd_steps<true>(p, attn_block(p, s, p.hpg, FW_BLOCK), len, most);
            if (within < at + x) {
                found[0] = s;
                found[1] = at;
                break;
            }
            at += x;
        }
    }
    __syncthreads();
    int64_t slot = cut ? uniform(found[0]) : 0, base = cut ? g * total + uniform(found[1]) : 0;   // first step of the block on the line
    for (int64_t at = cut ? begin : blockIdx.x; at < (cut ? end : units);) {   // (steps, or blocks)
        if (!cut) {
            const AttnPlace pl = attn_place(attn_zigzag((uint32_t)at, (uint32_t)units, p.G), p.slots, p.G);
            slot = p.slots - 1 - pl.item;   // (later blocks see more keys)
            g = pl.g;
        }
        AttnBlock b = attn_block(p, slot, p.hpg, FW_BLOCK);
        const int32_t steps = __builtin_amdgcn_readfirstlane(fwd_steps<true>(p, b, len, most));
        if (steps > 0) {
            // (all the same for every lane, which the compiler loses sight of)
            b.start = uniform(b.start);
            b.n = __builtin_amdgcn_readfirstlane(b.n);
            b.tokens = __builtin_amdgcn_readfirstlane(b.tokens);
            b.r0 = __builtin_amdgcn_readfirstlane(b.r0);
            b.r1 = __builtin_amdgcn_readfirstlane(b.r1);
            len = __builtin_amdgcn_readfirstlane(len);
            most = __builtin_amdgcn_readfirstlane(most);
            g = __builtin_amdgcn_readfirstlane(g);
            const int32_t t0 = __builtin_amdgcn_readfirstlane(cut ? (int32_t)(at - base) : 0);
            const int32_t t1 = __builtin_amdgcn_readfirstlane(cut && end - base < steps ? (int32_t)(end - base) : steps);
            const bool whole = t0 == 0 && t1 == steps;
            if (tid == 0) {   // for the joining: first piece (-1: nothing to join) and last
                int32_t* info = line_info(p) + 2 * (g * p.slots + slot);
                if (t0 == 0) info[0] = whole ? -1 : (int32_t)piece;
                if (t1 == steps) info[1] = (int32_t)piece;
            }
            fwd_block<D, true>(p, sh, b, g, len, most, t0, t1, whole ? nullptr : line_part<D>(p, piece, t0 == 0));
            tiles_barrier();   // (the tiles are the next block's)
            if (cut) at = base + t1;
        }
        if (!cut) {
            at += p.workgroups;
        } else if (at < end) {
            base += steps;
            if (++slot == p.slots) {
                slot = 0;
                ++g;
            }
        }
    }
}

// Rows of the blocks that were cut, and of those that see no key.  A wave has
// FW_BLOCK / 4 / LINE_JOIN rows, one after the other.
constexpr int LINE_JOIN = 8;   // workgroups per block
template <int D>
__global__ __launch_bounds__(256) void attn_fwd_line_join_kernel(AttnParams p) {
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const uint32_t unit = blockIdx.x / LINE_JOIN;
    const int64_t slot = unit % (uint32_t)p.slots;
    const int g = (int)(unit / (uint32_t)p.slots);
    const AttnBlock b = attn_block(p, slot, p.hpg, FW_BLOCK);
    if (b.j < 0) return;
    int32_t len, most, w0 = 0, w1 = -1;
    if (fwd_steps<true>(p, b, len, most) > 0) {
        w0 = line_info(p)[2 * (g * p.slots + slot)];
        w1 = line_info(p)[2 * (g * p.slots + slot) + 1];
        if (w0 < 0) return;
    }
    for (int r = (int)(blockIdx.x % LINE_JOIN) * 4 + wave; b.r0 + r < b.r1; r += 4 * LINE_JOIN) {
        float m = kAttnLowest, l = 0.f, o[D / 64] = {};
        for (int32_t w = w0; w <= w1; ++w) {
            const float* from = line_part<D>(p, w, w == w0) + r * (D + 4);
            const float to = fmaxf(m, from[D + 1]), f0 = attn_exp2(m - to), f1 = attn_exp2(from[D + 1] - to);
            m = to;
            l = l * f0 + from[D] * f1;
#pragma unroll
            for (int e = 0; e < D / 64; ++e) o[e] = o[e] * f0 + from[64 * e + lane] * f1;
        }
        const float inv = attn_inverse(l);
        const int row = b.r0 + r, t = row / p.hpg, head = g * p.hpg + row - t * p.hpg;
        __bf16* orow = (__bf16*)p.o + ((b.start + t) * p.H + head) * (int64_t)D;
#pragma unroll
        for (int e = 0; e < D / 64; ++e) orow[64 * e + lane] = (__bf16)(o[e] * inv);
        if (p.lse && lane == 0) p.lse[(b.start + t) * p.H + head] = attn_lse(m, l);
    }
}

template <int D>
static void run_fwd(const AttnParams& p, hipStream_t stream) {
    const dim3 grid((uint32_t)(p.slots * p.G));
    if (p.workgroups > 0) {
        attn_fwd_line_kernel<D><<<dim3((uint32_t)p.workgroups), FW_THREADS, 0, stream>>>(p);
        attn_fwd_line_join_kernel<D><<<dim3((uint32_t)(p.slots * p.G * LINE_JOIN)), 256, 0, stream>>>(p);
    } else if (p.lengths) {
        attn_fwd_bf16_kernel<D, true><<<grid, FW_THREADS, 0, stream>>>(p);
    } else {
        attn_fwd_bf16_kernel<D, false><<<grid, FW_THREADS, 0, stream>>>(p);
    }
}
hipError_t launch_attn_fwd_bf16(const AttnParams& p, hipStream_t stream) {
    if (p.slots == 0) return hipSuccess;
    if (p.D == 64) run_fwd<64>(p, stream);
    else run_fwd<128>(p, stream);
    return hipGetLastError();
}

}  // namespace kda
