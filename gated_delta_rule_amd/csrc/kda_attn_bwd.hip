// Gradients of softmax attention with bf16 inputs (gfx950).  Semantics:
// include/kda_attn.h.
//
// As in the float32 form, P and dP are formed twice, by the blocks of keys and
// by the blocks of rows, so that every sum stays in one wave's registers (no
// atomics).  Both kernels take 64 rows of the other side at a time, which
// come from memory straight into the other half of LDS while the half before
// is computed with:
//   keys: wave w has 32 keys and walks the rows (all heads of the group):
//     S = Q K^T, dP = dO V^T, then dV^T += dO^T P, dK^T += Q^T dS;
//   rows: wave w has 32 rows and walks the keys:
//     S^T = K Q^T, dP^T = V dO^T, then dQ^T += K^T dS^T.
// P and dS go from product to product in registers, rounded to bf16 once.
//   Bound by the matrix cores (0.46 and 0.50 busy, at 2.0 and 1.9 GHz) and by what stands between
// their products: two sums and two operands fill 192 of 256 registers, so that
// operands are read from LDS just before their turn and only the SIMD's other
// wave covers that.  2 x 4096 causal tokens, 32 heads of 128 on 8: 552 to 572 us
// by the keys, 394 to 411 by the rows on different machines, 26 to join the
// parts; 0.7 PFLOP/s of the formula's five products.  Reading operands two to four products ahead, pinned there, took 4
// to 11% longer.
#include "kda_attn_mma.h"

namespace kda {

constexpr int BW_THREADS = 256, BW_BLOCK = kAttnBlockBf16, BW_STEP = 64;

// grad_k and grad_v of 128 keys of one (sequence, group).
template <int D>
__global__ __launch_bounds__(BW_THREADS, 2) void attn_bwd_kv_kernel(AttnBwdParams a) {
    const AttnParams& p = a.f;
    constexpr int ROWB = 2 * D, UNITS = D / 8, TILE = BW_STEP * ROWB, LOADS = D / 32, RPL = 1024 / ROWB;
    constexpr int S = D / 16, O = D / 32;
    __shared__ __attribute__((aligned(1024))) char lds[4 * TILE];   // q, q, grad_o, grad_o
    __shared__ __attribute__((aligned(16))) float stat[2][2][BW_STEP];   // of each row: lse in base 2, -delta
    const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const AttnPlace pl = attn_place(attn_zigzag(blockIdx.x, gridDim.x, p.G), a.key_slots * a.parts, p.G);
    int64_t slot = pl.item / a.parts;
    const int part = (int)(pl.item % a.parts);
    if (!p.cu && p.causal) {   // the first blocks of all sequences, then the second ones: they have the most rows
        const int64_t each = a.key_slots / p.n_seqs;
        slot = (slot % p.n_seqs) * each + slot / p.n_seqs;
    }
    const AttnBlock b = attn_block(p, slot, 1, BW_BLOCK);
    if (b.j < 0) return;
    const int32_t key0 = b.r0 + wave * 32;   // this wave's first key

    bf16x8 k[S], v[S];
    {
        const int key = key0 + (lane & 31);
        const int64_t row = b.start + (key < b.r1 ? key : b.r0);
        const __bf16* kr = (const __bf16*)p.k + row * p.k_stride + (int64_t)pl.g * D + 8 * (lane >> 5);
        const __bf16* vr = (const __bf16*)p.v + row * p.v_stride + (int64_t)pl.g * D + 8 * (lane >> 5);
#pragma unroll
        for (int s = 0; s < S; ++s) {
            k[s] = *reinterpret_cast<const bf16x8*>(kr + 16 * s);
            v[s] = *reinterpret_cast<const bf16x8*>(vr + 16 * s);
        }
#pragma unroll
        for (int s = 0; s < S; ++s) {
            arrive(k[s]);
            arrive(v[s]);
        }
    }
    f32x16 gk[O], gv[O];
#pragma unroll
    for (int i = 0; i < O; ++i) gk[i] = gv[i] = zero16();

    const float c = p.scale * kLog2e;
    // rows [r_first, n_rows), of which this part takes whole steps
    const int32_t all_rows = b.tokens * p.hpg, r_all = p.causal ? (int32_t)((int64_t)b.r0 * p.hpg / BW_STEP * BW_STEP) : 0;
    const int64_t steps = ((int64_t)all_rows - r_all + BW_STEP - 1) / BW_STEP;
    const int32_t r_first = r_all + (int32_t)(steps * part / a.parts) * BW_STEP;
    const int32_t r_end = r_all + (int32_t)(steps * (part + 1) / a.parts) * BW_STEP, n_rows = r_end < all_rows ? r_end : all_rows;
    // key x is seen by the rows from x * hpg on
    // (a wave without keys only fetches)
    const int32_t from_least = key0 >= b.r1 ? INT32_MAX : p.causal ? key0 * p.hpg : 0, from_most = p.causal ? (key0 + 31) * p.hpg : 0;
    const uint32_t lds0 = (uint32_t)(uintptr_t)(__attribute__((address_space(3))) char*)lds;
    const int64_t gstride = (int64_t)p.H * D;
    const RowOf rows(p.hpg);
    float mine = 0.f;
    auto request = [&](int32_t r0, int buf) {
        const int32_t t0 = r0 / p.hpg, h0 = r0 - t0 * p.hpg;                  // first row of the tile
        const auto qrs = make_rsrc((const __bf16*)p.q + (b.start + t0) * p.q_stride + (int64_t)pl.g * p.hpg * D, 0x40000000);
        const auto grs = make_rsrc((const __bf16*)a.go + (b.start + t0) * gstride + (int64_t)pl.g * p.hpg * D, 0x40000000);
        const uint32_t to = lds0 + buf * TILE + wave * 16 * ROWB;
        int ln = lane;
        hide(ln);   // (offsets are formed anew: there are no registers to keep them)
#pragma unroll
        for (int i = 0; i < LOADS; ++i) {
            const int r = wave * 16 + i * RPL + ln / UNITS, u = (ln % UNITS) ^ tile_swap<D>(r);
            uint32_t t, hh;
            rows.of((uint32_t)(h0 + r), t, hh);
            const uint32_t at = hh * (2 * D) + u * 16;
            const bool in = r0 + r < n_rows;                                  // rows behind the last one read as zero
            load_pair_to_lds(qrs, in ? t * (uint32_t)(p.q_stride * 2) + at : 0x80000000u,
                             grs, in ? t * (uint32_t)(gstride * 2) + at : 0x80000000u, to + i * 1024, 2 * TILE);
        }
        if (tid < 2 * BW_STEP) {
            const int r = tid & (BW_STEP - 1);
            uint32_t t, hh;
            rows.of((uint32_t)(h0 + r), t, hh);
            if (r0 + r < n_rows) mine = (tid < BW_STEP ? p.lse : a.delta)[(b.start + t0 + t) * p.H + pl.g * p.hpg + hh];
        }
    };
    if (r_first < n_rows) request(r_first, 0);
    for (int32_t r0 = r_first; r0 < n_rows; r0 += BW_STEP) {
        const int buf = ((r0 - r_first) / BW_STEP) & 1;
        if (tid < 2 * BW_STEP) {   // (a row that is not there has weight e^{-inf})
            const int r = tid & (BW_STEP - 1);
            stat[buf][tid / BW_STEP][r] = tid < BW_STEP ? (r0 + r < n_rows ? mine * kLog2e : INFINITY) : -mine;
        }
        tiles_barrier();
        if (r0 + BW_STEP < n_rows) request(r0 + BW_STEP, buf ^ 1);
        if (r0 + BW_STEP <= from_least) continue;
        const char* qs = lds + buf * TILE;
        const char* gs = lds + 2 * TILE + buf * TILE;
#pragma unroll
        for (int rt = 0; rt < 2; ++rt) {
            const char *qt = qs + rt * 32 * ROWB, *gt = gs + rt * 32 * ROWB;
            int ln = lane;
            hide(ln);   // (nor any for these)
            const int half = ln >> 5, rat = lane_rows<D>(ln);
            const int2 cat = lane_cols<D>(ln);
            f32x16 x = zero16();
#pragma unroll
            for (int s = 0; s < S; ++s) x = mfma32x32(read_rows(qt, rat ^ (32 * s)), k[s], x);
#pragma unroll
            for (int e4 = 0; e4 < 4; ++e4) {
                const f32x4 lse2 = *reinterpret_cast<const f32x4*>(&stat[buf][0][32 * rt + 8 * e4 + 4 * half]);
#pragma unroll
                for (int i = 0; i < 4; ++i) x[4 * e4 + i] = attn_exp2(fmaf(x[4 * e4 + i], c, -lse2[i]));
            }
            if (r0 + 32 * rt < from_most) {
                const int32_t from = (key0 + (ln & 31)) * p.hpg;
#pragma unroll
                for (int e = 0; e < 16; ++e)
                    x[e] = r0 + 32 * rt + 8 * (e >> 2) + 4 * half + (e & 3) >= from ? x[e] : 0.f;
            }
            __builtin_amdgcn_sched_barrier(0);   // (registers: 192 of 256 are sums, keys and values)
#pragma unroll
            for (int s = 0; s < 2; ++s) {
                const bf16x8 pw = as_operand(x, s);
#pragma unroll
                for (int i = 0; i < O; ++i) gv[i] = mfma32x32(read_cols(gt + s * 16 * ROWB, cat, i), pw, gv[i]);
                __builtin_amdgcn_sched_barrier(0);
            }
            f32x16 y;   // dP - delta
#pragma unroll
            for (int e4 = 0; e4 < 4; ++e4) {
                const f32x4 less = *reinterpret_cast<const f32x4*>(&stat[buf][1][32 * rt + 8 * e4 + 4 * half]);
#pragma unroll
                for (int i = 0; i < 4; ++i) y[4 * e4 + i] = less[i];
            }
#pragma unroll
            for (int s = 0; s < S; ++s) {
                y = mfma32x32(read_rows(gt, rat ^ (32 * s)), v[s], y);
                if (s % 4 == 3) __builtin_amdgcn_sched_barrier(0);
            }
#pragma unroll
            for (int e = 0; e < 16; ++e) x[e] *= y[e];
            __builtin_amdgcn_sched_barrier(0);
#pragma unroll
            for (int s = 0; s < 2; ++s) {
                const bf16x8 ds = as_operand(x, s);
#pragma unroll
                for (int i = 0; i < O; ++i) gk[i] = mfma32x32(read_cols(qt + s * 16 * ROWB, cat, i), ds, gk[i]);
                __builtin_amdgcn_sched_barrier(0);
            }
        }
    }
    const int key = key0 + (lane & 31), half = lane >> 5;
    if (key >= b.r1) return;
    if (a.parts > 1) {
        float* to = a.part + (((part * p.rows + b.start + key) * p.G + pl.g) * 2) * D + 4 * half;
#pragma unroll
        for (int i = 0; i < O; ++i)
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const float y[4] = {gk[i][4 * e], gk[i][4 * e + 1], gk[i][4 * e + 2], gk[i][4 * e + 3]};
                const float z[4] = {gv[i][4 * e], gv[i][4 * e + 1], gv[i][4 * e + 2], gv[i][4 * e + 3]};
                store4(to + 32 * i + 8 * e, y);
                store4(to + D + 32 * i + 8 * e, z);
            }
        return;
    }
    __bf16* tk = (__bf16*)a.gk + (b.start + key) * a.gk_stride + (int64_t)pl.g * D + 4 * half;
    __bf16* tv = (__bf16*)a.gv + (b.start + key) * a.gv_stride + (int64_t)pl.g * D + 4 * half;
#pragma unroll
    for (int i = 0; i < O; ++i)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            float y[4], z[4];
#pragma unroll
            for (int n = 0; n < 4; ++n) {
                y[n] = gk[i][4 * e + n] * p.scale;
                z[n] = gv[i][4 * e + n];
            }
            store4(tk + 32 * i + 8 * e, y);
            store4(tv + 32 * i + 8 * e, z);
        }
}

// grad_q of 128 rows of one (sequence, group); leaves the rows' delta for the
// blocks of keys, which run afterwards.  A row's dS add up to 0 with the exact
// delta; with the one from o, which is rounded, to the difference.  So the
// blocks of keys get delta + sum_j dS_ij: grad_k is off by 2.4e-3 of its norm
// instead of 2.8e-3 for sequences of 64 tokens (the rounding of dS and its own
// make up 2.35e-3), for 1.3% of the backward pass's time.
template <int D>
__global__ __launch_bounds__(BW_THREADS, 2) void attn_bwd_q_kernel(AttnBwdParams a) {
    const AttnParams& p = a.f;
    constexpr int ROWB = 2 * D, UNITS = D / 8, TILE = BW_STEP * ROWB, LOADS = D / 32, RPL = 1024 / ROWB;
    constexpr int S = D / 16, O = D / 32;
    __shared__ __attribute__((aligned(1024))) char lds[4 * TILE];   // keys, keys, values, values
    const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int col = lane & 31, half = lane >> 5;
    const AttnPlace pl = attn_place(attn_turned(blockIdx.x, gridDim.x, p.G), p.slots, p.G);
    const AttnBlock b = attn_block(p, p.slots - 1 - pl.item, p.hpg, BW_BLOCK);   // (later blocks see more keys)
    if (b.j < 0) return;
    const int row = b.r0 + wave * 32 + col;
    const bool valid = row < b.r1;
    const int32_t t = (valid ? row : b.r1 - 1) / p.hpg;
    const int head = pl.g * p.hpg + (valid ? row - t * p.hpg : 0);
    const int64_t at = (b.start + t) * p.H + head;
    const int32_t sees = p.causal ? t + 1 : b.tokens, most = p.causal ? (b.r1 - 1) / p.hpg + 1 : b.tokens;
    const int32_t sees_least = __builtin_amdgcn_readfirstlane(sees);
    const int32_t sees_most = b.r0 + wave * 32 < b.r1 ? __builtin_amdgcn_readlane(sees, 31) : 0;   // (a wave without rows only fetches)

    bf16x8 q[S], go[S];
    {
        const __bf16* qr = (const __bf16*)p.q + (b.start + t) * p.q_stride + (int64_t)head * D + 8 * half;
        const __bf16* gr = (const __bf16*)a.go + at * D + 8 * half;
#pragma unroll
        for (int s = 0; s < S; ++s) {
            q[s] = *reinterpret_cast<const bf16x8*>(qr + 16 * s);
            go[s] = *reinterpret_cast<const bf16x8*>(gr + 16 * s);
        }
#pragma unroll
        for (int s = 0; s < S; ++s) {
            arrive(q[s]);
            arrive(go[s]);
        }
    }
    float lse2 = p.lse[at] * kLog2e, delta = 0.f;
#pragma unroll
    for (int s = 0; s < S; ++s) {
        float x[4], y[4];
        const __bf16* o = (const __bf16*)p.o + at * D + 16 * s + 8 * half;
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            load4(o + 4 * e, x);
            load4((const __bf16*)a.go + at * D + 16 * s + 8 * half + 4 * e, y);
#pragma unroll
            for (int k = 0; k < 4; ++k) delta += x[k] * y[k];
        }
    }
    delta += swap_halves(delta);
    asm volatile("" : "+v"(lse2), "+v"(delta));   // (arrive, too)
    const float c = p.scale * kLog2e;
    f32x16 gq[O];
    float rest[4] = {0.f, 0.f, 0.f, 0.f};   // sums of the row's dS
#pragma unroll
    for (int i = 0; i < O; ++i) gq[i] = zero16();

    const AttnKeys<__bf16, false> keys(p, b.n, b.start, pl.g);
    uint32_t koff[LOADS], voff[LOADS];
#pragma unroll
    for (int i = 0; i < LOADS; ++i) {
        const int r = i * RPL + lane / UNITS, u = (lane % UNITS) ^ tile_swap<D>(r);
        koff[i] = (uint32_t)(r * (int)keys.k_stride * 2 + u * 16);
        voff[i] = (uint32_t)(r * (int)keys.v_stride * 2 + u * 16);
    }
    const uint32_t lds0 = (uint32_t)(uintptr_t)(__attribute__((address_space(3))) char*)lds;
    auto request = [&](int32_t tile, int buf) {
        const int32_t key = tile * BW_STEP + 16 * wave;
        const int32_t left = most - key < 16 ? most - key : 16;
        const int64_t first = left > 0 ? key : 0;
        const auto krs = make_rsrc(keys.k + first * keys.k_stride, left > 0 ? ((left - 1) * (int)keys.k_stride + D) * 2 : 0);
        const auto vrs = make_rsrc(keys.v + first * keys.v_stride, left > 0 ? ((left - 1) * (int)keys.v_stride + D) * 2 : 0);
        const uint32_t to = lds0 + buf * TILE + wave * 16 * ROWB;
        // (single loads: 411 us at 2 x 4096 tokens, 32 heads of 128 on 8; as two blocks 419, the compiler puts products between these)
#pragma unroll
        for (int i = 0; i < LOADS; ++i) load_to_lds(krs, koff[i], to + i * 1024);
#pragma unroll
        for (int i = 0; i < LOADS; ++i) load_to_lds(vrs, voff[i], to + 2 * TILE + i * 1024);
    };
    const int rat = lane_rows<D>(lane);
    const int2 cat = lane_cols<D>(lane);
    const int32_t tiles = (most + BW_STEP - 1) / BW_STEP;
    request(0, 0);
    for (int32_t tile = 0; tile < tiles; ++tile) {
        const int buf = tile & 1;
        tiles_barrier();
        if (tile + 1 < tiles) request(tile + 1, buf ^ 1);
        const int32_t key0 = tile * BW_STEP;
        if (key0 >= sees_most) continue;
        const char* ks = lds + buf * TILE;
        const char* vs = lds + 2 * TILE + buf * TILE;
#pragma unroll
        for (int kt = 0; kt < 2; ++kt) {
            f32x16 x = zero16(), y = zero16();
#pragma unroll
            for (int s = 0; s < S; ++s) {
                x = mfma32x32(read_rows(ks + kt * 32 * ROWB, rat ^ (32 * s)), q[s], x);
                y = mfma32x32(read_rows(vs + kt * 32 * ROWB, rat ^ (32 * s)), go[s], y);
            }
#pragma unroll
            for (int e = 0; e < 16; ++e) x[e] = attn_exp2(fmaf(x[e], c, -lse2)) * (y[e] - delta);
            if (key0 + 32 * kt + 32 > sees_least) {
#pragma unroll
                for (int e = 0; e < 16; ++e)
                    x[e] = key0 + 32 * kt + 8 * (e >> 2) + 4 * half + (e & 3) < sees ? x[e] : 0.f;
            }
#pragma unroll
            for (int e = 0; e < 16; ++e) rest[e & 3] += x[e];
#pragma unroll
            for (int s = 0; s < 2; ++s) {
                const bf16x8 ds = as_operand(x, s);
#pragma unroll
                for (int i = 0; i < O; ++i) gq[i] = mfma32x32(read_cols(ks + (2 * kt + s) * 16 * ROWB, cat, i), ds, gq[i]);
            }
        }
    }
    float off = (rest[0] + rest[1]) + (rest[2] + rest[3]);
    off += swap_halves(off);
    if (!valid) return;
    if (half == 0) a.delta[at] = delta + off;
    __bf16* to = (__bf16*)a.gq + (b.start + t) * a.gq_stride + (int64_t)head * D + 4 * half;
#pragma unroll
    for (int i = 0; i < O; ++i)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            float y[4];
#pragma unroll
            for (int n = 0; n < 4; ++n) y[n] = gq[i][4 * e + n] * p.scale;
            store4(to + 32 * i + 8 * e, y);
        }
}

template <int D>
static void run_bwd(const AttnBwdParams& a, hipStream_t stream) {
    attn_bwd_q_kernel<D><<<dim3((uint32_t)(a.f.slots * a.f.G)), BW_THREADS, 0, stream>>>(a);
    attn_bwd_kv_kernel<D><<<dim3((uint32_t)(a.key_slots * a.f.G * a.parts)), BW_THREADS, 0, stream>>>(a);
    if (a.parts > 1)
        attn_bwd_join_kernel<__bf16, D><<<dim3((uint32_t)((a.f.rows * a.f.G * (D / 2) + 255) / 256)), 256, 0, stream>>>(a);
}

hipError_t launch_attn_bwd_bf16(const AttnBwdParams& a, hipStream_t stream) {
    if (a.f.rows == 0) return hipSuccess;
    const hipError_t e = launch_attn_bwd_rest(a, true, stream);
    if (e != hipSuccess) return e;
    if (a.f.D == 64) run_bwd<64>(a, stream);
    else run_bwd<128>(a, stream);
    return hipGetLastError();
}

}  // namespace kda
