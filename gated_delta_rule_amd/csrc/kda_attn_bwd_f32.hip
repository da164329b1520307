// Gradients of softmax attention in float32 (gfx950).  Semantics:
// include/kda_attn.h.
//
// P and dP are formed again from q, k, v, lse and grad_o, once by the blocks
// of keys (grad_k, grad_v) and once by the blocks of rows (grad_q), so that
// every sum stays in the registers of one wave: no atomics, seven products
// where five would do.  Blocks of keys walk their rows in parts where there are
// few of them; a third launch adds those in order.  Products that sum over
// the rows take S = Q K^T, whose place in registers (key l & 15, rows
// 4 (l >> 4) + i) is that of P^T as an operand of P^T dO; the one that sums
// over the keys takes S^T = K Q^T.
//   Bound as the forward pass is: 64 TFLOP/s of the formula's five products (90
// of the seven done) at 2048 causal tokens, 16 heads of 128: 382 us by the keys,
// 288 by the rows.
#include "kda_attn_mma.h"

namespace kda {

constexpr int AB_THREADS = 256, AB_BLOCK = kAttnBwdBlockF32;

// Rows of no sequence become zero in new gradients of a packed batch.
__global__ __launch_bounds__(256) void attn_bwd_rest_kernel(AttnBwdParams a, int32_t es) {
    const AttnParams& p = a.f;
    const int64_t first = attn_range(p.cu, p.rows, p.T, 0).start, last = attn_range(p.cu, p.rows, p.T, p.n_seqs - 1).end;
    const int32_t qp = p.H * p.D * es / 16, kp = p.G * p.D * es / 16, per = qp + 2 * kp;   // 16-byte pieces of a row
    const int64_t n = first + (p.rows - last);
    for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < n * per; i += (int64_t)gridDim.x * 256) {
        const int64_t at = i / per, row = at < first ? at : last + at - first;
        const int32_t c = (int32_t)(i - at * per);
        const int which = c < qp ? KDA_FRESH_Q : c < qp + kp ? KDA_FRESH_K : KDA_FRESH_V;
        if (!(a.zero_rest & which)) continue;
        char* to = which == KDA_FRESH_Q ? (char*)a.gq + row * a.gq_stride * es + (int64_t)c * 16
                 : which == KDA_FRESH_K ? (char*)a.gk + row * a.gk_stride * es + (int64_t)(c - qp) * 16
                                        : (char*)a.gv + row * a.gv_stride * es + (int64_t)(c - qp - kp) * 16;
        *reinterpret_cast<u32x4*>(to) = u32x4{0, 0, 0, 0};
    }
}
hipError_t launch_attn_bwd_rest(const AttnBwdParams& a, bool bf16_in, hipStream_t stream) {
    if (!a.f.cu || !a.zero_rest) return hipSuccess;
    attn_bwd_rest_kernel<<<kAttnRest, 256, 0, stream>>>(a, bf16_in ? 2 : 4);
    return hipGetLastError();
}

// Tiles of 16 float32 rows in LDS, 16-byte unit u of row r in place u ^ (r & 15).
template <int D>
struct F32Tile {
    static constexpr int ROWB = 4 * D, UNITS = D / 4, BYTES = 16 * ROWB, LOADS = BYTES / 1024, RPL = 1024 / ROWB;
    // row l & 15, values 16 s + 4 (l >> 4) .. + 3
    static __device__ __forceinline__ void rows(const char* tile, int col, int grp, int s, float (&x)[4]) {
        load4(reinterpret_cast<const float*>(tile + col * ROWB + ((4 * s + grp) ^ col) * 16), x);
    }
    // rows 4 (l >> 4) .. + 3, value 16 s + (l & 15)
    static __device__ __forceinline__ void cols(const char* tile, int col, int grp, int s, float (&x)[4]) {
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const int r = 4 * grp + e;
            x[e] = *reinterpret_cast<const float*>(tile + r * ROWB + ((4 * s + (col >> 2)) ^ r) * 16 + 4 * (col & 3));
        }
    }
};
// Sums of the four waves, [16][D] each, N of them, in `joint`; x: column l & 15, rows 16 s + 4 (l >> 4) .. + 3.
template <int D, int N>
__device__ __forceinline__ float* join_waves(char* lds, const f32x4 (&x)[N][D / 16]) {
    constexpr int PITCH = D + 4;
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    float* joint = reinterpret_cast<float*>(lds);
    __syncthreads();
#pragma unroll
    for (int n = 0; n < N; ++n)
#pragma unroll
        for (int s = 0; s < D / 16; ++s)
            *reinterpret_cast<f32x4*>(joint + ((wave * N + n) * 16 + (lane & 15)) * PITCH + 16 * s + 4 * (lane >> 4)) = x[n][s];
    __syncthreads();
    return joint;
}
template <int D, int N>
__device__ __forceinline__ void joint_sum(const float* joint, int n, int row, int d, float (&y)[4]) {
    constexpr int PITCH = D + 4;
#pragma unroll
    for (int e = 0; e < 4; ++e) y[e] = 0.f;
#pragma unroll
    for (int w = 0; w < 4; ++w) {
        const f32x4 z = *reinterpret_cast<const f32x4*>(joint + ((w * N + n) * 16 + row) * PITCH + d);
#pragma unroll
        for (int e = 0; e < 4; ++e) y[e] += z[e];
    }
}

// grad_k and grad_v of 16 keys of one (sequence, group): the four waves take 16
// rows each in turn, in LDS of their own, two deep, and join their sums at the
// end (as one workgroup of 64 keys whose waves share the rows, 517 tokens of 6
// heads took 72 us, with a quarter of the waves).
template <int D>
__global__ __launch_bounds__(AB_THREADS, D == 64 ? 2 : 1) void attn_bwd_kv_f32_kernel(AttnBwdParams a) {
    const AttnParams& p = a.f;
    typedef F32Tile<D> Tile;
    constexpr int S = D / 16, LOADS = Tile::LOADS, HALF = 2 * Tile::BYTES + 512;   // q, grad_o, lse and delta of 16 rows
    __shared__ __attribute__((aligned(1024))) char lds[4 * 2 * HALF];
    static_assert(4 * 2 * 16 * (D + 4) * 4 <= (int)sizeof(lds), "");
    const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6), col = lane & 15, grp = lane >> 4;
    const AttnPlace pl = attn_place(blockIdx.x, a.key_slots * a.parts, p.G);
    int64_t slot = pl.item / a.parts;
    const int part = (int)(pl.item % a.parts);
    if (!p.cu && p.causal) {   // the first blocks of all sequences, then the second ones: they have the most rows
        const int64_t each = a.key_slots / p.n_seqs;
        slot = (slot % p.n_seqs) * each + slot / p.n_seqs;
    }
    const AttnBlock b = attn_block(p, slot, 1, AB_BLOCK);
    if (b.j < 0) return;
    const int key = b.r0 + col;
    // rows [r_first, n_rows), of which this part takes whole steps of the four waves
    const int32_t all_rows = b.tokens * p.hpg, r_all = p.causal ? (int32_t)((int64_t)b.r0 * p.hpg / 16 * 16) : 0;
    const int64_t steps = ((int64_t)all_rows - r_all + 63) / 64;
    const int32_t r_first = r_all + (int32_t)(steps * part / a.parts) * 64;
    const int32_t r_end = r_all + (int32_t)(steps * (part + 1) / a.parts) * 64, n_rows = r_end < all_rows ? r_end : all_rows;
    const int64_t krow = b.start + (key < b.r1 ? key : b.r0);
    float k[S][4], v[S][4];
#pragma unroll
    for (int s = 0; s < S; ++s) {
        load4((const float*)p.k + krow * p.k_stride + (int64_t)pl.g * D + 16 * s + 4 * grp, k[s]);
        load4((const float*)p.v + krow * p.v_stride + (int64_t)pl.g * D + 16 * s + 4 * grp, v[s]);
    }
#pragma unroll
    for (int s = 0; s < S; ++s)
#pragma unroll
        for (int e = 0; e < 4; ++e) asm volatile("" : "+v"(k[s][e]), "+v"(v[s][e]));   // (arrive)
    const uint32_t lds0 = (uint32_t)(uintptr_t)(__attribute__((address_space(3))) char*)lds + wave * 2 * HALF;
    const char* own = lds + wave * 2 * HALF;
    const int64_t gstride = (int64_t)p.H * D;
    const RowOf rows(p.hpg);
    auto request = [&](int32_t r0, int buf) {
        const int32_t t0 = r0 / p.hpg, h0 = r0 - t0 * p.hpg;
        const int64_t head = (int64_t)pl.g * p.hpg;
        const auto qrs = make_rsrc((const float*)p.q + (b.start + t0) * p.q_stride + head * D, 0x40000000);
        const auto grs = make_rsrc((const float*)a.go + (b.start + t0) * gstride + head * D, 0x40000000);
        const auto lrs = make_rsrc(p.lse + (b.start + t0) * p.H + head, 0x40000000);
        const auto drs = make_rsrc(a.delta + (b.start + t0) * p.H + head, 0x40000000);
        uint32_t qoff[LOADS], goff[LOADS];
        const uint32_t to = lds0 + buf * HALF;
#pragma unroll
        for (int i = 0; i < LOADS; ++i) {
            const int r = i * Tile::RPL + lane / Tile::UNITS, u = (lane % Tile::UNITS) ^ r;
            uint32_t t, hh;
            rows.of((uint32_t)(h0 + r), t, hh);
            const uint32_t at = hh * (4 * D) + u * 16;
            const bool in = r0 + r < n_rows;                  // rows behind the last one read as zero
            qoff[i] = in ? t * (uint32_t)(p.q_stride * 4) + at : 0x80000000u;
            goff[i] = in ? t * (uint32_t)(gstride * 4) + at : 0x80000000u;
        }
        load_to_lds(qrs, qoff, to);
        load_to_lds(grs, goff, to + Tile::BYTES);
        uint32_t t, hh;
        rows.of((uint32_t)(h0 + col), t, hh);
        const uint32_t at = r0 + col < n_rows ? (t * (uint32_t)p.H + hh) * 4 : 0x80000000u;
        load4_pair_to_lds(lrs, drs, at, to + 2 * Tile::BYTES);
    };
    f32x4 g[2][S];   // grad_k, grad_v
#pragma unroll
    for (int s = 0; s < S; ++s) g[0][s] = g[1][s] = f32x4{0.f, 0.f, 0.f, 0.f};
    const float c = p.scale * kLog2e;
    const int32_t from = p.causal ? key * p.hpg : 0, from_most = p.causal ? (b.r0 + 15) * p.hpg : 0;
    const int32_t first = r_first + 16 * wave;
    if (first < n_rows) request(first, 0);
    for (int32_t r0 = first; r0 < n_rows; r0 += 64) {
        const int buf = ((r0 - first) >> 6) & 1;
        if (r0 + 64 < n_rows) {
            asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");   // (the other half has been read)
            request(r0 + 64, buf ^ 1);
            asm volatile("s_waitcnt vmcnt(%0)" ::"n"(2 * LOADS + 2) : "memory");
        } else {
            asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
        }
        const char *qs = own + buf * HALF, *gs = qs + Tile::BYTES;
        const float* stat = reinterpret_cast<const float*>(gs + Tile::BYTES);
        f32x4 x = {0.f, 0.f, 0.f, 0.f}, y = {0.f, 0.f, 0.f, 0.f};
        // operands are read one product ahead, where the fences keep them
        float zq[2][4], zg[2][4];
        Tile::rows(qs, col, grp, 0, zq[0]);
        Tile::rows(gs, col, grp, 0, zg[0]);
#pragma unroll
        for (int s = 0; s < S; ++s) {
            if (s + 1 < S) {
                Tile::rows(qs, col, grp, s + 1, zq[(s + 1) & 1]);
                Tile::rows(gs, col, grp, s + 1, zg[(s + 1) & 1]);
            } else {
                Tile::cols(qs, col, grp, 0, zq[0]);
                Tile::cols(gs, col, grp, 0, zg[0]);
            }
            __builtin_amdgcn_sched_barrier(0);
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                x = mfma4f(zq[s & 1][e], k[s][e], x);
                y = mfma4f(zg[s & 1][e], v[s][e], y);
            }
            __builtin_amdgcn_sched_barrier(0);
        }
        float lse[4], delta[4], w[4], ds[4];
        load4(stat + 4 * grp, lse);
        load4(stat + 64 + 4 * grp, delta);
        const bool some = r0 < from_most || r0 + 16 > n_rows;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int r = r0 + 4 * grp + i;
            w[i] = attn_exp2(fmaf(x[i], c, -lse[i] * kLog2e));
            if (some) w[i] = r >= from && r < n_rows ? w[i] : 0.f;
            ds[i] = w[i] * (y[i] - delta[i]);
        }
#pragma unroll
        for (int s = 0; s < S; ++s) {
            if (s + 1 < S) {
                Tile::cols(qs, col, grp, s + 1, zq[(s + 1) & 1]);
                Tile::cols(gs, col, grp, s + 1, zg[(s + 1) & 1]);
            }
            __builtin_amdgcn_sched_barrier(0);
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                g[0][s] = mfma4f(zq[s & 1][e], ds[e], g[0][s]);
                g[1][s] = mfma4f(zg[s & 1][e], w[e], g[1][s]);
            }
            __builtin_amdgcn_sched_barrier(0);
        }
    }
    const float* joint = join_waves<D, 2>(lds, g);
    const int mine = tid >> 4, d0 = (tid & 15) * 4;
    if (b.r0 + mine >= b.r1) return;
    float* tk = (float*)a.gk + (b.start + b.r0 + mine) * a.gk_stride + (int64_t)pl.g * D;
    float* tv = (float*)a.gv + (b.start + b.r0 + mine) * a.gv_stride + (int64_t)pl.g * D;
    float scale = p.scale;
    if (a.parts > 1) {
        tk = a.part + (((part * p.rows + b.start + b.r0 + mine) * p.G + pl.g) * 2) * D;
        tv = tk + D;
        scale = 1.f;
    }
#pragma unroll
    for (int n = 0; n < D / 64; ++n) {
        float z[4];
        joint_sum<D, 2>(joint, 0, mine, 64 * n + d0, z);
#pragma unroll
        for (int e = 0; e < 4; ++e) z[e] *= scale;
        store4(tk + 64 * n + d0, z);
        joint_sum<D, 2>(joint, 1, mine, 64 * n + d0, z);
        store4(tv + 64 * n + d0, z);
    }
}

// grad_q of 16 rows, the waves taking 16 keys each in turn; leaves the rows'
// delta for the blocks of keys, which run afterwards.
template <int D>
__global__ __launch_bounds__(AB_THREADS, D == 64 ? 2 : 1) void attn_bwd_q_f32_kernel(AttnBwdParams a) {
    const AttnParams& p = a.f;
    typedef F32Tile<D> Tile;
    constexpr int S = D / 16, LOADS = Tile::LOADS, HALF = 2 * Tile::BYTES;   // keys, values
    __shared__ __attribute__((aligned(1024))) char lds[4 * 2 * HALF];
    static_assert(4 * 16 * (D + 4) * 4 <= (int)sizeof(lds), "");
    const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6), col = lane & 15, grp = lane >> 4;
    const AttnPlace pl = attn_place(blockIdx.x, p.slots, p.G);
    const AttnBlock b = attn_block(p, p.slots - 1 - pl.item, p.hpg, AB_BLOCK);
    if (b.j < 0) return;
    const int row = b.r0 + col;
    const bool valid = row < b.r1;
    const int32_t t = (valid ? row : b.r1 - 1) / p.hpg;
    const int head = pl.g * p.hpg + (valid ? row - t * p.hpg : 0);
    const int64_t at = (b.start + t) * p.H + head;
    const int32_t sees = p.causal ? t + 1 : b.tokens, most = p.causal ? (b.r1 - 1) / p.hpg + 1 : b.tokens;
    const int32_t sees_least = __builtin_amdgcn_readfirstlane(sees);
    float q[S][4], go[S][4];
#pragma unroll
    for (int s = 0; s < S; ++s) {
        load4((const float*)p.q + (b.start + t) * p.q_stride + (int64_t)head * D + 16 * s + 4 * grp, q[s]);
        load4((const float*)a.go + at * D + 16 * s + 4 * grp, go[s]);
    }
    float lse2 = p.lse[at] * kLog2e, delta = 0.f;
#pragma unroll
    for (int s = 0; s < S; ++s) {
        float o[4];
        load4((const float*)p.o + at * D + 16 * s + 4 * grp, o);
#pragma unroll
        for (int e = 0; e < 4; ++e) delta += go[s][e] * o[e];
    }
    delta = groups_sum(delta);
    if (wave == 0 && grp == 0 && valid) a.delta[at] = delta;
#pragma unroll
    for (int s = 0; s < S; ++s)
#pragma unroll
        for (int e = 0; e < 4; ++e) asm volatile("" : "+v"(q[s][e]), "+v"(go[s][e]));   // (arrive)
    asm volatile("" : "+v"(lse2), "+v"(delta));
    const float c = p.scale * kLog2e;
    const AttnKeys<float, false> keys(p, b.n, b.start, pl.g);
    const uint32_t lds0 = (uint32_t)(uintptr_t)(__attribute__((address_space(3))) char*)lds + wave * 2 * HALF;
    const char* own = lds + wave * 2 * HALF;
    auto request = [&](int32_t key, int buf) {
        const int32_t left = most - key < 16 ? most - key : 16;
        const auto krs = make_rsrc(keys.k + key * keys.k_stride, ((left - 1) * (int)keys.k_stride + D) * 4);
        const auto vrs = make_rsrc(keys.v + key * keys.v_stride, ((left - 1) * (int)keys.v_stride + D) * 4);
        uint32_t koff[LOADS], voff[LOADS];
        const uint32_t to = lds0 + buf * HALF;
#pragma unroll
        for (int i = 0; i < LOADS; ++i) {
            const int r = i * Tile::RPL + lane / Tile::UNITS, u = (lane % Tile::UNITS) ^ r;
            koff[i] = (uint32_t)(r * (int)keys.k_stride * 4 + u * 16);
            voff[i] = (uint32_t)(r * (int)keys.v_stride * 4 + u * 16);
        }
        load_to_lds(krs, koff, to);
        load_to_lds(vrs, voff, to + Tile::BYTES);
    };
    f32x4 g[1][S];
#pragma unroll
    for (int s = 0; s < S; ++s) g[0][s] = f32x4{0.f, 0.f, 0.f, 0.f};
    const int32_t first = 16 * wave;
    if (first < most) request(first, 0);
    for (int32_t k0 = first; k0 < most; k0 += 64) {
        const int buf = (k0 >> 6) & 1;
        if (k0 + 64 < most) {
            asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");   // (the other half has been read)
            request(k0 + 64, buf ^ 1);
            asm volatile("s_waitcnt vmcnt(%0)" ::"n"(2 * LOADS) : "memory");
        } else {
            asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
        }
        const char *ks = own + buf * HALF, *vs = ks + Tile::BYTES;
        f32x4 x = {0.f, 0.f, 0.f, 0.f}, y = {0.f, 0.f, 0.f, 0.f};
        // (operands one product ahead, as above)
        float zk[2][4], zv[2][4];
        Tile::rows(ks, col, grp, 0, zk[0]);
        Tile::rows(vs, col, grp, 0, zv[0]);
#pragma unroll
        for (int s = 0; s < S; ++s) {
            if (s + 1 < S) {
                Tile::rows(ks, col, grp, s + 1, zk[(s + 1) & 1]);
                Tile::rows(vs, col, grp, s + 1, zv[(s + 1) & 1]);
            } else {
                Tile::cols(ks, col, grp, 0, zk[0]);
            }
            __builtin_amdgcn_sched_barrier(0);
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                x = mfma4f(zk[s & 1][e], q[s][e], x);
                y = mfma4f(zv[s & 1][e], go[s][e], y);
            }
            __builtin_amdgcn_sched_barrier(0);
        }
        float ds[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            ds[i] = attn_exp2(fmaf(x[i], c, -lse2)) * (y[i] - delta);
            if (k0 + 16 > sees_least) ds[i] = k0 + 4 * grp + i < sees ? ds[i] : 0.f;
        }
#pragma unroll
        for (int s = 0; s < S; ++s) {
            if (s + 1 < S) Tile::cols(ks, col, grp, s + 1, zk[(s + 1) & 1]);
            __builtin_amdgcn_sched_barrier(0);
            mma_k16<true, PLAIN>(g[0][s], zk[s & 1], ds);
            __builtin_amdgcn_sched_barrier(0);
        }
    }
    const float* joint = join_waves<D, 1>(lds, g);
    const int mine = b.r0 + (tid >> 4), d0 = (tid & 15) * 4;
    if (mine >= b.r1) return;
    const int32_t tm = mine / p.hpg;
    float* to = (float*)a.gq + (b.start + tm) * a.gq_stride + (int64_t)(pl.g * p.hpg + mine - tm * p.hpg) * D;
#pragma unroll
    for (int n = 0; n < D / 64; ++n) {
        float z[4];
        joint_sum<D, 1>(joint, 0, tid >> 4, 64 * n + d0, z);
#pragma unroll
        for (int e = 0; e < 4; ++e) z[e] *= p.scale;
        store4(to + 64 * n + d0, z);
    }
}

template <int D>
static void run_bwd(const AttnBwdParams& a, hipStream_t stream) {
    attn_bwd_q_f32_kernel<D><<<dim3((uint32_t)(a.f.slots * a.f.G)), AB_THREADS, 0, stream>>>(a);
    attn_bwd_kv_f32_kernel<D><<<dim3((uint32_t)(a.key_slots * a.f.G * a.parts)), AB_THREADS, 0, stream>>>(a);
    if (a.parts > 1)
        attn_bwd_join_kernel<float, D><<<dim3((uint32_t)((a.f.rows * a.f.G * (D / 2) + 255) / 256)), 256, 0, stream>>>(a);
}

hipError_t launch_attn_bwd_f32(const AttnBwdParams& a, hipStream_t stream) {
    if (a.f.rows == 0) return hipSuccess;
    const hipError_t e = launch_attn_bwd_rest(a, false, stream);
    if (e != hipSuccess) return e;
    a.f.D == 64 ? run_bwd<64>(a, stream) : run_bwd<128>(a, stream);
    return hipGetLastError();
}

}  // namespace kda
