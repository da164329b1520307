// Gradients of softmax attention in float32 (gfx950).  Semantics:
// include/kda_attn.h.
//
// P and dP are formed again from q, k, v, lse and grad_o, once by the blocks
// of keys (grad_k, grad_v) and once by the blocks of rows (grad_q), so that
// every sum stays in the registers of one wave: no atomics, no arrays of
// partial sums, seven products where five would do.  Products that sum over
// the rows take S = Q K^T, whose place in registers (key l & 15, rows
// 4 (l >> 4) + i) is that of P^T as an operand of P^T dO; the one that sums
// over the keys takes S^T = K Q^T.
#include "kda_attn_tile.h"

namespace kda {

constexpr int AB_THREADS = 256, AB_ROWS = 32, AB_BLOCK = 64;

// delta of every row; rows of no sequence become zero in new gradients.
template <typename InT, int D>
__global__ __launch_bounds__(256) void attn_delta_kernel(AttnBwdParams a) {
    const AttnParams& p = a.f;
    constexpr int EV = 16 / (int)sizeof(InT), LANES = D / EV;   // lanes of a row
    const int64_t i = ((int64_t)blockIdx.x * 256 + threadIdx.x) / LANES;
    const int c = (threadIdx.x % LANES) * EV;
    if (i >= p.rows * p.H) return;   // (whole rows: LANES divides 64)
    const int64_t row = i / p.H;
    const int h = (int)(i - row * p.H);
    if (p.cu) {
        const bool in = row >= attn_range(p.cu, p.rows, p.T, 0).start && row < attn_range(p.cu, p.rows, p.T, p.n_seqs - 1).end;
        if (!in) {
            const u32x4 z = {0, 0, 0, 0};
            if (a.zero_rest & KDA_FRESH_Q) *reinterpret_cast<u32x4*>((InT*)a.gq + row * a.gq_stride + (int64_t)h * D + c) = z;
            if (h % p.hpg == 0) {
                const int64_t g = (int64_t)(h / p.hpg) * D + c;
                if (a.zero_rest & KDA_FRESH_K) *reinterpret_cast<u32x4*>((InT*)a.gk + row * a.gk_stride + g) = z;
                if (a.zero_rest & KDA_FRESH_V) *reinterpret_cast<u32x4*>((InT*)a.gv + row * a.gv_stride + g) = z;
            }
            return;
        }
    }
    float s = 0.f;
#pragma unroll
    for (int e = 0; e < EV; e += 4) {
        float x[4], y[4];
        load4((const InT*)p.o + i * D + c + e, x);
        load4((const InT*)a.go + i * D + c + e, y);
#pragma unroll
        for (int k = 0; k < 4; ++k) s += x[k] * y[k];
    }
#pragma unroll
    for (int d = 1; d < LANES; d <<= 1) s += __shfl_xor(s, d);
    if (threadIdx.x % LANES == 0) a.delta[i] = s;
}

// grad_k and grad_v of 64 keys (16 per wave) of one (sequence, group), over
// 32 rows at a time.
template <typename InT, int D>
__global__ __launch_bounds__(AB_THREADS) void attn_bwd_kv_f32_kernel(AttnBwdParams a) {
    const AttnParams& p = a.f;
    constexpr int PITCH = D + 4, S = D / 16, PER = D / 8;
    __shared__ __attribute__((aligned(16))) float qs[AB_ROWS * PITCH], gs[AB_ROWS * PITCH];
    __shared__ float lse2[AB_ROWS], delta[AB_ROWS];
    __shared__ int32_t from[AB_ROWS];   // a row sees keys up to this one
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6, col = lane & 15, grp = lane >> 4;
    const AttnPlace pl = attn_place(blockIdx.x, a.key_slots, p.G);
    const AttnBlock b = attn_block(p, pl.item, 1, AB_BLOCK);
    if (b.j < 0) return;
    const int key = b.r0 + wave * 16 + col;
    const bool valid = key < b.r1;
    const int32_t n_rows = b.tokens * p.hpg;
    const int64_t krow = b.start + (valid ? key : b.r0);
    float k[S][4], v[S][4];
#pragma unroll
    for (int s = 0; s < S; ++s) {
        load4((const InT*)p.k + krow * p.k_stride + (int64_t)pl.g * D + 16 * s + 4 * grp, k[s]);
        load4((const InT*)p.v + krow * p.v_stride + (int64_t)pl.g * D + 16 * s + 4 * grp, v[s]);
    }
    f32x4 gk[S], gv[S];
#pragma unroll
    for (int s = 0; s < S; ++s) gk[s] = gv[s] = f32x4{0.f, 0.f, 0.f, 0.f};
    const float c = p.scale * kLog2e;
    const int32_t r_first = p.causal ? b.r0 * p.hpg / AB_ROWS * AB_ROWS : 0;
    for (int32_t r0 = r_first; r0 < n_rows; r0 += AB_ROWS) {
        __syncthreads();
        {
            const int row = r0 + (tid >> 3), cc = (tid & 7) * 4;
            const bool in = row < n_rows;
            const int32_t t = in ? row / p.hpg : 0;
            const int64_t at = (b.start + t) * p.H + pl.g * p.hpg + (in ? row - t * p.hpg : 0);
            const InT* qr = (const InT*)p.q + (b.start + t) * p.q_stride + (int64_t)(at - (b.start + t) * p.H) * D;
#pragma unroll
            for (int i = 0; i < PER / 4; ++i) {
                float x[4] = {0.f, 0.f, 0.f, 0.f}, y[4] = {0.f, 0.f, 0.f, 0.f};
                if (in) {
                    load4(qr + cc + 32 * i, x);
                    load4((const InT*)a.go + at * D + cc + 32 * i, y);
                }
                *reinterpret_cast<f32x4*>(qs + (tid >> 3) * PITCH + cc + 32 * i) = f32x4{x[0], x[1], x[2], x[3]};
                *reinterpret_cast<f32x4*>(gs + (tid >> 3) * PITCH + cc + 32 * i) = f32x4{y[0], y[1], y[2], y[3]};
            }
            if ((tid & 7) == 0) {
                lse2[tid >> 3] = in ? p.lse[at] * kLog2e : 0.f;
                delta[tid >> 3] = in ? a.delta[at] : 0.f;
                from[tid >> 3] = !in ? -1 : p.causal ? t : b.tokens;
            }
        }
        __syncthreads();
#pragma unroll
        for (int rt = 0; rt < 2; ++rt) {
            f32x4 sc = {0.f, 0.f, 0.f, 0.f}, dp = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
            for (int s = 0; s < S; ++s) {
                float x[4];
                load4(qs + (16 * rt + col) * PITCH + 16 * s + 4 * grp, x);
                mma_k16<true, PLAIN>(sc, x, k[s]);
                load4(gs + (16 * rt + col) * PITCH + 16 * s + 4 * grp, x);
                mma_k16<true, PLAIN>(dp, x, v[s]);
            }
            float w[4], ds[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int r = 16 * rt + 4 * grp + i;
                w[i] = valid && key <= from[r] ? attn_exp2(sc[i] * c - lse2[r]) : 0.f;
                ds[i] = w[i] * (dp[i] - delta[r]);
            }
#pragma unroll
            for (int s = 0; s < S; ++s) {
                float x[4], y[4];
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    x[e] = gs[(16 * rt + 4 * grp + e) * PITCH + 16 * s + col];
                    y[e] = qs[(16 * rt + 4 * grp + e) * PITCH + 16 * s + col];
                }
                mma_k16<true, PLAIN>(gv[s], w, x);
                mma_k16<true, PLAIN>(gk[s], ds, y);
            }
        }
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int mine = b.r0 + wave * 16 + 4 * grp + i;
        if (mine < b.r1) {
            InT* tk = (InT*)a.gk + (b.start + mine) * a.gk_stride + (int64_t)pl.g * D;
            InT* tv = (InT*)a.gv + (b.start + mine) * a.gv_stride + (int64_t)pl.g * D;
#pragma unroll
            for (int s = 0; s < S; ++s) {
                tk[16 * s + col] = (InT)(gk[s][i] * p.scale);
                tv[16 * s + col] = (InT)gv[s][i];
            }
        }
    }
}

// grad_q of 64 rows (16 per wave), over 32 keys at a time.
template <typename InT, int D>
__global__ __launch_bounds__(AB_THREADS) void attn_bwd_q_f32_kernel(AttnBwdParams a) {
    const AttnParams& p = a.f;
    constexpr int PITCH = D + 4, S = D / 16, PER = D / 8;
    __shared__ __attribute__((aligned(16))) float ks[AB_ROWS * PITCH], vs[AB_ROWS * PITCH];
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6, col = lane & 15, grp = lane >> 4;
    const AttnPlace pl = attn_place(blockIdx.x, p.slots, p.G);
    const AttnBlock b = attn_block(p, p.slots - 1 - pl.item, p.hpg, AB_BLOCK);
    if (b.j < 0) return;
    const int row = b.r0 + wave * 16 + col;
    const bool valid = row < b.r1;
    const int32_t t = valid ? row / p.hpg : 0;
    const int head = pl.g * p.hpg + (valid ? row - t * p.hpg : 0);
    const int64_t at = (b.start + t) * p.H + head;
    const int32_t sees = !valid ? 0 : p.causal ? t + 1 : b.tokens;
    const int32_t most = p.causal ? (b.r1 - 1) / p.hpg + 1 : b.tokens;
    float q[S][4], go[S][4];
#pragma unroll
    for (int s = 0; s < S; ++s) {
        load4((const InT*)p.q + (b.start + t) * p.q_stride + (int64_t)head * D + 16 * s + 4 * grp, q[s]);
        load4((const InT*)a.go + at * D + 16 * s + 4 * grp, go[s]);
    }
    const float lse2 = p.lse[at] * kLog2e, delta = a.delta[at], c = p.scale * kLog2e;
    f32x4 gq[S];
#pragma unroll
    for (int s = 0; s < S; ++s) gq[s] = f32x4{0.f, 0.f, 0.f, 0.f};
    for (int32_t k0 = 0; k0 < most; k0 += AB_ROWS) {
        __syncthreads();
        {
            const int key = k0 + (tid >> 3), cc = (tid & 7) * 4;
#pragma unroll
            for (int i = 0; i < PER / 4; ++i) {
                float x[4] = {0.f, 0.f, 0.f, 0.f}, y[4] = {0.f, 0.f, 0.f, 0.f};
                if (key < most) {
                    load4((const InT*)p.k + (b.start + key) * p.k_stride + (int64_t)pl.g * D + cc + 32 * i, x);
                    load4((const InT*)p.v + (b.start + key) * p.v_stride + (int64_t)pl.g * D + cc + 32 * i, y);
                }
                *reinterpret_cast<f32x4*>(ks + (tid >> 3) * PITCH + cc + 32 * i) = f32x4{x[0], x[1], x[2], x[3]};
                *reinterpret_cast<f32x4*>(vs + (tid >> 3) * PITCH + cc + 32 * i) = f32x4{y[0], y[1], y[2], y[3]};
            }
        }
        __syncthreads();
#pragma unroll
        for (int kt = 0; kt < 2; ++kt) {
            f32x4 sc = {0.f, 0.f, 0.f, 0.f}, dp = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
            for (int s = 0; s < S; ++s) {
                float x[4];
                load4(ks + (16 * kt + col) * PITCH + 16 * s + 4 * grp, x);
                mma_k16<true, PLAIN>(sc, x, q[s]);
                load4(vs + (16 * kt + col) * PITCH + 16 * s + 4 * grp, x);
                mma_k16<true, PLAIN>(dp, x, go[s]);
            }
            float ds[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const bool seen = k0 + 16 * kt + 4 * grp + i < sees;
                ds[i] = seen ? attn_exp2(sc[i] * c - lse2) * (dp[i] - delta) : 0.f;
            }
#pragma unroll
            for (int s = 0; s < S; ++s) {
                float x[4];
#pragma unroll
                for (int e = 0; e < 4; ++e) x[e] = ks[(16 * kt + 4 * grp + e) * PITCH + 16 * s + col];
                mma_k16<true, PLAIN>(gq[s], x, ds);
            }
        }
    }
    if (!valid) return;
    InT* to = (InT*)a.gq + (b.start + t) * a.gq_stride + (int64_t)head * D;
#pragma unroll
    for (int s = 0; s < S; ++s) {
        const float y[4] = {gq[s][0] * p.scale, gq[s][1] * p.scale, gq[s][2] * p.scale, gq[s][3] * p.scale};
        store4(to + 16 * s + 4 * grp, y);
    }
}

template <typename InT, int D>
static void run_delta(const AttnBwdParams& a, hipStream_t stream) {
    constexpr int LANES = D / (16 / (int)sizeof(InT));
    attn_delta_kernel<InT, D><<<dim3((uint32_t)((a.f.rows * a.f.H * LANES + 255) / 256)), 256, 0, stream>>>(a);
}
hipError_t launch_attn_delta(const AttnBwdParams& a, bool bf16_in, hipStream_t stream) {
    if (bf16_in) a.f.D == 64 ? run_delta<__bf16, 64>(a, stream) : run_delta<__bf16, 128>(a, stream);
    else a.f.D == 64 ? run_delta<float, 64>(a, stream) : run_delta<float, 128>(a, stream);
    return hipGetLastError();
}

template <typename InT, int D>
static void run_bwd(const AttnBwdParams& a, hipStream_t stream) {
    attn_bwd_kv_f32_kernel<InT, D><<<dim3((uint32_t)(a.key_slots * a.f.G)), AB_THREADS, 0, stream>>>(a);
    attn_bwd_q_f32_kernel<InT, D><<<dim3((uint32_t)(a.f.slots * a.f.G)), AB_THREADS, 0, stream>>>(a);
}

hipError_t launch_attn_bwd_f32(const AttnBwdParams& a, hipStream_t stream) {
    if (a.f.rows == 0) return hipSuccess;
    const hipError_t e = launch_attn_delta(a, false, stream);
    if (e != hipSuccess) return e;
    a.f.D == 64 ? run_bwd<float, 64>(a, stream) : run_bwd<float, 128>(a, stream);
    return hipGetLastError();
}

}  // namespace kda
