// Recurrent form of the state space scan (gfx950): a few tokens per request
// with replay, states in place.  Formulas and semantics: include/kda_ssm.h.
//
// Bound by HBM: a (request, head) state of N x P floats is read and written
// once (8 N P bytes) for 4 N P flops per token, so up to about ten tokens
// hide behind the state's traffic.  One workgroup per state holds it in
// registers: lane group (P / 4 lanes) r of the 256 threads owns rows
// r + R i (R groups) and four columns per lane, so every access of a wave to
// the state is whole rows of contiguous memory.  The sum over rows in
// y = S^T C runs over a lane's rows, then across the wave's row groups by
// lane permutes, then across the four waves through LDS; tokens are staged
// in LDS SR_TOK at a time, with one barrier before and one after each batch.
// Measured (MI355X): 256 requests, 64 heads of 64, N 128, 5 replayed and 5 new
// tokens 196 to 201 us, 5.5 TB/s of state, above the rate of a large copy; one
// token of one request, 24 heads, 4.8 us.
#include "kda_device.h"
#include "kda_ssm_launch.h"

namespace kda {

constexpr int SR_THREADS = 256;
constexpr int SR_TOK = 8;   // tokens staged at a time

__device__ __forceinline__ float sr_softplus(float x) {
    return fmaxf(x, 0.f) + log1pf(expf(-fabsf(x)));
}

template <typename InT, int N, int P>
__global__ __launch_bounds__(SR_THREADS) void ssm_recurrent_kernel(SsmRecParams p) {
    constexpr int QP = P / 4;                // lanes per row
    constexpr int RG = SR_THREADS / QP;      // row groups
    constexpr int NR = N / RG;               // rows per lane
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    const int q = tid % QP, rg = tid / QP;
    const int64_t bh = blockIdx.x;
    const int64_t b = bh / p.H;
    const int h = (int)(bh - b * p.H);
    const int grp = h / (p.H / p.G);
    f32x4* Sp = reinterpret_cast<f32x4*>(p.S + bh * (N * P));
    f32x4 s[NR];
#pragma unroll
    for (int i = 0; i < NR; ++i) s[i] = __builtin_nontemporal_load(&Sp[(rg + RG * i) * QP + q]);

    __shared__ __attribute__((aligned(16))) float sB[SR_TOK][N], sC[SR_TOK][N], sX[SR_TOK][P];
    __shared__ float sDt[SR_TOK], sE[SR_TOK];
    __shared__ __attribute__((aligned(16))) float sY[SR_TOK][SR_THREADS / 64][P];
    const float A = p.A[h], bias = p.dt_bias ? p.dt_bias[h] : 0.f, D = p.D ? p.D[h] : 0.f;

    auto stage = [&](const SsmTokens& src, int t0, int nt, bool emit) {
        for (int i = tid; i < nt * N; i += SR_THREADS) {
            const int t = i / N, n = i - t * N;
            const int64_t row = b * src.T + t0 + t;
            sB[t][n] = to_f32(((const InT*)src.Bm)[row * src.B_stride + grp * N + n]);
            if (emit) sC[t][n] = to_f32(((const InT*)src.C)[row * src.C_stride + grp * N + n]);
        }
        for (int i = tid; i < nt * P; i += SR_THREADS) {
            const int t = i / P, c = i - t * P;
            sX[t][c] = to_f32(((const InT*)src.x)[(b * src.T + t0 + t) * src.x_stride + (int64_t)h * P + c]);
        }
        if (tid < nt) {
            float dt = src.dt[(b * src.T + t0 + tid) * p.H + h] + bias;
            if (p.softplus) dt = sr_softplus(dt);
            sDt[tid] = dt;
            sE[tid] = expf(dt * A);
        }
    };
    auto store_state = [&]() {
#pragma unroll
        for (int i = 0; i < NR; ++i) __builtin_nontemporal_store(s[i], &Sp[(rg + RG * i) * QP + q]);
    };
    auto run = [&](const SsmTokens& src, int n, bool emit) {
        for (int t0 = 0; t0 < n; t0 += SR_TOK) {
            const int nt = n - t0 < SR_TOK ? n - t0 : SR_TOK;
            if (t0 > 0) __syncthreads();   // the last batch is consumed
            stage(src, t0, nt, emit);
            __syncthreads();
            for (int t = 0; t < nt; ++t) {
                const float e = sE[t], dt = sDt[t];
                const f32x4 x = *reinterpret_cast<const f32x4*>(&sX[t][4 * q]);
                f32x4 y = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
                for (int i = 0; i < NR; ++i) {
                    const float bn = dt * sB[t][rg + RG * i];
#pragma unroll
                    for (int k = 0; k < 4; ++k) s[i][k] = fmaf(bn, x[k], e * s[i][k]);
                    if (emit) {
                        const float cn = sC[t][rg + RG * i];
#pragma unroll
                        for (int k = 0; k < 4; ++k) y[k] = fmaf(cn, s[i][k], y[k]);
                    }
                }
                if (emit) {
#pragma unroll
                    for (int k = 0; k < 4; ++k) {
                        if constexpr (QP == 16) y[k] += __shfl_xor(y[k], 16);
                        y[k] += __shfl_xor(y[k], 32);
                    }
                    if (lane < QP) *reinterpret_cast<f32x4*>(&sY[t][wave][4 * q]) = y;
                }
            }
            if (emit) {
                __syncthreads();
                for (int i = tid; i < nt * P; i += SR_THREADS) {
                    const int t = i / P, c = i - t * P;
                    const float y = (sY[t][0][c] + sY[t][1][c]) + (sY[t][2][c] + sY[t][3][c]);
                    ((InT*)p.y)[((b * src.T + t0 + t) * p.H + h) * P + c] = (InT)fmaf(D, sX[t][c], y);
                }
            }
        }
    };
    int k = 0;
    if (p.rep.T > 0) {
        k = p.n_replay ? p.n_replay[b] : p.rep.T;
        k = k < 0 ? 0 : (k > p.rep.T ? p.rep.T : k);
        run(p.rep, k, false);
    }
    if (!p.commit && k > 0) store_state();
    if (p.out.T > 0) {
        if (k > 0) __syncthreads();
        run(p.out, p.out.T, true);
        if (p.commit) store_state();
    } else if (p.commit && k > 0) {
        store_state();
    }
}

template <typename InT>
static hipError_t run_ssm_recurrent(const SsmRecParams& p, hipStream_t stream) {
    const dim3 grid((unsigned)((int64_t)p.B * p.H)), block(SR_THREADS);
    if (p.N == 128 && p.P == 64) hipLaunchKernelGGL((ssm_recurrent_kernel<InT, 128, 64>), grid, block, 0, stream, p);
    else if (p.N == 128) hipLaunchKernelGGL((ssm_recurrent_kernel<InT, 128, 128>), grid, block, 0, stream, p);
    else if (p.P == 64) hipLaunchKernelGGL((ssm_recurrent_kernel<InT, 64, 64>), grid, block, 0, stream, p);
    else hipLaunchKernelGGL((ssm_recurrent_kernel<InT, 64, 128>), grid, block, 0, stream, p);
    return hipGetLastError();
}
hipError_t launch_ssm_recurrent(const SsmRecParams& p, bool bf16_in, hipStream_t stream) {
    return bf16_in ? run_ssm_recurrent<__bf16>(p, stream) : run_ssm_recurrent<float>(p, stream);
}

}  // namespace kda
