// Short causal depthwise convolution with SiLU (gfx950): whole sequences, a
// few tokens with replay, and the backward pass.  The formulas are in
// include/kda_ssm.h.
//
// Every form moves each element once and does about 2 W + 10 flops on it, so
// all are bound by HBM.  A lane owns 16 bytes of neighbouring channels (8 of
// bf16, 4 of float32) of a block of consecutive token rows, so that every
// access of a wave is a run of 512 contiguous bytes per row, and slides the
// last W - 1 inputs through registers: each input is read once per block plus
// the W - 1 rows before it.
#include "kda_device.h"
#include "kda_ssm_launch.h"

namespace kda {

constexpr int CV_LANES = 32;    // channel vectors per workgroup
constexpr int CV_BLOCKS = 8;    // row blocks per workgroup
constexpr int CV_THREADS = CV_LANES * CV_BLOCKS;
constexpr int CV_TOK = 16;      // rows per lane, forward

// 16 bytes of channels as floats, and back.
template <typename T>
struct Vec;
template <>
struct Vec<__bf16> {
    static constexpr int N = 8;
    static __device__ __forceinline__ void load(const void* base, int64_t e, float (&f)[8]) {
        const u32x4 u = *reinterpret_cast<const u32x4*>((const __bf16*)base + e);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            f[2 * i] = bf2_first(u[i]);
            f[2 * i + 1] = bf2_second(u[i]);
        }
    }
    static __device__ __forceinline__ void store(void* base, int64_t e, const float (&f)[8]) {
        u32x4 u;
#pragma unroll
        for (int i = 0; i < 4; ++i) u[i] = pack_bf2(f[2 * i], f[2 * i + 1]);
        *reinterpret_cast<u32x4*>((__bf16*)base + e) = u;
    }
};
template <>
struct Vec<float> {
    static constexpr int N = 4;
    static __device__ __forceinline__ void load(const void* base, int64_t e, float (&f)[4]) {
        const f32x4 u = *reinterpret_cast<const f32x4*>((const float*)base + e);
#pragma unroll
        for (int i = 0; i < 4; ++i) f[i] = u[i];
    }
    static __device__ __forceinline__ void store(void* base, int64_t e, const float (&f)[4]) {
        f32x4 u;
#pragma unroll
        for (int i = 0; i < 4; ++i) u[i] = f[i];
        *reinterpret_cast<f32x4*>((float*)base + e) = u;
    }
};
// N floats from a 16-byte aligned float array.
template <int N>
__device__ __forceinline__ void load_f(const float* p, float (&f)[N]) {
#pragma unroll
    for (int i = 0; i < N / 4; ++i) {
        const f32x4 u = reinterpret_cast<const f32x4*>(p)[i];
#pragma unroll
        for (int k = 0; k < 4; ++k) f[4 * i + k] = u[k];
    }
}

__device__ __forceinline__ float cv_sigm(float z) { return __builtin_amdgcn_rcpf(1.f + __expf(-z)); }

// Weights of a lane's channels: w[j][c], tap W - 1 for the token itself.
template <int W, int N>
__device__ __forceinline__ void load_w(const float* wp, int64_t c0, float (&w)[W][N]) {
    float f[W * N];
    load_f<W * N>(wp + c0 * W, f);   // [N, W] in memory; c0 * W floats is a multiple of 16 bytes
#pragma unroll
    for (int c = 0; c < N; ++c)
#pragma unroll
        for (int j = 0; j < W; ++j) w[j][c] = f[c * W + j];
}

// The sequence a row belongs to, its first row and end; rows outside every
// sequence have end <= row or start > row.  Ranges are clamped into
// [0, rows], so that a malformed table never addresses out of bounds.
struct Seq {
    int64_t n, start, end;
};
__device__ __forceinline__ Seq seq_range(const ConvParams& p, int64_t n) {
    if (!p.cu) return Seq{n, n * p.T, n * p.T + p.T};
    int64_t a = p.cu[n], b = p.cu[n + 1];
    a = a < 0 ? 0 : (a > p.rows ? p.rows : a);
    b = b < a ? a : (b > p.rows ? p.rows : b);
    return Seq{n, a, b};
}
__device__ __forceinline__ Seq seq_of_row(const ConvParams& p, int64_t row) {
    if (!p.cu) return seq_range(p, row / p.T);
    int lo = 0, hi = p.n_seqs;   // largest n with cu[n] <= row
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if ((int64_t)p.cu[mid] <= row) lo = mid;
        else hi = mid;
    }
    return seq_range(p, lo);
}

// x at position pos of sequence s (pos < 0: the cache's entry, or zero) for
// N channels from c0.
template <typename InT, int W, int N>
__device__ __forceinline__ void input_at(const ConvParams& p, const Seq& s, int64_t pos, int64_t c0,
                                         float (&f)[N]) {
    if (pos >= 0) {
        Vec<InT>::load(p.x, (s.start + pos) * p.x_stride + c0, f);
    } else if (p.cache && pos >= 1 - W) {
        load_f<N>(p.cache + (s.n * (W - 1) + (W - 1 + pos)) * p.channels + c0, f);
    } else {
#pragma unroll
        for (int i = 0; i < N; ++i) f[i] = 0.f;
    }
}

// Channel tiles of a row; a launch's workgroups run through them first, so
// that whole rows are in flight together.
template <int N>
__host__ __device__ __forceinline__ int64_t cv_tiles(int64_t channels) {
    return (channels + CV_LANES * N - 1) / (CV_LANES * N);
}

template <typename InT, int W>
__global__ __launch_bounds__(CV_THREADS) void conv_fwd_kernel(ConvParams p) {
    constexpr int N = Vec<InT>::N;
    const uint32_t tiles = (uint32_t)cv_tiles<N>(p.channels);
    const uint32_t rb = blockIdx.x / tiles;
    const int64_t c0 = ((int64_t)(blockIdx.x - rb * tiles) * CV_LANES + (threadIdx.x & (CV_LANES - 1))) * N;
    if (c0 >= p.channels) return;
    const int64_t r0 = ((int64_t)rb * CV_BLOCKS + threadIdx.x / CV_LANES) * CV_TOK;
    if (r0 >= p.rows) return;
    const int64_t r1 = r0 + CV_TOK < p.rows ? r0 + CV_TOK : p.rows;
    // all rows first: one round trip to memory
    float cur[CV_TOK][N];
#pragma unroll
    for (int i = 0; i < CV_TOK; ++i) {
        const int64_t r = r0 + i < r1 ? r0 + i : r1 - 1;
        Vec<InT>::load(p.x, r * p.x_stride + c0, cur[i]);
    }
    float w[W][N], b[N];
    load_w<W, N>(p.w, c0, w);
#pragma unroll
    for (int c = 0; c < N; ++c) b[c] = 0.f;
    if (p.bias) {
#pragma unroll
        for (int c = 0; c < N; ++c) b[c] = p.bias[c0 + c];
    }
    Seq s = seq_of_row(p, r0);
    float win[W - 1][N];
    bool fresh = true;
#pragma unroll
    for (int i = 0; i < CV_TOK; ++i) {
        const int64_t r = r0 + i;
        if (r >= r1) break;
        while (r >= s.end && s.n + 1 < p.n_seqs) {
            s = seq_range(p, s.n + 1);
            fresh = true;
        }
        if (r < s.start || r >= s.end) continue;   // outside every sequence
        if (fresh || r == s.start) {
#pragma unroll
            for (int j = 0; j < W - 1; ++j) input_at<InT, W, N>(p, s, r - s.start - (W - 1) + j, c0, win[j]);
            fresh = false;
        }
        float y[N];
#pragma unroll
        for (int c = 0; c < N; ++c) {
            float z = b[c];
#pragma unroll
            for (int j = 0; j < W - 1; ++j) z = fmaf(w[j][c], win[j][c], z);
            z = fmaf(w[W - 1][c], cur[i][c], z);
            y[c] = p.activation ? z * cv_sigm(z) : z;
#pragma unroll
            for (int j = 0; j + 1 < W - 1; ++j) win[j][c] = win[j + 1][c];
            win[W - 2][c] = cur[i][c];
        }
        Vec<InT>::store(p.y, r * p.channels + c0, y);
    }
}

// The cache after the call, as a launch of its own: no lane of the
// convolution reads an entry that another has replaced.
template <typename InT, int W>
__global__ __launch_bounds__(CV_THREADS) void conv_cache_update_kernel(ConvParams p) {
    constexpr int N = Vec<InT>::N;
    const int64_t nv = p.channels / N;
    const int64_t idx = (int64_t)blockIdx.x * CV_THREADS + threadIdx.x;
    if (idx >= nv * p.n_seqs) return;
    const int64_t n = idx / nv, c0 = (idx - n * nv) * N;
    const Seq s = seq_range(p, n);
    float f[W - 1][N];
#pragma unroll
    for (int m = 0; m < W - 1; ++m) input_at<InT, W, N>(p, s, s.end - s.start - (W - 1) + m, c0, f[m]);
#pragma unroll
    for (int m = 0; m < W - 1; ++m)
        Vec<float>::store(p.cache, (n * (W - 1) + m) * p.channels + c0, *reinterpret_cast<float(*)[4]>(f[m]));
    if constexpr (N == 8) {
#pragma unroll
        for (int m = 0; m < W - 1; ++m)
            Vec<float>::store(p.cache, (n * (W - 1) + m) * p.channels + c0 + 4,
                              *reinterpret_cast<float(*)[4]>(f[m] + 4));
    }
}

// A few tokens per request: a lane owns 4 channels of one request from its
// cache through the accepted replay tokens and the new ones to the cache it
// leaves, so one launch does all of it in place.
template <typename InT, int W>
__global__ __launch_bounds__(64) void conv_step_kernel(ConvParams p) {
    const int64_t nv = p.channels / 4;
    const int64_t idx = (int64_t)blockIdx.x * 64 + threadIdx.x;
    if (idx >= nv * p.n_seqs) return;
    const int64_t n = idx / nv, c0 = (idx - n * nv) * 4;
    auto load = [&](const void* base, int64_t e, float (&f)[4]) {
        if constexpr (sizeof(InT) == 4) {
            Vec<float>::load(base, e, f);
        } else {
            const u32x2 u = *reinterpret_cast<const u32x2*>((const __bf16*)base + e);
            f[0] = bf2_first(u[0]);
            f[1] = bf2_second(u[0]);
            f[2] = bf2_first(u[1]);
            f[3] = bf2_second(u[1]);
        }
    };
    float win[W - 1][4];
#pragma unroll
    for (int j = 0; j < W - 1; ++j) Vec<float>::load(p.cache, (n * (W - 1) + j) * p.channels + c0, win[j]);
    auto push = [&](const float (&f)[4]) {
#pragma unroll
        for (int c = 0; c < 4; ++c) {
#pragma unroll
            for (int j = 0; j + 1 < W - 1; ++j) win[j][c] = win[j + 1][c];
            win[W - 2][c] = f[c];
        }
    };
    auto keep = [&]() {
#pragma unroll
        for (int j = 0; j < W - 1; ++j) Vec<float>::store(p.cache, (n * (W - 1) + j) * p.channels + c0, win[j]);
    };
    if (p.Tr > 0) {
        int k = p.n_replay ? p.n_replay[n] : p.Tr;
        k = k < 0 ? 0 : (k > p.Tr ? p.Tr : k);
        for (int t = k > W - 1 ? k - (W - 1) : 0; t < k; ++t) {   // only the last W - 1 stay
            float f[4];
            load(p.rx, (n * p.Tr + t) * p.rx_stride + c0, f);
            push(f);
        }
    }
    if (!p.commit) keep();
    float w[W][4], b[4] = {0.f, 0.f, 0.f, 0.f};
    load_w<W, 4>(p.w, c0, w);
    if (p.bias) {
#pragma unroll
        for (int c = 0; c < 4; ++c) b[c] = p.bias[c0 + c];
    }
    for (int t = 0; t < (int)p.T; ++t) {
        const int64_t r = n * p.T + t;
        float f[4], y[4];
        load(p.x, r * p.x_stride + c0, f);
#pragma unroll
        for (int c = 0; c < 4; ++c) {
            float z = b[c];
#pragma unroll
            for (int j = 0; j < W - 1; ++j) z = fmaf(w[j][c], win[j][c], z);
            z = fmaf(w[W - 1][c], f[c], z);
            y[c] = p.activation ? z / (1.f + expf(-z)) : z;
        }
        push(f);
        if constexpr (sizeof(InT) == 4) {
            Vec<float>::store(p.y, r * p.channels + c0, y);
        } else {
            u32x2 u = {pack_bf2(y[0], y[1]), pack_bf2(y[2], y[3])};
            *reinterpret_cast<u32x2*>((__bf16*)p.y + r * p.channels + c0) = u;
        }
    }
    if (p.commit) keep();
}

// Backward.  With dz = dy silu'(z):
//   dx_t = sum_d w_{W-1-d} dz_{t+d},  dw_j = sum_t dz_t x_{t-W+1+j},  db = sum_t dz_t.
// A lane walks CB_TOK rows and the W - 1 rows after them (recomputing their
// dz, so that no dz goes through memory), with the W - 1 unfinished dx in
// registers; its part of dw and db is summed over the workgroup's row blocks
// in LDS and written as one partial sum per workgroup, which a second launch
// adds up in a fixed order.
constexpr int CB_TOK = (int)(kConvBwdRows / CV_BLOCKS);

template <typename InT, int W>
__global__ __launch_bounds__(CV_THREADS) void conv_bwd_kernel(ConvBwdParams q) {
    constexpr int N = Vec<InT>::N;
    const ConvParams& p = q.f;
    const int lane = threadIdx.x & (CV_LANES - 1), blk = threadIdx.x / CV_LANES;
    const uint32_t tiles = (uint32_t)cv_tiles<N>(p.channels);
    const uint32_t rb = blockIdx.x / tiles;
    const int64_t c0 = ((int64_t)(blockIdx.x - rb * tiles) * CV_LANES + lane) * N;
    const bool live = c0 < p.channels;
    const int64_t r0 = ((int64_t)rb * CV_BLOCKS + blk) * CB_TOK;
    float gw[W + 1][N];
#pragma unroll
    for (int j = 0; j <= W; ++j)
#pragma unroll
        for (int c = 0; c < N; ++c) gw[j][c] = 0.f;
    if (live && r0 < p.rows) {
        const int64_t r1 = r0 + CB_TOK < p.rows ? r0 + CB_TOK : p.rows;
        const int64_t r2 = r1 + W - 1 < p.rows ? r1 + W - 1 : p.rows;
        float w[W][N], b[N];
        load_w<W, N>(p.w, c0, w);
#pragma unroll
        for (int c = 0; c < N; ++c) b[c] = p.bias ? p.bias[c0 + c] : 0.f;
        Seq s = seq_of_row(p, r0);
        float win[W - 1][N], dx[W][N];   // dx[d]: the row d before the current one
#pragma unroll
        for (int d = 0; d < W; ++d)
#pragma unroll
            for (int c = 0; c < N; ++c) dx[d][c] = 0.f;
        // rows [lo, ...) of this walk belong to a sequence and are this lane's
        bool fresh = true;
        int64_t first = r0;   // first row of the current sequence in this walk
        auto finish = [&](int64_t r, const float (&f)[N]) {
            if (r >= first && r < r1) Vec<InT>::store(q.gx, r * p.channels + c0, f);
        };
        int64_t r = r0;
        for (; r < r2; ++r) {
            if (r >= s.end) {
                // the sequence ends: its last rows are complete
                if (!fresh) {
#pragma unroll
                    for (int d = 1; d < W; ++d) finish(r - d, dx[d - 1]);
                }
                while (r >= s.end && s.n + 1 < p.n_seqs) s = seq_range(p, s.n + 1);
                fresh = true;
            }
            if (r < s.start || r >= s.end) continue;
            if (fresh) {
                if (r >= r1) break;   // the next sequence's rows are another lane's
                first = r;
#pragma unroll
                for (int j = 0; j < W - 1; ++j) input_at<InT, W, N>(p, s, r - s.start - (W - 1) + j, c0, win[j]);
#pragma unroll
                for (int d = 0; d < W; ++d)
#pragma unroll
                    for (int c = 0; c < N; ++c) dx[d][c] = 0.f;
                fresh = false;
            }
            float x[N], g[N];
            Vec<InT>::load(p.x, r * p.x_stride + c0, x);
            Vec<InT>::load(q.gy, r * q.gy_stride + c0, g);
            const bool own = r < r1;
#pragma unroll
            for (int c = 0; c < N; ++c) {
                float dz = g[c];
                if (p.activation) {
                    float z = b[c];
#pragma unroll
                    for (int j = 0; j < W - 1; ++j) z = fmaf(w[j][c], win[j][c], z);
                    z = fmaf(w[W - 1][c], x[c], z);
                    const float sg = cv_sigm(z);
                    dz = g[c] * sg * fmaf(z, 1.f - sg, 1.f);
                }
#pragma unroll
                for (int d = W - 1; d >= 1; --d) dx[d][c] = fmaf(w[W - 1 - d][c], dz, dx[d - 1][c]);
                dx[0][c] = w[W - 1][c] * dz;
                if (own) {
#pragma unroll
                    for (int j = 0; j < W - 1; ++j) gw[j][c] = fmaf(dz, win[j][c], gw[j][c]);
                    gw[W - 1][c] = fmaf(dz, x[c], gw[W - 1][c]);
                    gw[W][c] += dz;
                }
#pragma unroll
                for (int j = 0; j + 1 < W - 1; ++j) win[j][c] = win[j + 1][c];
                win[W - 2][c] = x[c];
            }
            finish(r - (W - 1), dx[W - 1]);
        }
        if (!fresh) {   // the walk ended inside a sequence, or at its end with the rows
#pragma unroll
            for (int d = 1; d < W; ++d) finish(r - d, dx[d - 1]);
        }
    }
    __shared__ float sum[CV_BLOCKS / 2][W + 1][CV_LANES * N];
#pragma unroll
    for (int half = CV_BLOCKS / 2; half >= 1; half /= 2) {
        if (blk >= half && blk < 2 * half) {
#pragma unroll
            for (int j = 0; j <= W; ++j)
#pragma unroll
                for (int c = 0; c < N; ++c) sum[blk - half][j][lane * N + c] = gw[j][c];
        }
        __syncthreads();
        if (blk < half) {
#pragma unroll
            for (int j = 0; j <= W; ++j)
#pragma unroll
                for (int c = 0; c < N; ++c) gw[j][c] += sum[blk][j][lane * N + c];
        }
        __syncthreads();
    }
    if (blk == 0 && live) {
#pragma unroll
        for (int j = 0; j <= W; ++j)
#pragma unroll
            for (int c = 0; c < N; ++c)
                q.partial[((int64_t)rb * (W + 1) + j) * p.channels + c0 + c] = gw[j][c];
    }
}

// Sums the partial weight gradients: 64 columns by 4 strides per workgroup.
template <int W>
__global__ __launch_bounds__(256) void conv_bwd_reduce_kernel(ConvBwdParams q, int64_t n_part) {
    const int64_t cols = (int64_t)(W + 1) * q.f.channels;
    const int64_t col = (int64_t)blockIdx.x * 64 + (threadIdx.x & 63);
    const int k = threadIdx.x >> 6;
    float a = 0.f;
    if (col < cols)
        for (int64_t i = k; i < n_part; i += 4) a += q.partial[i * cols + col];
    __shared__ float s[4][64];
    s[k][threadIdx.x & 63] = a;
    __syncthreads();
    if (k == 0 && col < cols) {
        const int t = threadIdx.x;
        const float v = (s[0][t] + s[1][t]) + (s[2][t] + s[3][t]);
        const int64_t j = col / q.f.channels, c = col - j * q.f.channels;
        if (j < W) q.gw[c * W + j] = v;
        else if (q.gbias) q.gbias[c] = v;
    }
}

// Gradient of the cache: its entry m (position m - W + 1) is read by the
// positions t < W - 1 with t - (W - 1 - j) = m - W + 1, that is tap j = m - t.
template <typename InT, int W>
__global__ __launch_bounds__(CV_THREADS) void conv_bwd_cache_kernel(ConvBwdParams q) {
    constexpr int N = Vec<InT>::N;
    const ConvParams& p = q.f;
    const int64_t nv = p.channels / N;
    const int64_t idx = (int64_t)blockIdx.x * CV_THREADS + threadIdx.x;
    if (idx >= nv * p.n_seqs) return;
    const int64_t n = idx / nv, c0 = (idx - n * nv) * N;
    const Seq s = seq_range(p, n);
    float w[W][N], in[2 * (W - 1)][N], gc[W - 1][N];
    load_w<W, N>(p.w, c0, w);
    const int64_t len = s.end - s.start;
#pragma unroll
    for (int j = 0; j < 2 * (W - 1); ++j) {   // positions 1 - W .. W - 2
        const int64_t pos = j - (W - 1);
        if (pos < len) input_at<InT, W, N>(p, s, pos, c0, in[j]);
        else
            for (int c = 0; c < N; ++c) in[j][c] = 0.f;
    }
#pragma unroll
    for (int m = 0; m < W - 1; ++m)
#pragma unroll
        for (int c = 0; c < N; ++c) gc[m][c] = 0.f;
#pragma unroll
    for (int t = 0; t < W - 1; ++t) {
        if (t >= len) break;
        float g[N];
        Vec<InT>::load(q.gy, (s.start + t) * q.gy_stride + c0, g);
#pragma unroll
        for (int c = 0; c < N; ++c) {
            float dz = g[c];
            if (p.activation) {
                float z = p.bias ? p.bias[c0 + c] : 0.f;
#pragma unroll
                for (int j = 0; j < W; ++j) z = fmaf(w[j][c], in[t + j][c], z);
                const float sg = cv_sigm(z);
                dz = g[c] * sg * fmaf(z, 1.f - sg, 1.f);
            }
#pragma unroll
            for (int m = t; m < W - 1; ++m) gc[m][c] = fmaf(w[m - t][c], dz, gc[m][c]);
        }
    }
#pragma unroll
    for (int m = 0; m < W - 1; ++m)
#pragma unroll
        for (int c = 0; c < N; ++c) q.gcache[(n * (W - 1) + m) * p.channels + c0 + c] = gc[m][c];
}

template <typename InT, int W>
static hipError_t run_conv_fwd(const ConvParams& p, hipStream_t stream) {
    constexpr int N = Vec<InT>::N;
    if (p.rows > 0) {
        const dim3 grid((unsigned)(cv_tiles<N>(p.channels) * ((p.rows + CV_BLOCKS * CV_TOK - 1) / (CV_BLOCKS * CV_TOK))));
        hipLaunchKernelGGL((conv_fwd_kernel<InT, W>), grid, dim3(CV_THREADS), 0, stream, p);
    }
    if (p.cache) {
        const int64_t n = (int64_t)p.n_seqs * (p.channels / N);
        hipLaunchKernelGGL((conv_cache_update_kernel<InT, W>), dim3((unsigned)((n + CV_THREADS - 1) / CV_THREADS)),
                           dim3(CV_THREADS), 0, stream, p);
    }
    return hipGetLastError();
}
template <typename InT, int W>
static hipError_t run_conv_step(const ConvParams& p, hipStream_t stream) {
    const int64_t n = (int64_t)p.n_seqs * (p.channels / 4);
    hipLaunchKernelGGL((conv_step_kernel<InT, W>), dim3((unsigned)((n + 63) / 64)), dim3(64), 0, stream, p);
    return hipGetLastError();
}
template <typename InT, int W>
static hipError_t run_conv_bwd(const ConvBwdParams& q, hipStream_t stream) {
    constexpr int N = Vec<InT>::N;
    const ConvParams& p = q.f;
    const int64_t parts = (p.rows + kConvBwdRows - 1) / kConvBwdRows;
    if (parts > 0) {
        const dim3 grid((unsigned)(cv_tiles<N>(p.channels) * parts));
        hipLaunchKernelGGL((conv_bwd_kernel<InT, W>), grid, dim3(CV_THREADS), 0, stream, q);
    }
    const int64_t cols = (int64_t)(W + 1) * p.channels;
    hipLaunchKernelGGL((conv_bwd_reduce_kernel<W>), dim3((unsigned)((cols + 63) / 64)), dim3(256), 0, stream, q, parts);
    if (q.gcache && p.n_seqs > 0) {
        const int64_t n = (int64_t)p.n_seqs * (p.channels / N);
        hipLaunchKernelGGL((conv_bwd_cache_kernel<InT, W>), dim3((unsigned)((n + CV_THREADS - 1) / CV_THREADS)),
                           dim3(CV_THREADS), 0, stream, q);
    }
    return hipGetLastError();
}

#define KDA_BY_WIDTH(run, p, width, bf16_in, stream)                                               \
    do {                                                                                           \
        if (bf16_in)                                                                               \
            return (width) == 2 ? run<__bf16, 2>(p, stream)                                        \
                                : (width) == 3 ? run<__bf16, 3>(p, stream) : run<__bf16, 4>(p, stream); \
        return (width) == 2 ? run<float, 2>(p, stream)                                             \
                            : (width) == 3 ? run<float, 3>(p, stream) : run<float, 4>(p, stream);  \
    } while (0)

hipError_t launch_conv_fwd(const ConvParams& p, bool bf16_in, hipStream_t stream) {
    KDA_BY_WIDTH(run_conv_fwd, p, p.width, bf16_in, stream);
}
hipError_t launch_conv_step(const ConvParams& p, bool bf16_in, hipStream_t stream) {
    KDA_BY_WIDTH(run_conv_step, p, p.width, bf16_in, stream);
}
hipError_t launch_conv_bwd(const ConvBwdParams& p, bool bf16_in, hipStream_t stream) {
    KDA_BY_WIDTH(run_conv_bwd, p, p.f.width, bf16_in, stream);
}

}  // namespace kda
