// Short causal depthwise convolution with SiLU (gfx950): whole sequences, a
// few tokens with replay, and the backward pass.  The formulas are in
// include/kda_ssm.h.
//
// Every form moves each element once and does about 2 W + 10 flops on it, so
// all are bound by HBM.  A wave owns 256 neighbouring channels, four per lane
// (512 contiguous bytes of bf16 per row, 1 KB of float32), of a block of
// consecutive token rows, requests CV_AHEAD rows while it computes the
// CV_AHEAD before them and slides the last W - 1 inputs through registers:
// each input is read once per block plus the W - 1 rows before it.  Rows are
// the same for all lanes, so sequence boundaries cost scalar instructions
// only.  Eight channels per lane and all rows requested at once, the first
// form, needs 180 to 400 registers: 42 us forward and 121 us backward at 8192
// rows of 4352 channels, against 32 (4.4 TB/s) and 57 us (62 with a branch per
// channel).  Backward, about 30 vector instructions per element, two of them
// transcendental, take 40 us by themselves.
#include "kda_device.h"
#include "kda_ssm_launch.h"

#include <type_traits>

namespace kda {

constexpr int CV_WAVES = (int)kConvWaves;       // row blocks per workgroup, one per wave
constexpr int CV_THREADS = 64 * CV_WAVES;
constexpr int CV_AHEAD = 8;       // rows per request, forward
constexpr int CB_AHEAD = 4;       // ... backward (more registers per row)
constexpr int CV_CH = 256;        // channels per wave

// Four channels as floats, and back (stores that leave no copy in the L2,
// which is far smaller than any large output: forward 33 against 40 us).
template <typename T>
struct Vec;
template <>
struct Vec<__bf16> {
    typedef u32x2 raw;
    static __device__ __forceinline__ raw fetch(const void* base, int64_t e) {
        return *reinterpret_cast<const u32x2*>((const __bf16*)base + e);
    }
    static __device__ __forceinline__ void open(raw u, float (&f)[4]) {
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            f[2 * i] = bf2_first(u[i]);
            f[2 * i + 1] = bf2_second(u[i]);
        }
    }
    static __device__ __forceinline__ void store(void* base, int64_t e, const float (&f)[4]) {
        __builtin_nontemporal_store(u32x2{pack_bf2(f[0], f[1]), pack_bf2(f[2], f[3])},
                                    reinterpret_cast<u32x2*>((__bf16*)base + e));
    }
};
template <>
struct Vec<float> {
    typedef f32x4 raw;
    static __device__ __forceinline__ raw fetch(const void* base, int64_t e) {
        return *reinterpret_cast<const f32x4*>((const float*)base + e);
    }
    static __device__ __forceinline__ void open(raw u, float (&f)[4]) {
#pragma unroll
        for (int i = 0; i < 4; ++i) f[i] = u[i];
    }
    static __device__ __forceinline__ void store(void* base, int64_t e, const float (&f)[4]) {
        __builtin_nontemporal_store(f32x4{f[0], f[1], f[2], f[3]}, reinterpret_cast<f32x4*>((float*)base + e));
    }
};
template <typename T>
__device__ __forceinline__ void load4(const void* base, int64_t e, float (&f)[4]) {
    Vec<T>::open(Vec<T>::fetch(base, e), f);
}
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

// Sigmoid, the same in every form of the operator, so that a prompt and single
// tokens give the same bits.  The fast exponential is off by |z| 2^-24 and the
// hardware's reciprocal by a rounding: float32 results are 6.2e-8 off 64 bits,
// 6.1e-8 with expf and a division, which take 68.5 against 62 us (8192 rows of
// 4352 channels).
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
// four channels from c0.
template <typename InT, int W>
__device__ __forceinline__ void input_at(const ConvParams& p, const Seq& s, int64_t pos, int64_t c0, float (&f)[4]) {
    if (pos >= 0) {
        load4<InT>(p.x, (s.start + pos) * p.x_stride + c0, f);
    } else if (p.cache && pos >= 1 - W) {
        load4<float>(p.cache, (s.n * (W - 1) + (W - 1 + pos)) * p.channels + c0, f);
    } else {
#pragma unroll
        for (int i = 0; i < 4; ++i) f[i] = 0.f;
    }
}

// Channel strips of a row; a launch's workgroups run through them first, so
// that whole rows are in flight together.
__host__ __device__ __forceinline__ int64_t cv_strips(int64_t channels) { return (channels + CV_CH - 1) / CV_CH; }

// The rows of a walk, one after the other, all wave-uniform.
struct Walk {
    Seq s;
    __device__ __forceinline__ Walk(const ConvParams& p, int64_t row) : s(seq_of_row(p, row)) {}
    // moves to a row; whether it belongs to a sequence (then s is that one)
    __device__ __forceinline__ bool at(const ConvParams& p, int64_t row) {
        while (row >= s.end && s.n + 1 < p.n_seqs) s = seq_range(p, s.n + 1);
        return row >= s.start && row < s.end;
    }
};

template <typename InT, int W>
__global__ __launch_bounds__(CV_THREADS) void conv_fwd_kernel(ConvParams p, int32_t rows_per_wave) {
    const uint32_t strips = (uint32_t)cv_strips(p.channels);
    const uint32_t rb = blockIdx.x / strips;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int64_t c0 = (int64_t)(blockIdx.x - rb * strips) * CV_CH + 4 * (threadIdx.x & 63);
    if (c0 >= p.channels) return;
    const int64_t r0 = ((int64_t)rb * CV_WAVES + wave) * rows_per_wave;
    if (r0 >= p.rows) return;
    const int64_t r1 = r0 + rows_per_wave < p.rows ? r0 + rows_per_wave : p.rows;
    typename Vec<InT>::raw ahead[CV_AHEAD], now[CV_AHEAD];
    auto request = [&](int64_t r) {
#pragma unroll
        for (int i = 0; i < CV_AHEAD; ++i) {
            const int64_t k = r + i < p.rows ? r + i : p.rows - 1;
            ahead[i] = Vec<InT>::fetch(p.x, k * p.x_stride + c0);
        }
    };
    request(r0);
    float w[W][4], b[4] = {0.f, 0.f, 0.f, 0.f};
    load_w<W, 4>(p.w, c0, w);
    if (p.bias) {
#pragma unroll
        for (int c = 0; c < 4; ++c) b[c] = p.bias[c0 + c];
    }
    Walk k(p, r0);
    float win[W - 1][4];
#pragma unroll
    for (int j = 0; j < W - 1; ++j) input_at<InT, W>(p, k.s, r0 >= k.s.start && r0 < k.s.end ? r0 - k.s.start - (W - 1) + j : -W, c0, win[j]);
    for (int64_t r = r0; r < r1; r += CV_AHEAD) {
#pragma unroll
        for (int i = 0; i < CV_AHEAD; ++i) now[i] = ahead[i];
        if (r + CV_AHEAD < r1) request(r + CV_AHEAD);
#pragma unroll
        for (int i = 0; i < CV_AHEAD; ++i) {
            if (r + i >= r1) break;
            const bool in = k.at(p, r + i);
            if (in && r + i == k.s.start) {
#pragma unroll
                for (int j = 0; j < W - 1; ++j) input_at<InT, W>(p, k.s, j - (W - 1), c0, win[j]);
            }
            float x[4], y[4];
            Vec<InT>::open(now[i], x);
#pragma unroll
            for (int c = 0; c < 4; ++c) {
                float z = b[c];
#pragma unroll
                for (int j = 0; j < W - 1; ++j) z = fmaf(w[j][c], win[j][c], z);
                z = fmaf(w[W - 1][c], x[c], z);
                y[c] = p.activation ? z * cv_sigm(z) : z;
#pragma unroll
                for (int j = 0; j + 1 < W - 1; ++j) win[j][c] = win[j + 1][c];
                win[W - 2][c] = x[c];
            }
            if (in) Vec<InT>::store(p.y, (r + i) * p.channels + c0, y);
        }
    }
}

// The cache after the call, as a launch of its own: a sequence's first W - 1
// rows can belong to several waves, which all read the old entries.
template <typename InT, int W>
__global__ __launch_bounds__(64) void conv_cache_update_kernel(ConvParams p) {
    const int64_t nv = p.channels / 4;
    const int64_t idx = (int64_t)blockIdx.x * 64 + threadIdx.x;
    if (idx >= nv * p.n_seqs) return;
    const int64_t n = idx / nv, c0 = (idx - n * nv) * 4;
    const Seq s = seq_range(p, n);
    float f[W - 1][4];
#pragma unroll
    for (int m = 0; m < W - 1; ++m) input_at<InT, W>(p, s, s.end - s.start - (W - 1) + m, c0, f[m]);
#pragma unroll
    for (int m = 0; m < W - 1; ++m) Vec<float>::store(p.cache, (n * (W - 1) + m) * p.channels + c0, f[m]);
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
    float win[W - 1][4];
#pragma unroll
    for (int j = 0; j < W - 1; ++j) load4<float>(p.cache, (n * (W - 1) + j) * p.channels + c0, win[j]);
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
    float w[W][4], b[4] = {0.f, 0.f, 0.f, 0.f};
    load_w<W, 4>(p.w, c0, w);
    if (p.bias) {
#pragma unroll
        for (int c = 0; c < 4; ++c) b[c] = p.bias[c0 + c];
    }
    if (p.Tr > 0) {
        int k = p.n_replay ? p.n_replay[n] : p.Tr;
        k = k < 0 ? 0 : (k > p.Tr ? p.Tr : k);
        for (int t = k > W - 1 ? k - (W - 1) : 0; t < k; ++t) {   // only the last W - 1 stay
            float f[4];
            load4<InT>(p.rx, (n * p.Tr + t) * p.rx_stride + c0, f);
            push(f);
        }
    }
    if (!p.commit) keep();
    const int T = (int)p.T;
    for (int t0 = 0; t0 < T; t0 += CV_AHEAD) {
        typename Vec<InT>::raw xr[CV_AHEAD];
#pragma unroll
        for (int i = 0; i < CV_AHEAD; ++i)
            xr[i] = Vec<InT>::fetch(p.x, (n * T + (t0 + i < T ? t0 + i : T - 1)) * p.x_stride + c0);
#pragma unroll
        for (int i = 0; i < CV_AHEAD; ++i) {
            if (t0 + i >= T) break;
            float f[4], y[4];
            Vec<InT>::open(xr[i], f);
#pragma unroll
            for (int c = 0; c < 4; ++c) {
                float z = b[c];
#pragma unroll
                for (int j = 0; j < W - 1; ++j) z = fmaf(w[j][c], win[j][c], z);
                z = fmaf(w[W - 1][c], f[c], z);
                y[c] = p.activation ? z * cv_sigm(z) : z;
            }
            push(f);
            Vec<InT>::store(p.y, (n * T + t0 + i) * p.channels + c0, y);
        }
    }
    if (p.commit) keep();
}

// Backward.  With dz = dy silu'(z):
//   dx_t = sum_d w_{W-1-d} dz_{t+d},  dw_j = sum_t dz_t x_{t-W+1+j},  db = sum_t dz_t.
// A wave walks its rows and the W - 1 rows after them (recomputing their dz,
// so that no dz goes through memory), with the W - 1 unfinished dx in
// registers; its part of dw and db is summed over the workgroup's row blocks
// in LDS and written as one partial sum per workgroup, which a second launch
// adds up in a fixed order.
template <typename InT, int W>
__global__ __launch_bounds__(CV_THREADS) void conv_bwd_kernel(ConvBwdParams q) {
    const ConvParams& p = q.f;
    const uint32_t strips = (uint32_t)cv_strips(p.channels);
    const uint32_t rb = blockIdx.x / strips;
    const int lane = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int64_t c0 = (int64_t)(blockIdx.x - rb * strips) * CV_CH + 4 * lane;
    const bool live = c0 < p.channels;
    const int64_t r0 = ((int64_t)rb * CV_WAVES + wave) * q.rows_per_wave;
    float gw[W + 1][4];
#pragma unroll
    for (int j = 0; j <= W; ++j)
#pragma unroll
        for (int c = 0; c < 4; ++c) gw[j][c] = 0.f;
    if (live && r0 < p.rows) {
        const int64_t r1 = r0 + q.rows_per_wave < p.rows ? r0 + q.rows_per_wave : p.rows;
        const int64_t r2 = r1 + W - 1;
        typename Vec<InT>::raw xa[CB_AHEAD], ga[CB_AHEAD];   // the next rows, in order
        auto request = [&](int i, int64_t row) {
            const int64_t k = row < p.rows ? row : p.rows - 1;
            xa[i] = Vec<InT>::fetch(p.x, k * p.x_stride + c0);
            ga[i] = Vec<InT>::fetch(q.gy, k * q.gy_stride + c0);
        };
#pragma unroll
        for (int i = 0; i < CB_AHEAD; ++i) request(i, r0 + i);
        float w[W][4], b[4];
        load_w<W, 4>(p.w, c0, w);
#pragma unroll
        for (int c = 0; c < 4; ++c) b[c] = p.bias ? p.bias[c0 + c] : 0.f;
        Walk k(p, r0);
        float win[W - 1][4], dx[W][4];   // dx[d]: of the row d before the current one
#pragma unroll
        for (int j = 0; j < W - 1; ++j) input_at<InT, W>(p, k.s, r0 >= k.s.start && r0 < k.s.end ? r0 - k.s.start - (W - 1) + j : -W, c0, win[j]);
#pragma unroll
        for (int d = 0; d < W; ++d)
#pragma unroll
            for (int c = 0; c < 4; ++c) dx[d][c] = 0.f;
        uint32_t mine = 0;   // bit d: the row d before the current one is of a sequence and this wave's
        // One row.  INSIDE: it, the W - 1 rows before it and this wave's rows
        // are of one sequence and the activation is on, which nearly all rows
        // are: no branch per channel then.
        auto step = [&](auto inside, int i, int64_t row) {
            constexpr bool INSIDE = decltype(inside)::value;
            const bool in = INSIDE || (row < p.rows && k.at(p, row));
            if (!INSIDE && in && row == k.s.start) {
#pragma unroll
                for (int j = 0; j < W - 1; ++j) input_at<InT, W>(p, k.s, j - (W - 1), c0, win[j]);
            }
            const bool act = INSIDE || p.activation;
            mine = mine << 1 | (INSIDE || (in && row < r1) ? 1u : 0u);
            if (!INSIDE && q.zero_rest && !in && row < r1) {
                const float none[4] = {0.f, 0.f, 0.f, 0.f};
                Vec<InT>::store(q.gx, row * p.channels + c0, none);
            }
            // rows before this one that this row's z reaches (none outside its sequence)
            const int reach = INSIDE ? W - 1 : in ? (row - k.s.start < W - 1 ? (int)(row - k.s.start) : W - 1) : -1;
            float x[4], g[4];
            Vec<InT>::open(xa[i], x);
            Vec<InT>::open(ga[i], g);
            request(i, row + CB_AHEAD < r2 ? row + CB_AHEAD : r2);
#pragma unroll
            for (int c = 0; c < 4; ++c) {
                float dz = g[c];
                if (act) {
                    float z = b[c];
#pragma unroll
                    for (int j = 0; j < W - 1; ++j) z = fmaf(w[j][c], win[j][c], z);
                    z = fmaf(w[W - 1][c], x[c], z);
                    const float sg = cv_sigm(z);
                    dz = g[c] * sg * fmaf(z, 1.f - sg, 1.f);
                }
#pragma unroll
                for (int d = W - 1; d >= 1; --d)
                    dx[d][c] = INSIDE || d <= reach ? fmaf(w[W - 1 - d][c], dz, dx[d - 1][c]) : dx[d - 1][c];
                dx[0][c] = w[W - 1][c] * dz;
                if (INSIDE || (mine & 1)) {
#pragma unroll
                    for (int j = 0; j < W - 1; ++j) gw[j][c] = fmaf(dz, win[j][c], gw[j][c]);
                    gw[W - 1][c] = fmaf(dz, x[c], gw[W - 1][c]);
                    gw[W][c] += dz;
                }
#pragma unroll
                for (int j = 0; j + 1 < W - 1; ++j) win[j][c] = win[j + 1][c];
                win[W - 2][c] = x[c];
            }
            if (mine >> (W - 1) & 1) Vec<InT>::store(q.gx, (row - (W - 1)) * p.channels + c0, dx[W - 1]);
        };
        for (int64_t r = r0; r < r2;) {
            if (p.activation && r >= k.s.start + W - 1 && r + CB_AHEAD <= k.s.end && r + CB_AHEAD <= r1) {
#pragma unroll
                for (int i = 0; i < CB_AHEAD; ++i) {
                    step(std::true_type{}, i, r + i);
                    __builtin_amdgcn_sched_barrier(0);   // (four rows at once: 184 registers)
                }
                r += CB_AHEAD;
            } else {
                step(std::false_type{}, 0, r);
                const auto x0 = xa[0];
                const auto g0 = ga[0];
#pragma unroll
                for (int i = 0; i + 1 < CB_AHEAD; ++i) {
                    xa[i] = xa[i + 1];
                    ga[i] = ga[i + 1];
                }
                xa[CB_AHEAD - 1] = x0;
                ga[CB_AHEAD - 1] = g0;
                ++r;
            }
        }
    }
    __shared__ float sum[CV_WAVES / 2][W + 1][4][64];
#pragma unroll
    for (int half = CV_WAVES / 2; half >= 1; half /= 2) {
        if (wave >= half && wave < 2 * half) {
#pragma unroll
            for (int j = 0; j <= W; ++j)
#pragma unroll
                for (int c = 0; c < 4; ++c) sum[wave - half][j][c][lane] = gw[j][c];
        }
        __syncthreads();
        if (wave < half) {
#pragma unroll
            for (int j = 0; j <= W; ++j)
#pragma unroll
                for (int c = 0; c < 4; ++c) gw[j][c] += sum[wave][j][c][lane];
        }
        __syncthreads();
    }
    if (wave == 0 && live) {
#pragma unroll
        for (int j = 0; j <= W; ++j)
            Vec<float>::store(q.partial, ((int64_t)rb * (W + 1) + j) * p.channels + c0, gw[j]);
    }
}

constexpr int CB_TAIL = 256;   // threads of the launch behind it

// Sums the partial weight gradients: 64 columns by 4 strides per workgroup.
template <int W>
__device__ __forceinline__ void conv_bwd_reduce(const ConvBwdParams& q, int64_t n_part) {
    const int64_t cols = (int64_t)(W + 1) * q.f.channels;
    const int64_t col = (int64_t)blockIdx.x * 64 + (threadIdx.x & 63);
    const int k = threadIdx.x >> 6;
    float a = 0.f;
    if (col < cols)
        for (int64_t i = k; i < n_part; i += 32) {   // eight loads in flight
            float v[8];
#pragma unroll
            for (int j = 0; j < 8; ++j) v[j] = i + 4 * j < n_part ? q.partial[(i + 4 * j) * cols + col] : 0.f;
#pragma unroll
            for (int j = 0; j < 8; ++j) a += v[j];
        }
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
__device__ __forceinline__ void conv_bwd_cache(const ConvBwdParams& q, int64_t block) {
    constexpr int N = 4;
    const ConvParams& p = q.f;
    const int64_t nv = p.channels / N;
    const int64_t idx = block * CB_TAIL + threadIdx.x;
    if (idx >= nv * p.n_seqs) return;
    const int64_t n = idx / nv, c0 = (idx - n * nv) * N;
    const Seq s = seq_range(p, n);
    float w[W][N], in[2 * (W - 1)][N], gc[W - 1][N];
    load_w<W, N>(p.w, c0, w);
    const int64_t len = s.end - s.start;
#pragma unroll
    for (int j = 0; j < 2 * (W - 1); ++j) {   // positions 1 - W .. W - 2
        const int64_t pos = j - (W - 1);
        if (pos < len) input_at<InT, W>(p, s, pos, c0, in[j]);
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
        load4<InT>(q.gy, (s.start + t) * q.gy_stride + c0, g);
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

// Both in one launch: the first `sums` workgroups add up, the others take the
// cache.
template <typename InT, int W>
__global__ __launch_bounds__(CB_TAIL) void conv_bwd_tail_kernel(ConvBwdParams q, int64_t n_part, int64_t sums) {
    if (blockIdx.x < sums) conv_bwd_reduce<W>(q, n_part);
    else conv_bwd_cache<InT, W>(q, (int64_t)blockIdx.x - sums);
}

template <typename InT, int W>
static hipError_t run_conv_fwd(const ConvParams& p, hipStream_t stream) {
    if (p.rows > 0) {
        const int32_t rpw = (int32_t)conv_rows_per_wave(p.rows, p.channels);
        const dim3 grid((unsigned)(cv_strips(p.channels) * ((p.rows + CV_WAVES * rpw - 1) / (CV_WAVES * rpw))));
        hipLaunchKernelGGL((conv_fwd_kernel<InT, W>), grid, dim3(CV_THREADS), 0, stream, p, rpw);
    }
    if (p.cache) {
        const int64_t n = (int64_t)p.n_seqs * (p.channels / 4);
        hipLaunchKernelGGL((conv_cache_update_kernel<InT, W>), dim3((unsigned)((n + 63) / 64)), dim3(64), 0, stream, p);
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
    const ConvParams& p = q.f;
    const int64_t parts = conv_bwd_parts(p.rows, p.channels);
    if (parts > 0) {
        const dim3 grid((unsigned)(cv_strips(p.channels) * parts));
        hipLaunchKernelGGL((conv_bwd_kernel<InT, W>), grid, dim3(CV_THREADS), 0, stream, q);
    }
    const int64_t sums = ((int64_t)(W + 1) * p.channels + 63) / 64;
    const int64_t lanes = q.gcache ? (int64_t)p.n_seqs * (p.channels / 4) : 0;
    hipLaunchKernelGGL((conv_bwd_tail_kernel<InT, W>), dim3((unsigned)(sums + (lanes + CB_TAIL - 1) / CB_TAIL)),
                       dim3(CB_TAIL), 0, stream, q, parts, sums);
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
