// Verification of drafted tokens (gfx950).  Semantics: include/kda_spec.h.
//
// Per request: K pairs of gathered probabilities, then the sum of
// r = max(p - q, 0) over one row of the vocabulary and a search in its
// running sum.  Bound by HBM: the row of p and of q, read once.  A single
// compute unit reads far below the memory's rate, so the row is cut into
// parts of kVerifyPart entries: the first launch finds the row (every
// workgroup evaluates the K tests itself, one draft per lane) and sums its
// part of r and of p; the second finds the part that holds the threshold
// and searches that part only (32 KB at most, out of cache).
//
// All sums and products are float64: the drawn token is the first one whose
// running sum passes u * total, and float32 sums over 10^5 entries would move
// that border by whole tokens.  Vector float64 adds run at half the float32
// rate here, far above what the reads need.
#include "kda_device.h"
#include "kda_ssm_launch.h"

namespace kda {

constexpr int VF_THREADS = 256;
constexpr int VF_EACH = (int)(kVerifyPart / VF_THREADS);   // entries per thread of a part

// What is > 0 counts (NaN and negative values do not).
template <typename T>
__device__ __forceinline__ double vf_mass(T v) {
    const float f = to_f32(v);
    return f > 0.f ? (double)f : 0.0;
}

struct VerifyRow {
    int n_acc;       // drafts that stand
    int32_t cut;     // draft whose mass leaves the row when q is not given, or -1
    bool residual;   // a draft fell: r = max(p - q, 0)
};

// Every wave evaluates the tests of its request, draft i on lane i.
template <typename InT>
__device__ __forceinline__ VerifyRow verify_row(const VerifyParams& p, int64_t b) {
    const int lane = threadIdx.x & 63;
    int kb = p.n_draft ? p.n_draft[b] : p.K;
    kb = kb < 0 ? 0 : (kb > p.K ? p.K : kb);
    bool stands = false;
    int32_t d = -1;
    if (lane < kb) {
        d = p.drafts[b * p.K + lane];
        if (d >= 0 && d < p.V) {
            const double pd = vf_mass(((const InT*)p.p)[(b * (p.K + 1) + lane) * p.V + d]);
            const double qd = p.q ? vf_mass(((const InT*)p.q)[(b * p.K + lane) * p.V + d]) : 1.0;
            stands = (double)p.u[b * p.K + lane] * qd < pd;
        } else {
            d = -1;
        }
    }
    const uint64_t m = ~__ballot(stands);
    int n = m ? __ffsll((unsigned long long)m) - 1 : 64;
    n = n > kb ? kb : n;
    VerifyRow r;
    r.n_acc = n;
    r.residual = n < kb;
    r.cut = __shfl(d, n & 63);
    if (!r.residual || p.q) r.cut = -1;
    return r;
}

// r and p of entry v of the request's row.
template <typename InT>
struct VerifyEntry {
    const InT* pr;
    const InT* qr;   // nullptr: no q row to subtract
    int32_t cut;
    __device__ __forceinline__ VerifyEntry(const VerifyParams& p, int64_t b, const VerifyRow& r) {
        pr = (const InT*)p.p + (b * (p.K + 1) + r.n_acc) * p.V;
        qr = p.q && r.residual ? (const InT*)p.q + (b * p.K + r.n_acc) * p.V : nullptr;
        cut = r.cut;
    }
    __device__ __forceinline__ void get(int64_t v, double& rest, double& mass) const {
        mass = vf_mass(pr[v]);
        rest = mass;
        if (qr) {
            rest -= vf_mass(qr[v]);
            rest = rest > 0.0 ? rest : 0.0;
        }
        if (v == cut) rest = 0.0;
    }
};

__device__ __forceinline__ double vf_wave_sum(double x) {
#pragma unroll
    for (int o = 32; o > 0; o >>= 1) x += __shfl_xor(x, o);
    return x;
}

template <typename InT>
__global__ __launch_bounds__(VF_THREADS) void verify_sum_kernel(VerifyParams p) {
    const int64_t b = blockIdx.x / (uint32_t)p.n_parts;
    const int part = (int)(blockIdx.x - (uint32_t)b * p.n_parts);
    const VerifyRow row = verify_row<InT>(p, b);
    const VerifyEntry<InT> e(p, b, row);
    const int64_t v0 = (int64_t)part * kVerifyPart;
    double r = 0.0, m = 0.0;
#pragma unroll
    for (int i = 0; i < VF_EACH; ++i) {
        const int64_t v = v0 + i * VF_THREADS + threadIdx.x;
        if (v < p.V) {
            double a, c;
            e.get(v, a, c);
            r += a;
            m += c;
        }
    }
    r = vf_wave_sum(r);
    m = vf_wave_sum(m);
    __shared__ double s[2][VF_THREADS / 64];
    if ((threadIdx.x & 63) == 0) {
        s[0][threadIdx.x >> 6] = r;
        s[1][threadIdx.x >> 6] = m;
    }
    __syncthreads();
    if (threadIdx.x < 2)
        p.partial[(b * p.n_parts + part) * 2 + threadIdx.x] =
            (s[threadIdx.x][0] + s[threadIdx.x][1]) + (s[threadIdx.x][2] + s[threadIdx.x][3]);
}

// Exclusive prefix sum over the workgroup's threads; `total` gets the sum.
__device__ __forceinline__ double vf_scan(double x, double* lds, double& total) {
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    double inc = x;
#pragma unroll
    for (int o = 1; o < 64; o <<= 1) {
        const double y = __shfl_up(inc, o);
        if (lane >= o) inc += y;
    }
    __syncthreads();   // lds is free
    if (lane == 63) lds[wave] = inc;
    __syncthreads();
    double before = 0.0;
    total = 0.0;
#pragma unroll
    for (int w = 0; w < VF_THREADS / 64; ++w) {
        if (w < wave) before += lds[w];
        total += lds[w];
    }
    return before + (inc - x);
}

template <typename InT>
__global__ __launch_bounds__(VF_THREADS) void verify_pick_kernel(VerifyParams p) {
    const int64_t b = blockIdx.x;
    const int tid = threadIdx.x;
    __shared__ double lds[VF_THREADS / 64];
    __shared__ int s_part, s_last, s_token;
    __shared__ double s_before;
    const VerifyRow row = verify_row<InT>(p, b);
    const VerifyEntry<InT> e(p, b, row);
    const double* part = p.partial + b * p.n_parts * 2;
    // totals of r and of p over the parts
    double r = 0.0, m = 0.0, total_r, total_m;
    for (int i = tid; i < p.n_parts; i += VF_THREADS) {
        r += part[2 * i];
        m += part[2 * i + 1];
    }
    vf_scan(r, lds, total_r);
    vf_scan(m, lds, total_m);
    const int which = total_r > 0.0 ? 0 : 1;
    const double total = which ? total_m : total_r;
    int32_t token = 0;
    if (total > 0.0) {
        const double goal = (double)p.u_next[b] * total;
        // the part in which the running sum passes the goal, or the last
        // one that holds anything (rounding can leave the goal unpassed)
        if (tid == 0) {
            s_part = INT32_MAX;
            s_last = -1;
        }
        double base = 0.0;
        for (int i0 = 0; i0 < p.n_parts; i0 += VF_THREADS) {
            const int i = i0 + tid;
            const double x = i < p.n_parts ? part[2 * i + which] : 0.0;
            double sum;
            const double before = base + vf_scan(x, lds, sum);
            if (x > 0.0) {
                atomicMax(&s_last, i);
                if (before + x > goal) atomicMin(&s_part, i);
            }
            base += sum;
        }
        __syncthreads();
        const bool passed = s_part != INT32_MAX;
        const int hit = passed ? s_part : s_last;
        // running sum before that part: the same sums, so that it is below the goal
        base = 0.0;
        for (int i0 = 0; i0 <= hit; i0 += VF_THREADS) {
            const int i = i0 + tid;
            const double x = i < p.n_parts ? part[2 * i + which] : 0.0;
            double sum;
            const double before = base + vf_scan(x, lds, sum);
            if (i == hit) s_before = before;
            base += sum;
        }
        if (tid == 0) {
            s_token = INT32_MAX;
            s_last = -1;
        }
        __syncthreads();
        const double start = s_before;
        // a run of VF_EACH entries per thread
        const int64_t v0 = (int64_t)hit * kVerifyPart + (int64_t)tid * VF_EACH;
        double val[VF_EACH], mine = 0.0;
#pragma unroll
        for (int i = 0; i < VF_EACH; ++i) {
            val[i] = 0.0;
            if (v0 + i < p.V) {
                double a, c;
                e.get(v0 + i, a, c);
                val[i] = which ? c : a;
            }
            mine += val[i];
        }
        double sum;
        double run = start + vf_scan(mine, lds, sum);
        int found = INT32_MAX, last = -1;
#pragma unroll
        for (int i = 0; i < VF_EACH; ++i) {
            run += val[i];
            if (val[i] > 0.0) {
                last = (int)(v0 + i);
                if (run > goal && found == INT32_MAX) found = (int)(v0 + i);
            }
        }
        if (found != INT32_MAX) atomicMin(&s_token, found);
        if (last >= 0) atomicMax(&s_last, last);
        __syncthreads();
        token = passed && s_token != INT32_MAX ? s_token : s_last;
    }
    if (tid == 0) p.n_accepted[b] = row.n_acc;
    if (tid <= p.K)
        p.tokens[b * (p.K + 1) + tid] = tid < row.n_acc ? p.drafts[b * p.K + tid] : (tid == row.n_acc ? token : -1);
}

hipError_t launch_verify(const VerifyParams& p, bool bf16_in, hipStream_t stream) {
    const dim3 grid((unsigned)p.n_parts * (unsigned)p.B), block(VF_THREADS);
    if (bf16_in) {
        hipLaunchKernelGGL(verify_sum_kernel<__bf16>, grid, block, 0, stream, p);
        hipLaunchKernelGGL(verify_pick_kernel<__bf16>, dim3((unsigned)p.B), block, 0, stream, p);
    } else {
        hipLaunchKernelGGL(verify_sum_kernel<float>, grid, block, 0, stream, p);
        hipLaunchKernelGGL(verify_pick_kernel<float>, dim3((unsigned)p.B), block, 0, stream, p);
    }
    return hipGetLastError();
}

}  // namespace kda
