// Verification of drafted tokens (gfx950).  Semantics: include/kda_spec.h.
//
// Per request: K pairs of gathered probabilities, then the sum of
// r = max(p - q, 0) over one row of the vocabulary and a search in its
// running sum.  Bound by HBM: the row of p and of q, read once.  A single
// compute unit reads far below the memory's rate, so the row is cut into
// parts of kVerifyPart entries.  The first launch finds the row (every
// workgroup evaluates the K tests itself, one draft per lane) and sums r and
// p over its parts; the second finds the part that holds the threshold and
// searches that part only (32 KB at most, out of cache).  The tests are three
// dependent reads before the first one of the row, so a workgroup takes as
// many parts as still leave every compute unit full (p.run), each requested
// before the one before it is summed.
//
// All sums and products are float64: the drawn token is the first one whose
// running sum passes u * total, and float32 sums over 10^5 entries would move
// that border by whole tokens.  Vector float64 adds run at half the float32
// rate here, far above what the reads need.
#include "kda_ssm_tile.h"

namespace kda {

constexpr int VF_THREADS = kVerifyThreads;
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
    if (lane < p.K) {
        d = p.drafts[b * p.K + lane];
        const float u = p.u[b * p.K + lane];
        if (d >= 0 && d < p.V && lane < kb) {
            const double pd = vf_mass(((const InT*)p.p)[(b * (p.K + 1) + lane) * p.V + d]);
            const double qd = p.q ? vf_mass(((const InT*)p.q)[(b * p.K + lane) * p.V + d]) : 1.0;
            stands = (double)u * qd < pd;
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

// Entries of a request's row, as rows of any alignment (V may be odd) and 16
// bytes at a time.
template <typename InT>
struct VfRow {
    static constexpr int W = 16 / (int)sizeof(InT);
    typedef InT Vec __attribute__((ext_vector_type(W), aligned(sizeof(InT))));
    const InT* pr;
    const InT* qr;   // nullptr: no q row to subtract
    int64_t V;
    int32_t cut;
    // n: the row; q's is there for a draft that fell
    __device__ __forceinline__ VfRow(const VerifyParams& p, int64_t b, int n, bool residual, int32_t c) {
        pr = (const InT*)p.p + (b * (p.K + 1) + n) * p.V;
        qr = p.q && residual ? (const InT*)p.q + (b * p.K + n) * p.V : nullptr;
        V = p.V;
        cut = c;
    }
    struct Piece {
        Vec p, q;
    };
    // entries v .. v + W - 1; zeros behind the row's end
    __device__ __forceinline__ void load(Piece& to, int64_t v) const {
        if (v + W <= V) {
            to.p = *reinterpret_cast<const Vec*>(pr + v);
            if (qr) to.q = *reinterpret_cast<const Vec*>(qr + v);
        } else {
#pragma unroll
            for (int i = 0; i < W; ++i) {
                to.p[i] = v + i < V ? pr[v + i] : (InT)0.f;
                if (qr) to.q[i] = v + i < V ? qr[v + i] : (InT)0.f;
            }
        }
    }
    // r and p of entry i of a piece that starts at v
    __device__ __forceinline__ void get(const Piece& from, int i, int64_t v, double& rest, double& mass) const {
        mass = vf_mass((InT)from.p[i]);
        rest = mass;
        if (qr) {
            rest -= vf_mass((InT)from.q[i]);
            rest = rest > 0.0 ? rest : 0.0;
        }
        if (v + i == cut) rest = 0.0;
    }
};

// What the first launch leaves in tokens[n_accepted] for the second (a cut
// draft's number: that draft's mass leaves the row).
constexpr int32_t kVfResidual = -1, kVfAll = -2;

template <typename InT>
__global__ __launch_bounds__(VF_THREADS) void verify_sum_kernel(VerifyParams p) {
    constexpr int W = VfRow<InT>::W, PIECES = VF_EACH / W;
    const int tid = threadIdx.x;
    const int runs = (p.n_parts + p.run - 1) / p.run;
    const int64_t b = blockIdx.x / (uint32_t)runs;
    const int part0 = (int)(blockIdx.x - (uint32_t)b * runs) * p.run;
    const int part1 = part0 + p.run < p.n_parts ? part0 + p.run : p.n_parts;
    const VerifyRow row = verify_row<InT>(p, b);
    const VfRow<InT> e(p, b, row.n_acc, row.residual, row.cut);
    if (part0 == 0 && tid <= p.K) {
        if (tid == 0) p.n_accepted[b] = row.n_acc;
        const int32_t code = !row.residual ? kVfAll : row.cut >= 0 ? row.cut : kVfResidual;
        p.tokens[b * (p.K + 1) + tid] = tid < row.n_acc ? p.drafts[b * p.K + tid] : (tid == row.n_acc ? code : -1);
    }
    __shared__ double s[2][2][VF_THREADS / 64];
    typename VfRow<InT>::Piece now[PIECES], next[PIECES];
    auto load = [&](typename VfRow<InT>::Piece (&to)[PIECES], int part) {
#pragma unroll
        for (int i = 0; i < PIECES; ++i) e.load(to[i], part * kVerifyPart + (i * VF_THREADS + tid) * W);
    };
    load(now, part0);
    for (int part = part0; part < part1; ++part) {
        if (part + 1 < part1) load(next, part + 1);
        double r = 0.0, m = 0.0;
#pragma unroll
        for (int i = 0; i < PIECES; ++i)
#pragma unroll
            for (int k = 0; k < W; ++k) {
                double a, c;
                e.get(now[i], k, part * kVerifyPart + (i * VF_THREADS + tid) * W, a, c);
                r += a;
                m += c;
            }
        r = wave_last_f64(wave_scan_f64(r));
        m = wave_last_f64(wave_scan_f64(m));
        auto& to = s[part & 1];   // (two: the last part's may still be read)
        if ((tid & 63) == 0) {
            to[0][tid >> 6] = r;
            to[1][tid >> 6] = m;
        }
        lds_barrier();
        if (tid < 2) p.partial[(b * p.n_parts + part) * 2 + tid] = (to[tid][0] + to[tid][1]) + (to[tid][2] + to[tid][3]);
#pragma unroll
        for (int i = 0; i < PIECES; ++i) now[i] = next[i];
    }
}

// Exclusive prefix sum over the workgroup's threads; `total` gets the sum.
__device__ __forceinline__ double vf_scan(double x, double* lds, double& total) {
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const double inc = wave_scan_f64(x);
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

// Steps of few reads in sequence, bound by their latency.
template <typename InT>
__global__ __launch_bounds__(VF_THREADS) void verify_pick_kernel(VerifyParams p) {
    constexpr int W = VfRow<InT>::W, PIECES = VF_EACH / W;
    const int64_t b = blockIdx.x;
    const int tid = threadIdx.x, lane = tid & 63;
    __shared__ double lds[3][VF_THREADS / 64];
    __shared__ int s_part, s_last, s_token, s_end;
    __shared__ double s_before;
    if (tid == 0) {
        s_part = s_token = INT32_MAX;
        s_last = s_end = -1;
    }
    int32_t* tokens = p.tokens + b * (p.K + 1);
    const int n = p.n_accepted[b];
    const int32_t left = lane < p.K ? tokens[lane] : kVfAll;
    const float u = p.u_next[b];
    // totals of r and of p over the parts, a run of them per thread
    const double* part = p.partial + b * p.n_parts * 2;
    const int each = (p.n_parts + VF_THREADS - 1) / VF_THREADS;
    const int i0 = tid * each < p.n_parts ? tid * each : p.n_parts;
    const int i1 = i0 + each < p.n_parts ? i0 + each : p.n_parts;
    double r = 0.0, m = 0.0, total_r, total_m;
    for (int i = i0; i < i1; ++i) {
        r += part[2 * i];
        m += part[2 * i + 1];
    }
    const double before_r = vf_scan(r, lds[0], total_r), before_m = vf_scan(m, lds[1], total_m);
    const int32_t code = n < 64 ? __shfl(left, n) : kVfAll;   // (lane K and later: all stand)
    const VfRow<InT> e(p, b, n, code != kVfAll, code >= 0 ? code : -1);
    const int which = total_r > 0.0 ? 0 : 1;
    const double total = which ? total_m : total_r;
    int32_t token = 0;
    if (total > 0.0) {
        const double goal = (double)u * total;
        // the part in which the running sum passes the goal, or the last
        // one that holds anything (rounding can leave the goal unpassed)
        double run = which ? before_m : before_r;
        int first = INT32_MAX, last = -1;
        double start = 0.0;
        for (int i = i0; i < i1; ++i) {
            const double x = part[2 * i + which];
            if (x > 0.0) {
                if (run + x > goal && first == INT32_MAX) {
                    first = i;
                    start = run;
                }
                last = i;
                if (first == INT32_MAX) start = run;
            }
            run += x;
        }
        if (first != INT32_MAX) atomicMin(&s_part, first);
        if (last >= 0) atomicMax(&s_last, last);
        __syncthreads();
        const bool passed = s_part != INT32_MAX;
        const int hit = passed ? s_part : s_last;
        if ((passed ? first : last) == hit) s_before = start;
        // a run of VF_EACH entries per thread
        const int64_t v0 = (int64_t)hit * kVerifyPart + (int64_t)tid * VF_EACH;
        typename VfRow<InT>::Piece in[PIECES];
#pragma unroll
        for (int i = 0; i < PIECES; ++i) e.load(in[i], v0 + i * W);
        double val[VF_EACH], mine = 0.0;
#pragma unroll
        for (int i = 0; i < VF_EACH; ++i) {
            double a, c;
            e.get(in[i / W], i % W, v0 + i / W * W, a, c);
            val[i] = which ? c : a;
            mine += val[i];
        }
        double sum;
        run = vf_scan(mine, lds[2], sum);
        run += s_before;
        int found = INT32_MAX, end = -1;
#pragma unroll
        for (int i = 0; i < VF_EACH; ++i) {
            run += val[i];
            if (val[i] > 0.0) {
                end = (int)(v0 + i);
                if (run > goal && found == INT32_MAX) found = (int)(v0 + i);
            }
        }
        if (found != INT32_MAX) atomicMin(&s_token, found);
        if (end >= 0) atomicMax(&s_end, end);
        __syncthreads();
        token = passed && s_token != INT32_MAX ? s_token : s_end;
    }
    if (tid == 0) tokens[n] = token;
}

hipError_t launch_verify(const VerifyParams& p, bool bf16_in, hipStream_t stream) {
    const dim3 grid((unsigned)((p.n_parts + p.run - 1) / p.run) * (unsigned)p.B), block(VF_THREADS);
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
