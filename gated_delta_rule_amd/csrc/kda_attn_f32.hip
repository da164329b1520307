// Softmax attention in float32, of whole sequences and of new tokens over a
// paged cache (gfx950).  Semantics: include/kda_attn.h.
//
// One pass over the keys with the running maximum m and sum l of each row:
//   m' = max(m, s), o' = e^{m - m'} o + e^{s - m'} v, l' = e^{m - m'} l + e^{s - m'}.
// A workgroup has 64 rows (4 waves of 16) of one (sequence, group); keys and
// values come 32 at a time through LDS.  S^T = K Q^T leaves lane l with row
// l & 15 and keys 4 (l >> 4) + i: the place that P^T takes as an operand of
// O^T = V^T P^T, so weights go from product to product in registers, and a
// row's maximum and sum are one lane's values and two exchanges.  The next
// tile's rows are requested before the products of this one.
//   Bound by the float32 matrix instructions and the LDS reads in front of them:
// 94 TFLOP/s at 2048 causal tokens, 16 heads of 128 (182 us; 195 with operands
// read as they are needed), where a large product reaches 153.  Heads of 64 are
// held to four waves per SIMD: with three, which the compiler takes by itself,
// chunks of 2 x 1000 tokens over 8000 and 5000, 32 heads on 8, took 1292 us, and
// 1103 with four.
#include "kda_attn_tile.h"

namespace kda {

constexpr int AF_THREADS = 256, AF_KEYS = 32, AF_BLOCK = kAttnBlockF32;

// Rows of a tile of AF_KEYS keys, as float32: eight threads to a row.
template <int D, bool PAGED>
struct KeyStage {
    static constexpr int PER = D / 8;     // values per thread
    float k[PER], v[PER];
    bool ok;
    // key: this thread's; len: keys that exist
    __device__ __forceinline__ void load(const AttnKeys<float, PAGED>& a, int32_t key, int32_t len) {
        int64_t ko = 0, vo = 0;
        ok = key < len && a.at(key, ko, vo);
        const int c = (threadIdx.x & 7) * 4;
#pragma unroll
        for (int i = 0; i < PER / 4; ++i) {
            float x[4] = {0.f, 0.f, 0.f, 0.f}, y[4] = {0.f, 0.f, 0.f, 0.f};
            if (ok) {
                load4(a.k + ko + c + 32 * i, x);
                load4(a.v + vo + c + 32 * i, y);
            }
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                k[4 * i + e] = x[e];
                v[4 * i + e] = y[e];
            }
        }
    }
    __device__ __forceinline__ void put(float* ks, float* vs, int pitch) const {
        const int row = threadIdx.x >> 3, c = (threadIdx.x & 7) * 4;
#pragma unroll
        for (int i = 0; i < PER / 4; ++i) {
            *reinterpret_cast<f32x4*>(ks + row * pitch + c + 32 * i) = f32x4{k[4 * i], k[4 * i + 1], k[4 * i + 2], k[4 * i + 3]};
            *reinterpret_cast<f32x4*>(vs + row * pitch + c + 32 * i) = f32x4{v[4 * i], v[4 * i + 1], v[4 * i + 2], v[4 * i + 3]};
        }
    }
};

// The rows of this wave that `odds` names (by their lanes) once more (attn_row_again), over what has been written of them.
template <int D, bool PAGED>
__device__ __forceinline__ void f32_again(const AttnBlock& b, int g, uint64_t odds, int64_t slot, int split) {
    const AttnParams& p = attn_params_again();
    if (!p.causal) return;
    const int lane = thread_again() & 63, wave = thread_again() >> 6;
    const int32_t len = PAGED ? attn_length(p, b.n) : b.tokens, first = len - b.tokens, most = first + (b.r1 - 1) / p.hpg + 1;
    const int32_t tiles = most > 0 ? (most + AF_KEYS - 1) / AF_KEYS : 0;
    const int32_t t0 = (int32_t)((int64_t)tiles * split / p.splits), t1 = (int32_t)((int64_t)tiles * (split + 1) / p.splits);
    const int32_t k1 = t1 * AF_KEYS < most ? t1 * AF_KEYS : most;
    asm volatile("s_waitcnt vmcnt(0)" ::: "memory");   // (written)
    odds |= odds >> 32;
    for (uint32_t left = (uint32_t)(odds | odds >> 16) & 0xffff; left; left &= left - 1) {
        const int r = __builtin_ctz(left), row = b.r0 + wave * 16 + r, t = row / p.hpg, head = g * p.hpg + row - t * p.hpg;
        float y[D / 64], m, l;
        if (!attn_row_again<float, D, PAGED>(p, b.n, b.start, g, b.start + t, head, t0 * AF_KEYS, first + t + 1, k1, y, m, l)) continue;
        const float inv = attn_inverse(l);
        float* to = p.part + (((slot * p.G + g) * p.splits + split) * AF_BLOCK + wave * 16 + r) * (D + 2);
#pragma unroll
        for (int e = 0; e < D / 64; ++e) {
            if (p.splits > 1) to[64 * e + lane] = y[e];
            else ((float*)p.o)[((b.start + t) * p.H + head) * D + 64 * e + lane] = y[e] * inv;
        }
        if (p.splits > 1 && lane == 0) {
            to[D] = l;
            to[D + 1] = m;
        }
    }
}

template <int D, bool PAGED>
__global__ __launch_bounds__(AF_THREADS, D == 64 ? 4 : 1) void attn_fwd_f32_kernel(AttnParams p) {
    constexpr int PITCH = D + 4, S = D / 16;
    __shared__ __attribute__((aligned(16))) float ks[AF_KEYS * PITCH], vs[AF_KEYS * PITCH];
    __shared__ uint8_t there[AF_KEYS];
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6, col = lane & 15, grp = lane >> 4;
    // (2048 tokens, 16 heads of 128: 196 us with every second round turned, 241 without; 4096: 677 and 707)
    const AttnPlace pl = attn_place(attn_zigzag(blockIdx.x, gridDim.x, p.G), p.slots * p.splits, p.G);
    const int64_t slot = p.slots - 1 - pl.item / p.splits;   // (later blocks see more keys)
    const int split = (int)(pl.item % p.splits);
    const AttnBlock b = attn_block(p, slot, p.hpg, AF_BLOCK);
    if (b.j < 0) return;
    const int32_t len = PAGED ? attn_length(p, b.n) : b.tokens;
    const int32_t first = len - b.tokens;                    // position of the first query token
    const int row = b.r0 + wave * 16 + col;
    const bool valid = row < b.r1, idle = b.r0 + __builtin_amdgcn_readfirstlane(wave) * 16 >= b.r1;   // (idle: only fetches)
    const int32_t t = valid ? row / p.hpg : 0;
    const int head = pl.g * p.hpg + (valid ? row - t * p.hpg : 0);
    const int32_t sees = !valid ? 0 : p.causal ? first + t + 1 : len;   // keys [0, sees)
    const int32_t most = p.causal ? first + (b.r1 - 1) / p.hpg + 1 : len;
    const int32_t tiles = most > 0 ? (most + AF_KEYS - 1) / AF_KEYS : 0;
    const int32_t t0 = (int32_t)((int64_t)tiles * split / p.splits), t1 = (int32_t)((int64_t)tiles * (split + 1) / p.splits);

    float q[S][4];
    const float* qrow = (const float*)p.q + (b.start + t) * p.q_stride + (int64_t)head * D;
#pragma unroll
    for (int s = 0; s < S; ++s) load4(qrow + 16 * s + 4 * grp, q[s]);

    const AttnKeys<float, PAGED> keys(p, b.n, b.start, pl.g);
    f32x4 o[S];
#pragma unroll
    for (int s = 0; s < S; ++s) o[s] = f32x4{0.f, 0.f, 0.f, 0.f};
    float m = -INFINITY, l = 0.f;
    const float c = p.scale * kLog2e;
    KeyStage<D, PAGED> st;
    if (t0 < t1) st.load(keys, t0 * AF_KEYS + (tid >> 3), most);
    for (int32_t tile = t0; tile < t1; ++tile) {
        __syncthreads();
        st.put(ks, vs, PITCH);
        if ((tid & 7) == 0) there[tid >> 3] = st.ok;
        __syncthreads();
        if (tile + 1 < t1) st.load(keys, (tile + 1) * AF_KEYS + (tid >> 3), most);
        if (idle) continue;
        // operands are read one product (of 16 keys or values) ahead, where the fences keep them
        float kf[2][2][4], vf[2][4];
        auto key_rows = [&](int s, float (&a)[2][4]) {
#pragma unroll
            for (int kt = 0; kt < 2; ++kt) load4(ks + (16 * kt + col) * PITCH + 16 * s + 4 * grp, a[kt]);
        };
        auto value_cols = [&](int i, float (&a)[4]) {   // i = kt S + s
#pragma unroll
            for (int e = 0; e < 4; ++e) a[e] = vs[(16 * (i / S) + 4 * grp + e) * PITCH + 16 * (i % S) + col];
        };
        f32x4 acc[2] = {{0.f, 0.f, 0.f, 0.f}, {0.f, 0.f, 0.f, 0.f}};
        key_rows(0, kf[0]);
#pragma unroll
        for (int s = 0; s < S; ++s) {
            if (s + 1 < S) key_rows(s + 1, kf[(s + 1) & 1]);
            else value_cols(0, vf[0]);
            __builtin_amdgcn_sched_barrier(0);
#pragma unroll
            for (int e = 0; e < 4; ++e)
#pragma unroll
                for (int kt = 0; kt < 2; ++kt) acc[kt] = mfma4f(kf[s & 1][kt][e], q[s][e], acc[kt]);
            __builtin_amdgcn_sched_barrier(0);
        }
        float x[2][4], top = m;
#pragma unroll
        for (int kt = 0; kt < 2; ++kt)
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int key = 16 * kt + 4 * grp + i;
                x[kt][i] = tile * AF_KEYS + key < sees && (!PAGED || there[key]) ? acc[kt][i] * c : -INFINITY;
                top = fmaxf(top, x[kt][i]);
            }
        top = groups_max(top);
        const float base = top == -INFINITY ? 0.f : top, fade = attn_exp2(m - base);
        m = top;
        l *= fade;
#pragma unroll
        for (int s = 0; s < S; ++s) o[s] *= fade;
#pragma unroll
        for (int kt = 0; kt < 2; ++kt)
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                x[kt][i] = attn_exp2(x[kt][i] - base);
                l += x[kt][i];
            }
#pragma unroll
        for (int i = 0; i < 2 * S; ++i) {
            if (i + 1 < 2 * S) value_cols(i + 1, vf[(i + 1) & 1]);
            __builtin_amdgcn_sched_barrier(0);
            mma_k16<true, PLAIN>(o[i % S], vf[i & 1], x[i / S]);
            __builtin_amdgcn_sched_barrier(0);
        }
    }
    l = groups_sum(l);
    float odd = 0.f;   // NaN if a sum is not finite
#pragma unroll
    for (int s = 0; s < S; ++s)
#pragma unroll
        for (int i = 0; i < 4; ++i) odd = fmaf(o[s][i], 0.f, odd);
    const uint64_t odds = __ballot(valid && odd != 0.f && l - l == 0.f);
    if (valid && p.splits > 1) {
        float* to = p.part + (((slot * p.G + pl.g) * p.splits + split) * AF_BLOCK + (row - b.r0)) * (D + 2);
#pragma unroll
        for (int s = 0; s < S; ++s)
#pragma unroll
            for (int i = 0; i < 4; ++i) to[16 * s + 4 * grp + i] = o[s][i];
        if (grp == 0) {
            to[D] = l;
            to[D + 1] = m;
        }
    } else if (valid) {
        const float inv = attn_inverse(l);
        float* orow = (float*)p.o + ((b.start + t) * p.H + head) * (int64_t)D;
#pragma unroll
        for (int s = 0; s < S; ++s) {
            const float y[4] = {o[s][0] * inv, o[s][1] * inv, o[s][2] * inv, o[s][3] * inv};
            store4(orow + 16 * s + 4 * grp, y);
        }
        if (p.lse && grp == 0) p.lse[(b.start + t) * p.H + head] = attn_lse(m, l);
    }
    if (odds) f32_again<D, PAGED>(b, pl.g, odds, slot, split);
}

// The parts of a split block: o = sum_s e^{m_s - m} o_s / sum_s e^{m_s - m} l_s,
// in the order of the parts.  A wave has a row.
template <int D>
__global__ __launch_bounds__(256) void attn_join_kernel(AttnParams p) {
    constexpr int block = AF_BLOCK;
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const uint32_t per = (uint32_t)block / 4;                 // workgroups of a block
    const uint32_t unit = blockIdx.x / per;
    const int64_t slot = unit / (uint32_t)p.G;
    const int g = (int)(unit % (uint32_t)p.G);
    const AttnBlock b = attn_block(p, slot, p.hpg, block);
    const int r = (int)(blockIdx.x % per) * 4 + wave;
    if (b.j < 0 || b.r0 + r >= b.r1) return;
    const float* from = p.part + ((slot * p.G + g) * p.splits * block + r) * (int64_t)(D + 2);
    const int64_t step = (int64_t)block * (D + 2);
    float m = -INFINITY;
    for (int s = 0; s < p.splits; ++s) m = fmaxf(m, from[s * step + D + 1]);
    const float base = m == -INFINITY ? 0.f : m;
    float l = 0.f, o0 = 0.f, o1 = 0.f;
    for (int s = 0; s < p.splits; ++s) {
        const float* at = from + s * step;
        const float w = attn_exp2(at[D + 1] - base);
        l += w * at[D];
        o0 += w * at[lane];
        if constexpr (D == 128) o1 += w * at[64 + lane];
    }
    const float inv = attn_inverse(l);
    const int row = b.r0 + r, t = row / p.hpg, head = g * p.hpg + row - t * p.hpg;
    float* orow = (float*)p.o + ((b.start + t) * p.H + head) * (int64_t)D;
    orow[lane] = o0 * inv;
    if constexpr (D == 128) orow[64 + lane] = o1 * inv;
    if (p.lse && lane == 0) p.lse[(b.start + t) * p.H + head] = attn_lse(m, l);
}

template <int D>
static void run_fwd(const AttnParams& p, hipStream_t stream) {
    const dim3 grid((uint32_t)(p.slots * p.G * p.splits));
    if (p.lengths) attn_fwd_f32_kernel<D, true><<<grid, AF_THREADS, 0, stream>>>(p);
    else attn_fwd_f32_kernel<D, false><<<grid, AF_THREADS, 0, stream>>>(p);
    if (p.splits > 1) attn_join_kernel<D><<<dim3((uint32_t)(p.slots * p.G * (AF_BLOCK / 4))), 256, 0, stream>>>(p);
}

hipError_t launch_attn_fwd_f32(const AttnParams& p, hipStream_t stream) {
    if (p.slots == 0) return hipSuccess;
    p.D == 64 ? run_fwd<64>(p, stream) : run_fwd<128>(p, stream);
    return hipGetLastError();
}

}  // namespace kda
