// Device-side pieces shared by the attention kernels (gfx950 only): which rows
// a workgroup has, and where its keys and values lie.
#pragma once

#include "kda_attn_launch.h"
#include "kda_device.h"

namespace kda {

constexpr float kLog2e = 1.44269504088896340736f, kLn2 = 0.69314718055994530942f;
constexpr float kAttnLowest = -3.0e38f;   // below every score
__device__ __forceinline__ float attn_exp2(float x) { return __builtin_amdgcn_exp2f(x); }

// Token rows [start, end) of sequence n, clamped into [0, rows].
struct AttnRange {
    int64_t start, end;
};
__device__ __forceinline__ AttnRange attn_range(const int32_t* cu, int64_t rows, int64_t T, int64_t n) {
    if (!cu) return AttnRange{n * T, n * T + T};
    int64_t a = cu[n], b = cu[n + 1];
    a = a < 0 ? 0 : (a > rows ? rows : a);
    b = b < a ? a : (b > rows ? rows : b);
    return AttnRange{a, b};
}

// The block of `block` rows (`per` rows to a token) that a slot stands for
// (see AttnParams); j -1: an unused slot.
struct AttnBlock {
    int64_t start;     // first token row of the sequence
    int32_t n, j;      // sequence, block of it
    int32_t tokens;    // of the sequence
    int32_t r0, r1;    // rows [r0, r1) of the sequence's tokens * per
};
__device__ __forceinline__ AttnBlock attn_block(const AttnParams& p, int64_t slot, int per, int block) {
    AttnBlock b;
    int64_t j;
    if (!p.cu) {
        const int64_t each = (p.T * per + block - 1) / block;
        b.n = (int32_t)(slot / each);
        j = slot - (int64_t)b.n * each;
    } else {
        int lo = 0, hi = p.n_seqs;   // largest n whose first slot is not past this one
        while (hi - lo > 1) {
            const int mid = (lo + hi) >> 1;
            if (attn_range(p.cu, p.rows, p.T, mid).start * per / block + mid <= slot) lo = mid;
            else hi = mid;
        }
        b.n = lo;
        j = slot - (attn_range(p.cu, p.rows, p.T, lo).start * per / block + lo);
    }
    const AttnRange r = attn_range(p.cu, p.rows, p.T, b.n);
    b.start = r.start;
    b.tokens = (int32_t)(r.end - r.start);
    const int64_t n_rows = (int64_t)b.tokens * per, r0 = j * block;
    b.j = j < 0 || r0 >= n_rows ? -1 : (int32_t)j;
    b.r0 = b.j < 0 ? 0 : (int32_t)r0;
    b.r1 = b.j < 0 ? 0 : (int32_t)(r0 + block < n_rows ? r0 + block : n_rows);
    return b;
}

// Tokens that request n holds, in [0, max_pages * page].
__device__ __forceinline__ int32_t attn_length(const AttnParams& p, int n) {
    const int64_t most = (int64_t)p.max_pages << p.page_shift;
    const int32_t len = p.lengths[n];
    return len < 0 ? 0 : (int32_t)(len < most ? len : most);
}

// Keys and values of one (sequence, group).
template <typename InT, bool PAGED>
struct AttnKeys {
    const InT *k, *v;          // first token's row, or page 0, of this group
    int64_t k_stride, v_stride;
    const int32_t* pages;      // of this request
    int32_t n_pages, shift, D;
    __device__ __forceinline__ AttnKeys(const AttnParams& p, int n, int64_t start, int g) {
        D = p.D;
        if constexpr (PAGED) {
            shift = p.page_shift;
            k = (const InT*)p.k + ((int64_t)g << shift) * D;
            v = (const InT*)p.v + ((int64_t)g << shift) * D;
            k_stride = v_stride = p.page_stride;
            pages = p.table + (int64_t)n * p.max_pages;
            n_pages = p.n_pages;
        } else {
            k = (const InT*)p.k + start * p.k_stride + (int64_t)g * D;
            v = (const InT*)p.v + start * p.v_stride + (int64_t)g * D;
            k_stride = p.k_stride;
            v_stride = p.v_stride;
        }
    }
    // Offsets of token x's rows (0 <= x < the sequence's length); false: its page is none.
    __device__ __forceinline__ bool at(int32_t x, int64_t& ko, int64_t& vo) const {
        if constexpr (PAGED) {
            const int32_t page = pages[x >> shift];
            ko = vo = (int64_t)page * k_stride + (int64_t)(x & ((1 << shift) - 1)) * D;
            return page >= 0 && page < n_pages;
        } else {
            ko = (int64_t)x * k_stride;
            vo = (int64_t)x * v_stride;
            return true;
        }
    }
};

// Four values as float32.
__device__ __forceinline__ void load4(const float* p, float (&x)[4]) {
    const f32x4 r = *reinterpret_cast<const f32x4*>(p);
#pragma unroll
    for (int i = 0; i < 4; ++i) x[i] = r[i];
}
__device__ __forceinline__ void load4(const __bf16* p, float (&x)[4]) {
    const u32x2 r = *reinterpret_cast<const u32x2*>(p);
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        x[2 * i] = bf2_first(r[i]);
        x[2 * i + 1] = bf2_second(r[i]);
    }
}
__device__ __forceinline__ void store4(float* p, const float (&x)[4]) {
    f32x4 r;
#pragma unroll
    for (int i = 0; i < 4; ++i) r[i] = x[i];
    *reinterpret_cast<f32x4*>(p) = r;
}
__device__ __forceinline__ void store4(__bf16* p, const float (&x)[4]) {
    *reinterpret_cast<u32x2*>(p) = u32x2{pack_bf2(x[0], x[1]), pack_bf2(x[2], x[3])};
}

// A value that every lane has, where the compiler does not know that.
__device__ __forceinline__ int64_t uniform(int64_t x) {
    const uint32_t lo = __builtin_amdgcn_readfirstlane((uint32_t)x), hi = __builtin_amdgcn_readfirstlane((uint32_t)((uint64_t)x >> 32));
    return (int64_t)((uint64_t)hi << 32 | lo);
}
// 1 / l and lse of a row with the sum of weights l over its maximum m (base 2); a
// row that sees nothing has l = 0, and a NaN (from q or k) stays one.
__device__ __forceinline__ float attn_inverse(float l) { return l == 0.f ? 0.f : 1.f / l; }
__device__ __forceinline__ float attn_lse(float m, float l) { return l == 0.f ? -INFINITY : (m + log2f(l)) * kLn2; }
// Over the four 16-lane groups of a wave (lanes with equal l & 15).
__device__ __forceinline__ float groups_max(float x) {
    x = fmaxf(x, __shfl_xor(x, 16));
    return fmaxf(x, __shfl_xor(x, 32));
}
__device__ __forceinline__ float groups_sum(float x) {
    x += __shfl_xor(x, 16);
    return x + __shfl_xor(x, 32);
}

// The kernel's AttnParams (its first argument), read anew: what only the rare path
// below needs is not to be held in registers through the loops before it.
__device__ __forceinline__ const AttnParams& attn_params_again() {
    const char* at = (const char*)__builtin_amdgcn_kernarg_segment_ptr();
    asm volatile("" : "+s"(at));
    return *reinterpret_cast<const AttnParams*>(at);
}

// (and the thread's number, so that nothing is formed from it ahead of the path)
__device__ __forceinline__ int thread_again() {
    int tid = threadIdx.x;
    asm volatile("" : "+v"(tid));
    return tid;
}

// A row once more, key by key.  The products of a tile take every key's values
// with the row's weight, which is zero for a key that the row does not see, and
// zero times a NaN or an infinity is NaN.  So a row whose sums are not finite,
// though its weights are, comes here: false if those sums stand (unless
// `anyway`), which is where no key in [sees, k1), which its tiles held beside
// those that it sees, has such a value at the same place, or one that it sees
// has, too; else of its keys in [k0, sees) the largest score m (base 2), l = sum
// of e^{s - m} and y = sum of e^{s - m} v, value 64 e + lane in y[e].  All lanes
// of a wave share one row.
template <typename InT, int D, bool PAGED>
__device__ __forceinline__ bool attn_row_again(const AttnParams& p, int n, int64_t start, int g, int64_t row, int head, int32_t k0,
                                               int32_t sees, int32_t k1, float (&y)[D / 64], float& m, float& l, bool anyway = false) {
    const AttnKeys<InT, PAGED> keys(p, n, start, g);
    const InT* q = (const InT*)p.q + row * p.q_stride + (int64_t)head * D;
    const float c = p.scale * kLog2e;
    const int lane = thread_again() & 63;
    const int32_t end = sees < k1 ? sees : k1;
    int64_t ko, vo;
    if (!anyway) {
        auto not_finite = [&](int32_t j) {   // bit e: value 64 e + lane of key j
            uint32_t bits = 0;
            if (j >= k0 && keys.at(j, ko, vo)) {
#pragma unroll
                for (int e = 0; e < D / 64; ++e) {
                    const float x = to_f32(keys.v[vo + 64 * e + lane]);
                    bits |= (x - x == 0.f ? 0u : 1u) << e;
                }
            }
            return bits;
        };
        uint32_t odd = 0;
#pragma unroll 1
        for (int32_t j = sees > k0 ? sees : k0; j < k1; ++j) odd |= not_finite(j);
        for (int32_t j = end - 1; j >= k0 && __any(odd); j -= 8) {
            uint32_t had = 0;
#pragma unroll
            for (int i = 0; i < 8; ++i) had |= not_finite(j - i);
            odd &= ~had;
        }
        if (!__any(odd)) return false;
    }
    m = kAttnLowest;
    l = 0.f;
#pragma unroll
    for (int e = 0; e < D / 64; ++e) y[e] = 0.f;
    for (int32_t j0 = k0; j0 < end; j0 += 64) {
        const bool there = j0 + lane < end && keys.at(j0 + lane, ko, vo);
        if (!there) ko = vo = 0;
        float s = 0.f;
        if (there)
#pragma unroll 4
            for (int d = 0; d < D; d += 4) {
                float a[4], b[4];
                load4(q + d, a);
                load4(keys.k + ko + d, b);
#pragma unroll
                for (int e = 0; e < 4; ++e) s = fmaf(a[e], b[e], s);
            }
        float top = there ? s * c : kAttnLowest;
#pragma unroll
        for (int d = 1; d < 64; d <<= 1) top = fmaxf(top, __shfl_xor(top, d));
        const float to = fmaxf(m, top), fade = attn_exp2(m - to);
        m = to;
        const float w = there ? attn_exp2(fmaf(s, c, -m)) : 0.f;
        float sum = w;
#pragma unroll
        for (int d = 1; d < 64; d <<= 1) sum += __shfl_xor(sum, d);
        l = l * fade + sum;
#pragma unroll
        for (int e = 0; e < D / 64; ++e) y[e] *= fade;
        const uint64_t some = __ballot(there);
#pragma unroll 1
        for (int i0 = 0; i0 < 64; i0 += 8) {
            float x[8][D / 64];
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const InT* at = keys.v + (((int64_t)__shfl((int32_t)(vo >> 32), i0 + i) << 32) | (uint32_t)__shfl((int32_t)vo, i0 + i));
#pragma unroll
                for (int e = 0; e < D / 64; ++e) x[i][e] = some >> (i0 + i) & 1 ? to_f32(at[64 * e + lane]) : 0.f;
            }
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const float wi = __shfl(w, i0 + i);
#pragma unroll
                for (int e = 0; e < D / 64; ++e) y[e] = fmaf(wi, x[i][e], y[e]);
            }
        }
    }
    return true;
}

// Workgroup numbers for work that shrinks from the first workgroup to the last:
// every second round of one workgroup per compute unit (32 of each XCD) is
// turned round, so that the units' shares are alike.
__device__ __forceinline__ uint32_t attn_zigzag(uint32_t w, uint32_t n, int32_t G) {
    const uint32_t x = G % 8 == 0 ? w & 7 : 0, step = G % 8 == 0 ? 8 : 1, wide = 256 / step;
    const uint32_t i = w / step, round = i / wide;
    if (!(round & 1) || (round + 1) * wide > n / step) return w;
    return (2 * round * wide + wide - 1 - i) * step + x;
}

// The same for kernels of two workgroups per compute unit whose workgroups come
// and go: turned if there are two rounds of them at most.  Causal prompts of
// 2048 / 4096 / 8192 tokens, 32 heads of 128 on 8 (512 / 1024 / 2048
// workgroups), on one machine: 47, 145 and 522 us turned, 49, 147 and 514 as
// they are.
__device__ __forceinline__ uint32_t attn_turned(uint32_t w, uint32_t n, int32_t G) {
    return n <= 1024 ? attn_zigzag(w, n, G) : w;
}

// Workgroups of one (sequence, group) on one XCD (workgroup w starts on XCD w
// mod 8), so that its keys and values stay in that L2: workgroup w works on
// item `at` of group `g`.  Groups are dealt to the XCDs in turn; where they do
// not divide by 8, the items are dealt in their own order.
struct AttnPlace {
    int64_t item;
    int32_t g;
};
__device__ __forceinline__ AttnPlace attn_place(uint32_t w, int64_t items, int32_t G) {
    AttnPlace a;
    if (G % 8 == 0) {
        const uint32_t x = w & 7, i = w >> 3;
        a.g = (int32_t)(x + 8 * (i / (uint32_t)items));
        a.item = i % (uint32_t)items;
    } else {
        a.g = (int32_t)(w % (uint32_t)G);
        a.item = w / (uint32_t)G;
    }
    return a;
}

// grad_k and grad_v from their parts, in order.
template <typename OutT, int D>
__global__ __launch_bounds__(256) void attn_bwd_join_kernel(AttnBwdParams a) {
    const AttnParams& p = a.f;
    const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x, item = i / (D / 2);   // (row, group); four values per thread
    if (item >= p.rows * p.G) return;
    const int64_t row = item / p.G;
    const int g = (int)(item - row * p.G), d = (int)(i % (D / 2)) * 4;
    if (p.cu && (row < attn_range(p.cu, p.rows, p.T, 0).start || row >= attn_range(p.cu, p.rows, p.T, p.n_seqs - 1).end)) return;
    float s[4] = {0.f, 0.f, 0.f, 0.f};
    for (int part = 0; part < a.parts; ++part) {
        float x[4];
        load4(a.part + ((part * p.rows * p.G + item) * 2) * D + d, x);
#pragma unroll
        for (int e = 0; e < 4; ++e) s[e] += x[e];
    }
    if (d < D) {
#pragma unroll
        for (int e = 0; e < 4; ++e) s[e] *= p.scale;
        store4((OutT*)a.gk + row * a.gk_stride + (int64_t)g * D + d, s);
    } else {
        store4((OutT*)a.gv + row * a.gv_stride + (int64_t)g * D + d - D, s);
    }
}

}  // namespace kda
