// Device-side pieces shared by the scan's forward and backward kernels
// (gfx950 only): the sequence table, the decay sums of a chunk, and operand
// tiles in LDS.
//
// Operands of the bf16 16x16x32 matrix instruction: lane l supplies row (A)
// or column (B) l & 15 and k = 8 (l >> 4) .. + 7; it receives column l & 15,
// rows 4 (l >> 4) .. + 3 of the product.  The two operands have the same
// form, so swapping them transposes the product.
//
// A tile is [rows][columns] of bf16 in LDS, in 16-byte units of 8 columns
// whose place in the row is exclusive-ored with the row number, so that 16
// rows' units of one column block fall into different banks.  A fragment
// whose k runs along the tile's columns is one 16-byte read per lane; one
// whose k runs along its rows takes two transposing reads.
//
// A float32 value enters a product as the sum of bf16 parts (8 significant
// bits each): parts i and j of the two operands are multiplied while
// i + j < 3, the rest is below 2^-24 of the product.  bf16 inputs have one
// part, float32 inputs three (three planes of the tile).
#pragma once

#include "kda_device.h"
#include "kda_ssm_launch.h"

namespace kda {

constexpr int SS_THREADS = 256;

__device__ __forceinline__ float ss_softplus(float x) { return fmaxf(x, 0.f) + log1pf(expf(-fabsf(x))); }

// Token rows [start, end) of sequence n, clamped into [0, rows].
struct SsmRange {
    int64_t start, end;
};
__device__ __forceinline__ SsmRange ssm_range(const int32_t* cu, int64_t rows, int64_t T, int64_t n) {
    if (!cu) return SsmRange{n * T, n * T + T};
    int64_t a = cu[n], b = cu[n + 1];
    a = a < 0 ? 0 : (a > rows ? rows : a);
    b = b < a ? a : (b > rows ? rows : b);
    return SsmRange{a, b};
}
// The sequence and the piece of `len` tokens that a slot stands for (see
// SsmScanParams); piece -1: an unused slot.  Its rows are [r0, r1).
struct SsmPiece {
    int64_t n, piece, r0, r1, start, end;   // start, end: the sequence's
};
__device__ __forceinline__ SsmPiece ssm_piece(const int32_t* cu, int64_t rows, int64_t T, int32_t n_seqs,
                                              int64_t len, int64_t slot) {
    SsmPiece s;
    if (!cu) {
        const int64_t per = (T + len - 1) / len;
        s.n = slot / per;
        s.piece = slot - s.n * per;
    } else {
        int lo = 0, hi = n_seqs;   // largest n with cu[n] / len + n <= slot
        while (hi - lo > 1) {
            const int mid = (lo + hi) >> 1;
            if (ssm_range(cu, rows, T, mid).start / len + mid <= slot) lo = mid;
            else hi = mid;
        }
        s.n = lo;
        s.piece = slot - (ssm_range(cu, rows, T, lo).start / len + lo);
    }
    const SsmRange r = ssm_range(cu, rows, T, s.n);
    s.start = r.start;
    s.end = r.end;
    if (s.piece < 0 || s.piece * len >= r.end - r.start) {
        s.piece = -1;
        s.r0 = s.r1 = r.end;
        return s;
    }
    s.r0 = r.start + s.piece * len;
    s.r1 = s.r0 + len < r.end ? s.r0 + len : r.end;
    return s;
}

// The k-th longest of up to 64 packed sequences (the first of equal ones
// first), by the whole wave: chains start with the longest, so that none of
// them is left over at the end (16 sequences of 150 to 1000 tokens, 96 heads
// of 128: 226 us, 246 in their own order).  Beyond 64 sequences they come in
// their own order; the last ones are then a small part of the whole.
__device__ __forceinline__ int64_t ssm_longest(const int32_t* cu, int64_t rows, int32_t n_seqs, int k) {
    const int i = threadIdx.x & 63;
    const SsmRange r = ssm_range(cu, rows, rows, i < n_seqs ? i : 0);
    const int64_t len64 = r.end - r.start;
    const int len = i < n_seqs ? (int)(len64 < INT32_MAX ? len64 : INT32_MAX) : -1;
    int rank = 0;
    for (int j = 0; j < n_seqs; ++j) {
        const int other = __builtin_amdgcn_readlane(len, j);
        rank += other > len || (other == len && j < i);
    }
    return __ffsll((unsigned long long)__ballot(i < n_seqs && rank == k)) - 1;
}

// Where the walks leave a state's four columns 16 ct + 4 (l >> 4) .. + 3 of row
// 16 m + (l & 15), in 16-byte pieces: tiles of 16 x 16, each 1 KB as a wave
// holds it, so that a store is contiguous (rows of the state in order would
// be 64-byte pieces: 97 against 82 us for 0.27 GB).
template <int N>
__device__ __forceinline__ int walk_at(int ct, int m, int l) {
    return (ct * (N / 16) + m) * 64 + l;
}

typedef short s16x4 __attribute__((ext_vector_type(4)));

// Place of unit u (8 columns) of a row in a tile with U units per row: the 16
// units of the 64 banks.  A number made of the row's bits b3 .. b0 is
// exclusive-ored in, (b1 b0 b3^b2 b2) for 16 units, so that each access's
// lanes, as the hardware groups them, find their units in different places:
// one unit of 16 rows, with its neighbour for half of them (frag_row, 16
// lanes: rows 0-3 and 12-15 of one, 4-11 of the other), and two or four
// neighbouring units of rows 0-3 and 8-11 (frag_col, 32 lanes).  With (b3 b2
// b1 b0) the latter met in twos and fours: 38% of the LDS cycles of the scan's
// full pass, 18% now, 126 against 122.5 us for 8192 tokens of 64 heads.
template <int U>
__device__ __forceinline__ int ss_unit(int row, int u) {
    static_assert(U == 4 || U == 8 || U == 16, "");
    const int low = U == 16 ? (row & 3) << 2 : U == 8 ? (row & 2) << 1 : 0;
    return row * U + (u ^ (low | (((row >> 2) ^ ((row >> 1) & 2)) & 3)));
}

// Where a lane reads its fragments: byte offsets within a tile, for row 0 and
// column 0.  Every other fragment of the tile is that offset with the bytes
// of its first column exclusive-ored in (the columns of a row are whole
// powers of two, and the row's own exclusive-or commutes with it) plus the
// bytes of its first row, so that a fragment costs one instruction of
// address at most.  The kernels hide these offsets from the compiler once per
// chunk: it would otherwise keep all of a loop's addresses in registers, more
// than there are.
//
// k along the columns: row l & 15, columns 8 (l >> 4) .. + 7.
template <int COLS>
__device__ __forceinline__ int lane_row(int l) {
    return 16 * ss_unit<COLS / 8>(l & 15, l >> 4);
}
// k along the rows: lane i = l & 15 supplies rows 8 (l >> 4) + (i >> 2) and 4
// more (x, y), columns STEP (i & 3) .. + 3.
template <int COLS, int STEP>
__device__ __forceinline__ int2 lane_col(int l) {
    const int i = l & 15, c = STEP * (i & 3), r = 8 * (l >> 4) + (i >> 2);
    return make_int2(16 * ss_unit<COLS / 8>(r, c >> 3) + 2 * (c & 7), 16 * ss_unit<COLS / 8>(r + 4, c >> 3) + 2 * (c & 7));
}
__device__ __forceinline__ void hide(int& x) { asm volatile("" : "+v"(x)); }
__device__ __forceinline__ void hide(int2& x) { asm volatile("" : "+v"(x.x), "+v"(x.y)); }

// Fragment with k along the columns: lane l gets row r0 + (l & 15) (r0 a
// multiple of 16), columns 32 ks + 8 (l >> 4) .. + 7.
template <int COLS>
__device__ __forceinline__ bf16x8 frag_row(const __bf16* tile, int r0, int ks, int at) {
    return *reinterpret_cast<const bf16x8*>(reinterpret_cast<const char*>(tile) + r0 * COLS * 2 + (at ^ (64 * ks)));
}
// Fragment with k along the rows: lane i = l & 15 gets column
// c0 + STEP (i >> 2) + (i & 3), rows 32 ks + 8 (l >> 4) .. + 7.  STEP 4 (c0 a
// multiple of 16): 16 neighbouring columns; STEP 8: the pair of calls with c0
// and c0 + 4 (c0 a multiple of 32) covers 32 columns so that a lane's four
// rows of each of the two products (rows 4 (l >> 4) .. + 3) are eight
// neighbouring columns 8 (l >> 4) .. + 7 of the 32.
template <int COLS>
__device__ __forceinline__ bf16x8 frag_col(const __bf16* tile, int c0, int ks, int2 at) {
    const char* t = reinterpret_cast<const char*>(tile) + 32 * ks * COLS * 2;
    const s16x4 lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16((__attribute__((address_space(3))) s16x4*)(t + (at.x ^ (2 * c0))));
    const s16x4 hi = __builtin_amdgcn_ds_read_tr16_b64_v4i16((__attribute__((address_space(3))) s16x4*)(t + (at.y ^ (2 * c0))));
    bf16x8 f;
    __builtin_memcpy(&f, &lo, 8);
    __builtin_memcpy(reinterpret_cast<char*>(&f) + 8, &hi, 8);
    return f;
}

// NP bf16 parts of 8 float32 values; the last part is rounded, so the sum is
// off by at most 2^-8NP of the value.
template <int NP>
__device__ __forceinline__ void parts8(const float (&x)[8], bf16x8 (&p)[NP]) {
    float r[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) r[i] = x[i];
#pragma unroll
    for (int k = 0; k < NP; ++k) {
        u32x4 w;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            w[i] = pack_bf2(r[2 * i], r[2 * i + 1]);
            if (k + 1 < NP) {
                r[2 * i] -= bf2_first(w[i]);
                r[2 * i + 1] -= bf2_second(w[i]);
            }
        }
        p[k] = __builtin_bit_cast(bf16x8, w);
    }
}
// c += sum over parts i of a, j of b with i + j < 3, smallest first.
template <int NA, int NB>
__device__ __forceinline__ f32x4 mma_parts(const bf16x8 (&a)[NA], const bf16x8 (&b)[NB], f32x4 c) {
#pragma unroll
    for (int s = NA + NB - 2; s >= 0; --s) {
        if (s > 2) continue;
#pragma unroll
        for (int i = 0; i < NA; ++i) {
            const int j = s - i;
            if (j >= 0 && j < NB) c = mfma32(a[i], b[j], c);
        }
    }
    return c;
}

// Global memory -> registers -> LDS of a tile of L rows by COLS columns:
// PER 16-byte pieces per thread, rows past `valid` as zeros.
template <typename InT, int L, int COLS, int THREADS>
struct Stager {
    static constexpr int EV = 16 / (int)sizeof(InT);      // elements per piece
    static constexpr int PPR = COLS / EV;                 // pieces per row
    static constexpr int PER = L * PPR / THREADS;
    static constexpr int PARTS = sizeof(InT) == 2 ? 1 : 3;
    static constexpr int ROWS = THREADS / PPR;            // rows per piece of all threads
    static_assert(L * PPR % THREADS == 0 && THREADS % PPR == 0, "whole pieces per thread, whole rows");
    u32x4 r[PER];

    // base: first row's first column; cols: columns that exist (the others read as zero)
    __device__ __forceinline__ void load(const InT* base, int64_t stride, int valid, int cols) {
        const int row = (int)threadIdx.x / PPR, c = ((int)threadIdx.x - row * PPR) * EV;
        const uint32_t off = c < cols ? (uint32_t)(row * (int)stride + c) * (uint32_t)sizeof(InT) : 0x80000000u;
#pragma unroll
        for (int j = 0; j < PER; ++j) {   // (a buffer of the rows that exist: further ones read as zero)
            const int left = valid - j * ROWS;
            const auto rs = make_rsrc(base + j * ROWS * stride, left > 0 ? ((left - 1) * (int)stride + cols) * (int)sizeof(InT) : 0);
            r[j] = __builtin_bit_cast(u32x4, __builtin_amdgcn_raw_buffer_load_b128(rs, off, 0, 0));
        }
    }
    // planes of L * COLS bf16 each
    __device__ __forceinline__ void put(__bf16* tile) const {
#pragma unroll
        for (int j = 0; j < PER; ++j) {
            const int idx = (int)threadIdx.x + THREADS * j;
            const int row = idx / PPR, c = (idx - row * PPR) * EV;
            __bf16* at = tile + 8 * ss_unit<COLS / 8>(row, c >> 3) + (c & 7);
            if constexpr (PARTS == 1) {
                *reinterpret_cast<u32x4*>(at) = r[j];
            } else {
                float f[4];
#pragma unroll
                for (int i = 0; i < 4; ++i) f[i] = __uint_as_float(r[j][i]);
#pragma unroll
                for (int k = 0; k < 3; ++k) {
                    u32x2 w = {pack_bf2(f[0], f[1]), pack_bf2(f[2], f[3])};
                    *reinterpret_cast<u32x2*>(at + k * L * COLS) = w;
#pragma unroll
                    for (int i = 0; i < 2; ++i) {
                        f[2 * i] -= bf2_first(w[i]);
                        f[2 * i + 1] -= bf2_second(w[i]);
                    }
                }
            }
        }
    }
};

// Decay sums of one head's chunk, one token per lane (lanes >= L idle):
// g_t = sum_{s<=t} a_s in float64, kept as hi + lo floats, so that g_t - g_s
// is good to float32 rounding of the difference itself however far both are
// from the chunk's start.
template <int L>
struct __attribute__((aligned(16))) ChunkDecay {
    float gh[L], gl[L];   // g_t
    float dt[L];          // after softplus; 0 past the end
    float eg[L];          // e^{g_t}
    float w[L];           // e^{g_end - g_t} dt_t
    float eL;             // e^{g_end}
};
// Inclusive sum over the wave's lanes up to each one, by DPP row shifts and
// row broadcasts (no LDS round trips).
template <int CTRL, int ROWS>
__device__ __forceinline__ double dpp_add_f64(double x) {
    const uint64_t u = __builtin_bit_cast(uint64_t, x);
    const uint32_t lo = (uint32_t)__builtin_amdgcn_update_dpp(0, (int)(uint32_t)u, CTRL, ROWS, 0xf, false);
    const uint32_t hi = (uint32_t)__builtin_amdgcn_update_dpp(0, (int)(uint32_t)(u >> 32), CTRL, ROWS, 0xf, false);
    return x + __builtin_bit_cast(double, (uint64_t)lo | ((uint64_t)hi << 32));
}
__device__ __forceinline__ double wave_scan_f64(double x) {
    x = dpp_add_f64<0x111, 0xf>(x);   // row_shr:1
    x = dpp_add_f64<0x112, 0xf>(x);   // row_shr:2
    x = dpp_add_f64<0x114, 0xf>(x);   // row_shr:4
    x = dpp_add_f64<0x118, 0xf>(x);   // row_shr:8
    x = dpp_add_f64<0x142, 0xa>(x);   // row_bcast:15 into rows 1 and 3
    x = dpp_add_f64<0x143, 0xc>(x);   // row_bcast:31 into rows 2 and 3
    return x;
}
// The value of lane LANE (the last: 63), for all lanes.
template <int LANE = 63>
__device__ __forceinline__ double wave_last_f64(double x) {
    const uint64_t u = __builtin_bit_cast(uint64_t, x);
    const uint32_t lo = (uint32_t)__builtin_amdgcn_readlane((int)(uint32_t)u, LANE);
    const uint32_t hi = (uint32_t)__builtin_amdgcn_readlane((int)(uint32_t)(u >> 32), LANE);
    return __builtin_bit_cast(double, (uint64_t)lo | ((uint64_t)hi << 32));
}
// Sums over a lane and the later lanes of its 16, and over it and the earlier ones.
__device__ __forceinline__ double row_suffix_f64(double x) {
    x = dpp_add_f64<0x101, 0xf>(x);   // row_shl:1
    x = dpp_add_f64<0x102, 0xf>(x);
    x = dpp_add_f64<0x104, 0xf>(x);
    return dpp_add_f64<0x108, 0xf>(x);
}
__device__ __forceinline__ double row_prefix_f64(double x) {
    x = dpp_add_f64<0x111, 0xf>(x);   // row_shr:1
    x = dpp_add_f64<0x112, 0xf>(x);
    x = dpp_add_f64<0x114, 0xf>(x);
    return dpp_add_f64<0x118, 0xf>(x);
}
// A token's decay below this ends all memory: e^a is zero in float32 (half the
// least subnormal number is e^-103.97).  Decays are cut off at kDecayCut, which
// changes no factor and keeps the sums where their differences are exact to
// float32 rounding: beside a term of -2^40 or an overflow they are not.
constexpr float kDecayEnds = -104.f, kDecayCut = -256.f;
// dt_raw: this lane's token, `valid` whether it exists.  Returns g_end.  The
// factors are stored with the signs se (eg), sw (w) and sL (eL).
template <int L>
__device__ __forceinline__ double chunk_decay(ChunkDecay<L>& d, float dt_raw, bool valid, float bias, int softplus,
                                              float A, float se = 1.f, float sw = 1.f, float sL = 1.f) {
    const int lane = threadIdx.x & 63;
    float dt = 0.f;
    if (valid) {
        dt = dt_raw + bias;
        if (softplus) dt = ss_softplus(dt);
    }
    const float a = dt * A;   // (NaN stays)
    const double g = wave_scan_f64((double)(a < kDecayCut ? kDecayCut : a));
    const double end = wave_last_f64<L - 1>(g);
    if (lane < L) {
        const float h = (float)g;
        d.gh[lane] = h;
        d.gl[lane] = (float)(g - (double)h);
        d.dt[lane] = dt;
        d.eg[lane] = se * expf(h);
        d.w[lane] = sw * (expf((float)(end - g)) * dt);
        if (lane == 0) d.eL = sL * expf((float)end);
    }
    return end;
}

}  // namespace kda
