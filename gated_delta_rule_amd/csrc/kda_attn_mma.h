// Tiles of bf16 rows in LDS and the 32x32x16 matrix instruction, for the
// attention kernels with bf16 inputs (gfx950 only).
//
// Operands of the instruction: lane l supplies row (A) or column (B) l & 31
// and k = 8 (l >> 5) .. + 7; it receives column l & 31, rows 8 b + 4 (l >> 5) + i
// of the product in register 4 b + i.  Two operands may agree on any order of
// k, so registers 8 s .. 8 s + 7 of a product, as bf16, are the operand whose
// k are its rows 16 s .. 16 s + 15: lane half h has k = 4 h .. + 3 and 8 + 4 h .. + 3
// of the 16, and the transposing reads below give the other operand in that
// order.
#pragma once

#include "kda_attn_tile.h"

namespace kda {

typedef float f32x16 __attribute__((ext_vector_type(16)));
typedef short s16x4 __attribute__((ext_vector_type(4)));

__device__ __forceinline__ f32x16 mfma32x32(bf16x8 a, bf16x8 b, f32x16 c) {
    return __builtin_amdgcn_mfma_f32_32x32x16_bf16(a, b, c, 0, 0, 0);
}

// Place of 16-byte unit u of a row in LDS is u ^ tile_swap(row): the 16 rows of
// one unit (operand rows, 16 lanes at a time) fall into 16 places of the banks'
// 256 bytes, and so do four neighbouring units of four rows (transposed reads,
// 32 lanes at a time).
template <int D>
__device__ __forceinline__ int tile_swap(int row) {
    return D == 128 ? ((row & 3) << 2) | ((row >> 2) & 3) : ((row & 2) << 1) | ((row >> 2) & 3);
}

#pragma clang diagnostic ignored "-Winline-asm"   // (m0 as a clobber)

// A pointer that every lane has, in scalar registers: the compiler may know
// that it is the same everywhere and still form it in vector registers, which
// the buffers of the loads below cannot be given in.
template <typename T>
__device__ __forceinline__ T* in_scalars(T* p) {
    uint32_t lo = (uint32_t)(uint64_t)p, hi = (uint32_t)((uint64_t)p >> 32);
    asm("" : "+v"(lo), "+v"(hi));
    lo = __builtin_amdgcn_readfirstlane(lo);
    hi = __builtin_amdgcn_readfirstlane(hi);
    asm volatile("" : "+s"(lo), "+s"(hi));
    return (T*)((uint64_t)hi << 32 | lo);
}

// Loads from a buffer to LDS, 16 bytes per lane, written out because the
// compiler would wait for them before every LDS read.  It counts no wait states
// in front of assembly either, and may form a buffer's words, or bring them
// back, with vector instructions at any place: so every block begins with the
// five that a load needs behind such a write (a move to m0 and s_nop 3), and
// within a block nothing can come between.  A load needs one behind m0's write.
#define KDA_LDS_FIRST "s_mov_b32 m0, %0\n\ts_nop 3\n\t"
#define KDA_LDS_NEXT "s_add_u32 m0, m0, 0x400\n\ts_nop 0\n\t"
#define KDA_LDS_LOAD(off, rs) "buffer_load_dwordx4 %" #off ", %" #rs ", 0 offen lds\n\t"
__device__ __forceinline__ void load_to_lds(__amdgpu_buffer_rsrc_t rs, uint32_t off, uint32_t to) {   // to `to` + 16 lane
    asm volatile(KDA_LDS_FIRST KDA_LDS_LOAD(1, 2) :: "s"(to), "v"(off), "s"(rs) : "memory", "m0");
}
// Load n to `to` + 1024 n + 16 lane.
template <int N>
__device__ __forceinline__ void load_to_lds(__amdgpu_buffer_rsrc_t rs, const uint32_t (&off)[N], uint32_t to) {
    static_assert(N == 2 || N == 4 || N == 8, "");
    if constexpr (N == 8) {
        asm volatile(KDA_LDS_FIRST KDA_LDS_LOAD(1, 9) KDA_LDS_NEXT KDA_LDS_LOAD(2, 9) KDA_LDS_NEXT KDA_LDS_LOAD(3, 9)
                     KDA_LDS_NEXT KDA_LDS_LOAD(4, 9) KDA_LDS_NEXT KDA_LDS_LOAD(5, 9) KDA_LDS_NEXT KDA_LDS_LOAD(6, 9)
                     KDA_LDS_NEXT KDA_LDS_LOAD(7, 9) KDA_LDS_NEXT KDA_LDS_LOAD(8, 9)
                     :: "s"(to), "v"(off[0]), "v"(off[1]), "v"(off[2]), "v"(off[3]), "v"(off[4]), "v"(off[5]), "v"(off[6]),
                        "v"(off[7]), "s"(rs) : "memory", "m0", "scc");
    } else if constexpr (N == 2) {
        asm volatile(KDA_LDS_FIRST KDA_LDS_LOAD(1, 3) KDA_LDS_NEXT KDA_LDS_LOAD(2, 3)
                     :: "s"(to), "v"(off[0]), "v"(off[1]), "s"(rs) : "memory", "m0", "scc");
    } else {
        asm volatile(KDA_LDS_FIRST KDA_LDS_LOAD(1, 5) KDA_LDS_NEXT KDA_LDS_LOAD(2, 5) KDA_LDS_NEXT KDA_LDS_LOAD(3, 5)
                     KDA_LDS_NEXT KDA_LDS_LOAD(4, 5)
                     :: "s"(to), "v"(off[0]), "v"(off[1]), "v"(off[2]), "v"(off[3]), "s"(rs) : "memory", "m0", "scc");
    }
}
// One load of each of two buffers, to `to` + 16 lane and `to` + `apart` + 16 lane.
__device__ __forceinline__ void load_pair_to_lds(__amdgpu_buffer_rsrc_t a, uint32_t aoff, __amdgpu_buffer_rsrc_t b, uint32_t boff,
                                                 uint32_t to, uint32_t apart) {
    asm volatile(KDA_LDS_FIRST KDA_LDS_LOAD(2, 4) "s_add_u32 m0, m0, %1\n\ts_nop 0\n\t" KDA_LDS_LOAD(3, 5)
                 :: "s"(to), "s"(apart), "v"(aoff), "v"(boff), "s"(a), "s"(b) : "memory", "m0", "scc");
}
// The same with 4 bytes per lane, the second load to `to` + 256 + 4 lane.
__device__ __forceinline__ void load4_pair_to_lds(__amdgpu_buffer_rsrc_t a, __amdgpu_buffer_rsrc_t b, uint32_t off, uint32_t to) {
    asm volatile(KDA_LDS_FIRST "buffer_load_dword %1, %2, 0 offen lds\n\t"
                 "s_add_u32 m0, m0, 0x100\n\ts_nop 0\n\tbuffer_load_dword %1, %3, 0 offen lds\n\t"
                 :: "s"(to), "v"(off), "s"(a), "s"(b) : "memory", "m0", "scc");
}
// All of this wave's loads to LDS have arrived and its LDS reads are done; then the workgroup's barrier.
__device__ __forceinline__ void tiles_barrier() {
    asm volatile("s_waitcnt vmcnt(0) lgkmcnt(0)\n\ts_barrier" ::: "memory");
}

// Keeps the compiler from holding what is formed from x in registers across a loop.
__device__ __forceinline__ void hide(int& x) { asm volatile("" : "+v"(x)); }

// Has x arrive here.  A register that a loop only reads is otherwise waited for
// in the loop, as if its load could still be under way, and with it for the
// loads to LDS that were requested since.
__device__ __forceinline__ void arrive(bf16x8& x) { asm volatile("" : "+v"(x)); }

// Where a lane reads its operands in a tile of rows of D values (byte offsets).
// k along the row: row l & 31 (+ 32 kt rows), values 16 s + 8 (l >> 5) .. + 7: at ^ 32 s.
template <int D>
__device__ __forceinline__ int lane_rows(int lane) {
    const int r = lane & 31;
    return r * 2 * D + (((lane >> 5) ^ tile_swap<D>(r)) * 16);
}
// k along the rows: column 32 c + (l & 31), rows 16 s + 4 (l >> 5) .. + 3 (x)
// and 8 more (y): at ^ 64 c, + 16 s rows.
template <int D>
__device__ __forceinline__ int2 lane_cols(int lane) {
    const int i = lane & 15, r = 4 * (lane >> 5) + (i >> 2), u = 2 * ((lane >> 4) & 1) + ((i & 3) >> 1);
    return make_int2(r * 2 * D + ((u ^ tile_swap<D>(r)) * 16) + 8 * (i & 1),
                     (r + 8) * 2 * D + ((u ^ tile_swap<D>(r + 8)) * 16) + 8 * (i & 1));
}
__device__ __forceinline__ bf16x8 read_rows(const char* tile, int at) { return *reinterpret_cast<const bf16x8*>(tile + at); }
__device__ __forceinline__ bf16x8 read_cols(const char* tile, int2 at, int c) {
    const s16x4 a = __builtin_amdgcn_ds_read_tr16_b64_v4i16((__attribute__((address_space(3))) s16x4*)(tile + (at.x ^ (64 * c))));
    const s16x4 b = __builtin_amdgcn_ds_read_tr16_b64_v4i16((__attribute__((address_space(3))) s16x4*)(tile + (at.y ^ (64 * c))));
    bf16x8 f;
    __builtin_memcpy(&f, &a, 8);
    __builtin_memcpy(reinterpret_cast<char*>(&f) + 8, &b, 8);
    return f;
}
// Registers 8 s .. of a product as an operand.
__device__ __forceinline__ bf16x8 as_operand(const f32x16& x, int s) {
    float w[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) w[e] = x[8 * s + e];
    return round8(w);
}
__device__ __forceinline__ f32x16 zero16() {
    f32x16 z;
#pragma unroll
    for (int e = 0; e < 16; ++e) z[e] = 0.f;
    return z;
}

// Token and head of the group that row x of `per` rows to a token is, x <
// 2^16: x / per = x * ceil(2^32 / per) >> 32.
struct RowOf {
    uint32_t per, inv;
    __device__ __forceinline__ explicit RowOf(int32_t hpg) : per((uint32_t)hpg), inv(hpg > 1 ? 0xffffffffu / (uint32_t)hpg + 1 : 0) {}
    __device__ __forceinline__ void of(uint32_t x, uint32_t& t, uint32_t& hh) const {
        t = per > 1 ? __umulhi(x, inv) : x;
        hh = x - t * per;
    }
};

}  // namespace kda
