// Softmax attention with bf16 inputs, of whole sequences and of chunks of new
// tokens over a paged cache (gfx950).  Semantics: include/kda_attn.h.
//
// One pass over the keys with each row's running maximum m and sum l.  A
// workgroup has 128 rows of one (sequence, group), 32 per wave, and takes 64
// keys at a time: while one tile is computed with, the next one comes from
// memory straight into the other half of LDS (no registers in between).
//   S^T = K Q^T leaves lane l with row l & 31 and keys 8 b + 4 (l >> 5) + i: the
// place of P^T as an operand of O^T = V^T P^T, whose other operand the
// transposing LDS reads give for any order of keys.  So the weights stay in
// registers, and a row's maximum and sum are one lane's values and one
// exchange with lane l ^ 32.
//   m moves only when a row's maximum has grown by more than 2^8 over it: the
// weights are then up to 2^8 instead of 1, which costs no precision (l and o
// are float32, a bf16 weight has the same relative error), and the products
// with e^{m - m'} are left out of nearly all tiles.
#include "kda_attn_mma.h"

namespace kda {

constexpr int FW_THREADS = 256, FW_BLOCK = kAttnBlockBf16, FW_KEYS = 64;

template <int D, bool PAGED>
__global__ __launch_bounds__(FW_THREADS, 2) void attn_fwd_bf16_kernel(AttnParams p) {
    constexpr int ROWB = 2 * D, UNITS = D / 8, TILE = FW_KEYS * ROWB;   // bytes
    constexpr int LOADS = D / 32, RPL = 1024 / ROWB;                    // loads per wave and tile, rows of each
    constexpr int S = D / 16, O = D / 32;
    __shared__ __attribute__((aligned(1024))) char lds[4 * TILE];       // keys, keys, values, values
    __shared__ int32_t there[2][4];                                     // of each 16 keys: their page exists
    const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int col = lane & 31, half = lane >> 5;
    const AttnPlace pl = attn_place(blockIdx.x, p.slots * p.splits, p.G);
    const int64_t slot = p.slots - 1 - pl.item / p.splits;   // (later blocks see more keys)
    const int split = (int)(pl.item % p.splits);
    const AttnBlock b = attn_block(p, slot, p.hpg, FW_BLOCK);
    if (b.j < 0) return;
    const int32_t len = PAGED ? attn_length(p, b.n) : b.tokens;
    const int32_t first = len - b.tokens;                    // position of the first query token
    const int row = b.r0 + wave * 32 + col;
    const bool valid = row < b.r1;
    const int32_t most = p.causal ? first + (b.r1 - 1) / p.hpg + 1 : len;
    const int32_t t = valid ? row / p.hpg : (b.r1 - 1) / p.hpg;
    const int head = pl.g * p.hpg + (valid ? row - t * p.hpg : 0);
    const int32_t sees = p.causal ? first + t + 1 : len;     // keys [0, sees)
    const int32_t tiles = most > 0 ? (most + FW_KEYS - 1) / FW_KEYS : 0;
    const int32_t t0 = (int32_t)((int64_t)tiles * split / p.splits), t1 = (int32_t)((int64_t)tiles * (split + 1) / p.splits);
    // rows come in order of their tokens
    const int32_t sees_least = __builtin_amdgcn_readfirstlane(sees), sees_most = __builtin_amdgcn_readlane(sees, 31);

    // scores are scale * q . k with scale > 0: its sign goes to q
    const float scale = p.scale < 0.f ? -p.scale : p.scale > 0.f ? p.scale : 1.f;
    const uint32_t keep = p.scale == 0.f ? 0u : ~0u, flip = p.scale < 0.f ? 0x80008000u : 0u;
    bf16x8 q[S];
    const __bf16* qrow = (const __bf16*)p.q + (b.start + t) * p.q_stride + (int64_t)head * D + 8 * half;
#pragma unroll
    for (int s = 0; s < S; ++s) {
        u32x4 w = *reinterpret_cast<const u32x4*>(qrow + 16 * s);
#pragma unroll
        for (int i = 0; i < 4; ++i) w[i] = (w[i] & keep) ^ flip;
        q[s] = __builtin_bit_cast(bf16x8, w);
    }
#pragma unroll
    for (int s = 0; s < S; ++s) arrive(q[s]);
    const float c = scale * kLog2e;

    // this wave's 16 rows of each tile
    const AttnKeys<__bf16, PAGED> keys(p, b.n, b.start, pl.g);
    const int64_t kstep = PAGED ? D : keys.k_stride, vstep = PAGED ? D : keys.v_stride;
    uint32_t koff[LOADS], voff[LOADS];
#pragma unroll
    for (int i = 0; i < LOADS; ++i) {
        const int r = i * RPL + lane / UNITS, u = (lane % UNITS) ^ tile_swap<D>(r);
        koff[i] = (uint32_t)(r * (int)kstep * 2 + u * 16);
        voff[i] = (uint32_t)(r * (int)vstep * 2 + u * 16);
    }
    const uint32_t lds0 = (uint32_t)(uintptr_t)(__attribute__((address_space(3))) char*)lds;
    auto page_of = [&](int32_t tile) -> int32_t {
        if constexpr (PAGED) {
            const int32_t key = tile * FW_KEYS + 16 * wave;
            return key < most ? keys.pages[key >> keys.shift] : -1;
        }
        return 0;
    };
    int32_t page = t0 < t1 ? page_of(t0) : 0;   // of the next tile to be requested
    auto request = [&](int32_t tile, int buf) {
        const int32_t key = tile * FW_KEYS + 16 * wave;
        const int32_t left = most - key < 16 ? most - key : 16;
        const __bf16 *kb, *vb;
        bool ok = left > 0;
        if constexpr (PAGED) {
            ok = ok && page >= 0 && page < keys.n_pages;
            const int64_t at = (int64_t)page * keys.k_stride + (int64_t)(key & ((1 << keys.shift) - 1)) * D;
            kb = keys.k + (ok ? at : 0);
            vb = keys.v + (ok ? at : 0);
            if (lane == 0) there[buf][wave] = ok;
        } else {
            kb = keys.k + (ok ? (int64_t)key : 0) * kstep;
            vb = keys.v + (ok ? (int64_t)key : 0) * vstep;
        }
        const auto krs = make_rsrc(kb, ok ? ((left - 1) * (int)kstep + D) * 2 : 0);
        const auto vrs = make_rsrc(vb, ok ? ((left - 1) * (int)vstep + D) * 2 : 0);
        const uint32_t to = lds0 + buf * TILE + wave * 16 * ROWB;
#pragma unroll
        for (int i = 0; i < LOADS; ++i) load_to_lds(krs, koff[i], to + i * 1024);
#pragma unroll
        for (int i = 0; i < LOADS; ++i) load_to_lds(vrs, voff[i], to + 2 * TILE + i * 1024);
        if (PAGED && tile + 1 < t1) page = page_of(tile + 1);
    };

    // where this lane reads its operands
    const int kat = lane_rows<D>(lane);
    const int2 vat = lane_cols<D>(lane);

    f32x16 o[O];
#pragma unroll
    for (int i = 0; i < O; ++i) o[i] = zero16();
    float m = kAttnLowest, l = 0.f;

    if (t0 < t1) request(t0, 0);
    for (int32_t tile = t0; tile < t1; ++tile) {
        const int buf = (tile - t0) & 1;
        tiles_barrier();
        if (tile + 1 < t1) request(tile + 1, buf ^ 1);
        const int32_t key0 = tile * FW_KEYS;
        if (key0 >= sees_most) continue;
        const char* ks = lds + buf * TILE;
        const char* vs = lds + 2 * TILE + buf * TILE;
        f32x16 x[2];
#pragma unroll
        for (int kt = 0; kt < 2; ++kt) {
            x[kt] = zero16();
#pragma unroll
            for (int s = 0; s < S; ++s) x[kt] = mfma32x32(read_rows(ks + kt * 32 * ROWB, kat ^ (32 * s)), q[s], x[kt]);
        }
        bool whole = key0 + FW_KEYS <= sees_least;
        if constexpr (PAGED) whole = whole && (there[buf][0] & there[buf][1] & there[buf][2] & there[buf][3]);
        if (!__builtin_amdgcn_readfirstlane(whole)) {
#pragma unroll
            for (int kt = 0; kt < 2; ++kt)
#pragma unroll
                for (int e = 0; e < 16; ++e) {
                    const int key = 32 * kt + 8 * (e >> 2) + 4 * half + (e & 3);
                    const bool seen = key0 + key < sees && (!PAGED || there[buf][2 * kt + (e >> 3)]);
                    x[kt][e] = seen ? x[kt][e] : -INFINITY;
                }
        }
        float top = x[0][0];
#pragma unroll
        for (int e = 1; e < 16; ++e) top = fmaxf(top, x[0][e]);
#pragma unroll
        for (int e = 0; e < 16; ++e) top = fmaxf(top, x[1][e]);
        top = fmaxf(top, swap_halves(top));
        top = fmaxf(top * c, kAttnLowest);
        if (__any(top > m + 8.f)) {
            const float to = fmaxf(m, top), fade = attn_exp2(m - to);
            m = to;
            l *= fade;
#pragma unroll
            for (int i = 0; i < O; ++i)
#pragma unroll
                for (int e = 0; e < 16; ++e) o[i][e] *= fade;
        }
#pragma unroll
        for (int kt = 0; kt < 2; ++kt) {
            float sum[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
            for (int e = 0; e < 16; ++e) {
                x[kt][e] = attn_exp2(fmaf(x[kt][e], c, -m));
                sum[e & 3] += x[kt][e];
            }
            l += (sum[0] + sum[1]) + (sum[2] + sum[3]);
#pragma unroll
            for (int s = 0; s < 2; ++s) {
                const bf16x8 pw = as_operand(x[kt], s);
                const int at = (2 * kt + s) * 16 * ROWB;
#pragma unroll
                for (int i = 0; i < O; ++i)
                    o[i] = mfma32x32(read_cols(vs + at, vat, i), pw, o[i]);
            }
        }
    }
    l += swap_halves(l);
    if (!valid) return;
    if (p.splits > 1) {
        float* to = p.part + (((slot * p.G + pl.g) * p.splits + split) * FW_BLOCK + (row - b.r0)) * (D + 2);
#pragma unroll
        for (int i = 0; i < O; ++i)
#pragma unroll
            for (int e = 0; e < 16; ++e) to[32 * i + 8 * (e >> 2) + 4 * half + (e & 3)] = o[i][e];
        if (half == 0) {
            to[D] = l;
            to[D + 1] = l > 0.f ? m : -INFINITY;
        }
        return;
    }
    const float inv = l > 0.f ? 1.f / l : 0.f;
    __bf16* orow = (__bf16*)p.o + ((b.start + t) * p.H + head) * (int64_t)D;
#pragma unroll
    for (int i = 0; i < O; ++i)
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            const float y[4] = {o[i][4 * k] * inv, o[i][4 * k + 1] * inv, o[i][4 * k + 2] * inv, o[i][4 * k + 3] * inv};
            store4(orow + 32 * i + 8 * k + 4 * half, y);
        }
    if (p.lse && half == 0) p.lse[(b.start + t) * p.H + head] = l > 0.f ? (m + log2f(l)) * kLn2 : -INFINITY;
}

hipError_t launch_attn_fwd_bf16(const AttnParams& p, hipStream_t stream) {
    if (p.slots == 0) return hipSuccess;
    const dim3 grid((uint32_t)(p.slots * p.G * p.splits));
    if (p.lengths) {
        if (p.D == 64) attn_fwd_bf16_kernel<64, true><<<grid, FW_THREADS, 0, stream>>>(p);
        else attn_fwd_bf16_kernel<128, true><<<grid, FW_THREADS, 0, stream>>>(p);
    } else {
        if (p.D == 64) attn_fwd_bf16_kernel<64, false><<<grid, FW_THREADS, 0, stream>>>(p);
        else attn_fwd_bf16_kernel<128, false><<<grid, FW_THREADS, 0, stream>>>(p);
    }
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess || p.splits == 1) return e;
    return launch_attn_join(p, true, FW_BLOCK, stream);
}

}  // namespace kda
