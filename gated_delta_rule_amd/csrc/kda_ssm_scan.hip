// Selective state space scan over whole sequences (gfx950).  Formulas:
// include/kda_ssm.h.
//
// Chunk form, with g_t the sum of a over the chunk's tokens up to t and S the
// state at its start:
//   y_t  = e^{g_t} S^T C_t + sum_{s<=t} (C_t . B_s) e^{g_t - g_s} dt_s x_s + D x_t
//   S'   = e^{g_end} S + sum_s B_s (e^{g_end - g_s} dt_s x_s)^T
// Every exponent is <= 0, so nothing overflows however strong the decay.
//
// A workgroup runs one chain of chunks for 128 columns of x: two heads of 64
// of one group, which share the B and C tiles and the products C . B, or one
// head of 128.  A wave owns 32 columns and keeps its part of the state in
// accumulator registers in an order in which it is, without any move, also
// the operand of the next chunk's S^T C.  Per chunk: the next chunk's rows are
// requested, the four waves share out the 16 x 16 tiles of C . B below the
// diagonal and put them, weighted and with D on the diagonal, into LDS while
// each also computes its S^T C; after one barrier each adds M x, stores y and
// updates its state.
//
// Chains: one per (sequence, head pair) where those fill the GPU; otherwise
// each sequence is cut into segments.  A first pass computes each segment's
// final state from zero (state products only, no scores), the merge turns
// them into incoming states (the transition of a segment is one number per
// head), and the full pass runs all segments side by side.
#include "kda_ssm_tile.h"

namespace kda {

template <typename InT, int N, int P>
struct ScanCfg {
    static constexpr bool BF = sizeof(InT) == 2;
    static constexpr int L = BF ? 64 : 32;     // tokens per chunk (float32: three planes per tile)
    static constexpr int XP = BF ? 1 : 3;      // bf16 parts of an input
    static constexpr int MP = BF ? 1 : 3;      // ... of M
    static constexpr int SP = BF ? 1 : 3;      // ... of S in S^T C
    static constexpr int WP = 3;               // ... of w x in the state update
    static constexpr int HPW = 128 / P;        // heads per workgroup
};

// What a launch computes along its chains.
enum ScanMode {
    kOut = 0,      // y and the final states
    kLocal = 1,    // each segment's final state from zero, and its decay
    kWalk = 2,     // the state before every chunk
};
// REV: from the sequence's end to its start, for the state gradient
//   dS' = e^{g_end} dS + sum_t C_t (e^{g_t} dy_t)^T
// (C takes B's place, dy takes x's).
template <typename InT, int N, int P, int MODE, bool REV>
__global__ __launch_bounds__(SS_THREADS, 2) void ssm_scan_kernel(SsmScanParams p, int32_t hblocks) {
    constexpr bool OUT = MODE == kOut;
    static_assert(!(OUT && REV), "outputs run forward");
    using Cfg = ScanCfg<InT, N, P>;
    constexpr int L = Cfg::L, XP = Cfg::XP, MP = Cfg::MP, SP = Cfg::SP, WP = Cfg::WP, HPW = Cfg::HPW;
    constexpr int TT = L / 16, NT = N / 16;
    __shared__ __attribute__((aligned(16))) __bf16 tB[XP * L * N];
    __shared__ __attribute__((aligned(16))) __bf16 tC[OUT ? XP * L * N : 8];
    __shared__ __attribute__((aligned(16))) __bf16 tX[XP * L * 128];
    __shared__ __attribute__((aligned(16))) __bf16 tM[OUT ? HPW * MP * L * L : 8];
    __shared__ ChunkDecay<L> dec[HPW];

    const int tid = threadIdx.x, lane = tid & 63;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int l15 = lane & 15, lg = lane >> 4;
    const int64_t slot = blockIdx.x / (uint32_t)hblocks;
    const int hb = (int)(blockIdx.x - (uint32_t)slot * hblocks);
    const int hpg = p.H / p.G, bpg = (hpg + HPW - 1) / HPW;
    const int gw = hb / bpg, grp = p.g0 + gw;
    const int h0 = grp * hpg + (hb - gw * bpg) * HPW;
    const int64_t heads = (int64_t)p.gn * hpg;    // of the seg, seg_decay and states arrays
    const int hfirst = p.g0 * hpg;
    const int nh = (grp + 1) * hpg - h0 < HPW ? (grp + 1) * hpg - h0 : HPW;
    const int wh = wave * 32 / P;                 // this wave's head of the workgroup's
    const bool live = wh < nh;
    const int h = h0 + (live ? wh : 0);
    const int pc = (wave * 32) % P;               // first column within the head
    SsmPiece s;
    if (p.cut) {
        s = ssm_piece(p.cu, p.rows, p.T, p.n_seqs, p.seg_len, slot);
        if (s.piece < 0) return;
        // nothing follows the last segment (the full pass gives its final state)
        if (MODE == kLocal && (REV ? s.r0 == s.start : s.r1 == s.end)) return;
    } else {
        const SsmRange r = ssm_range(p.cu, p.rows, p.T, slot);
        s = SsmPiece{slot, 0, r.start, r.end, r.start, r.end};
    }

    // State in accumulator registers.  With outputs: element (tile m = 2 j + o,
    // register r) is row 32 j + 8 lg + 4 o + r, column pc + 16 c + l15, the
    // order in which it is an operand of S^T C.  Without: row 16 m + l15,
    // columns pc + 16 c + 4 lg + r, the order in which a lane's four registers
    // are neighbours in memory.
    auto state_at = [&](int c, int m, int r) {
        return OUT ? (32 * (m >> 1) + 8 * lg + 4 * (m & 1) + r) * P + pc + 16 * c + l15
                   : (16 * m + l15) * P + pc + 16 * c + 4 * lg + r;
    };
    f32x4 S[2][NT];
    const int64_t seg_at = (slot * heads + h - hfirst) * (N * P), seq_at = (s.n * p.H + h) * (N * P);
    const float* init = MODE == kLocal ? nullptr : p.cut ? p.seg + seg_at : p.S0 ? p.S0 + seq_at : nullptr;
#pragma unroll
    for (int c = 0; c < 2; ++c)
#pragma unroll
        for (int m = 0; m < NT; ++m)
#pragma unroll
            for (int r = 0; r < 4; ++r) S[c][m][r] = init ? init[state_at(c, m, r)] : 0.f;
    auto save = [&](float* to) {
        if (!live) return;
#pragma unroll
        for (int c = 0; c < 2; ++c)
#pragma unroll
            for (int m = 0; m < NT; ++m) {
                if constexpr (OUT) {
#pragma unroll
                    for (int r = 0; r < 4; ++r) to[state_at(c, m, r)] = S[c][m][r];
                } else {
                    *reinterpret_cast<f32x4*>(to + state_at(c, m, 0)) = S[c][m];
                }
            }
    };

    if constexpr (OUT) {   // tiles above the diagonal that a 32-token slab reaches
        for (int i = tid; i < HPW * MP * L * L / 8; i += SS_THREADS)
            reinterpret_cast<u32x4*>(tM)[i] = u32x4{0, 0, 0, 0};
    }

    // requests for a chunk's rows, one chunk ahead
    Stager<InT, L, N> gB, gC;
    Stager<InT, L, 128> gX;
    float gdt = 0.f;
    auto fetch = [&](int64_t row0) {
        const int valid = s.r1 - row0 < L ? (s.r1 > row0 ? (int)(s.r1 - row0) : 0) : L;
        const int64_t r = valid > 0 ? row0 : s.r0;
        gB.load((const InT*)p.B + r * p.B_stride + grp * N, p.B_stride, valid, N);
        if constexpr (OUT) gC.load((const InT*)p.C + r * p.C_stride + grp * N, p.C_stride, valid, N);
        gX.load((const InT*)p.x + r * p.x_stride + (int64_t)h0 * P, p.x_stride, valid, nh * P);
        if (wave < nh) gdt = lane < valid ? p.dt[(r + lane) * p.H + h0 + wave] : 0.f;
    };
    const float bias = p.dt_bias && wave < nh ? p.dt_bias[h0 + wave] : 0.f;
    const float Ah = wave < nh ? p.A[h0 + wave] : 0.f;
    double total = 0.0;
    const int64_t chunks = (s.r1 - s.r0 + L - 1) / L;
    // this chain's first chunk among the slots of the states array
    const int64_t chunk0 = (p.cu ? s.start / L + s.n : s.n * ((p.T + L - 1) / L)) + (s.r0 - s.start) / L;
    fetch(chunks == 0 ? s.r1 : REV ? s.r0 + (chunks - 1) * L : s.r0);   // (an empty sequence: no row)

    for (int64_t i = 0; i < chunks; ++i) {
        const int64_t ch = REV ? chunks - 1 - i : i;
        const int64_t row0 = s.r0 + ch * L;
        const int valid = s.r1 - row0 < L ? (int)(s.r1 - row0) : L;
        gB.put(tB);
        if constexpr (OUT) gC.put(tC);
        gX.put(tX);
        if (wave < HPW) total += chunk_decay<L>(dec[wave], gdt, wave < nh && lane < valid, bias, p.softplus, Ah);
        __syncthreads();
        fetch(REV ? (ch > 0 ? row0 - L : s.r1) : row0 + L);
        const ChunkDecay<L>& d = dec[wh];
        if constexpr (MODE == kWalk) save(p.states + ((chunk0 + ch) * heads + h - hfirst) * (N * P));

        f32x4 Y[2][TT];
        if constexpr (OUT) {
            // M tiles: rows s (B), columns t (C) of the transposed product, so
            // that a lane holds four neighbouring s of one t
#pragma unroll
            for (int k = 0; k < (TT * (TT + 1) / 2 + 3) / 4; ++k) {
                const int idx = wave + 4 * k;
                if (idx >= TT * (TT + 1) / 2) break;
                int tt = 0;
                while ((tt + 1) * (tt + 2) / 2 <= idx) ++tt;
                const int st = idx - tt * (tt + 1) / 2;
                f32x4 acc = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
                for (int ks = 0; ks < N / 32; ++ks) {
                    bf16x8 fb[XP], fc[XP];
#pragma unroll
                    for (int i = 0; i < XP; ++i) {
                        fb[i] = frag_row<N>(tB + i * L * N, 16 * st, ks);
                        fc[i] = frag_row<N>(tC + i * L * N, 16 * tt, ks);
                    }
                    acc = mma_parts<XP, XP>(fb, fc, acc);
                }
                const int t = 16 * tt + l15, s0 = 16 * st + 4 * lg;
#pragma unroll
                for (int hh = 0; hh < HPW; ++hh) {
                    const ChunkDecay<L>& dh = dec[hh];
                    const float ht = dh.gh[t], lt = dh.gl[t];
                    const f32x4 hs = *reinterpret_cast<const f32x4*>(&dh.gh[s0]);
                    const f32x4 ls = *reinterpret_cast<const f32x4*>(&dh.gl[s0]);
                    const f32x4 ds = *reinterpret_cast<const f32x4*>(&dh.dt[s0]);
                    const float Dh = p.D && hh < nh ? p.D[h0 + hh] : 0.f;
                    float m[4];
#pragma unroll
                    for (int r = 0; r < 4; ++r) {
                        m[r] = s0 + r <= t ? acc[r] * (__expf((ht - hs[r]) + (lt - ls[r])) * ds[r]) : 0.f;
                        if (s0 + r == t) m[r] += Dh;
                    }
                    __bf16* at = tM + hh * MP * L * L + 8 * ss_unit<L / 8>(t, s0 >> 3) + (s0 & 7);
#pragma unroll
                    for (int i = 0; i < MP; ++i) {
                        const u32x2 w = {pack_bf2(m[0], m[1]), pack_bf2(m[2], m[3])};
                        *reinterpret_cast<u32x2*>(at + i * L * L) = w;
                        if (i + 1 < MP) {
#pragma unroll
                            for (int r = 0; r < 2; ++r) {
                                m[2 * r] -= bf2_first(w[r]);
                                m[2 * r + 1] -= bf2_second(w[r]);
                            }
                        }
                    }
                }
            }
            // Y^T = S^T C^T, rows p, columns t
#pragma unroll
            for (int c = 0; c < 2; ++c)
#pragma unroll
                for (int tt = 0; tt < TT; ++tt) Y[c][tt] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
            for (int j = 0; j < N / 32; ++j) {
                bf16x8 fs[2][SP];
#pragma unroll
                for (int c = 0; c < 2; ++c) {
                    float v[8];
#pragma unroll
                    for (int r = 0; r < 4; ++r) {
                        v[r] = S[c][2 * j][r];
                        v[4 + r] = S[c][2 * j + 1][r];
                    }
                    parts8<SP>(v, fs[c]);
                }
#pragma unroll
                for (int tt = 0; tt < TT; ++tt) {
                    bf16x8 fc[XP];
#pragma unroll
                    for (int i = 0; i < XP; ++i) fc[i] = frag_row<N>(tC + i * L * N, 16 * tt, j);
#pragma unroll
                    for (int c = 0; c < 2; ++c) Y[c][tt] = mma_parts<SP, XP>(fs[c], fc, Y[c][tt]);
                }
            }
#pragma unroll
            for (int tt = 0; tt < TT; ++tt) {
                const float e = d.eg[16 * tt + l15];
#pragma unroll
                for (int c = 0; c < 2; ++c) Y[c][tt] *= e;
            }
            __syncthreads();   // M is whole
        }

        // x columns as operands: k runs over the tokens
        bf16x8 fx[2][L / 32][XP];
#pragma unroll
        for (int c = 0; c < 2; ++c)
#pragma unroll
            for (int ks = 0; ks < L / 32; ++ks)
#pragma unroll
                for (int i = 0; i < XP; ++i)
                    fx[c][ks][i] = frag_col<128, 4>(tX + i * L * 128, 32 * wave + 16 * c, ks);

        if constexpr (OUT) {
            const __bf16* M = tM + wh * MP * L * L;
#pragma unroll
            for (int tt = 0; tt < TT; ++tt)
#pragma unroll
                for (int ks = 0; ks <= tt / 2; ++ks) {
                    bf16x8 fm[MP];
#pragma unroll
                    for (int i = 0; i < MP; ++i) fm[i] = frag_row<L>(M + i * L * L, 16 * tt, ks);
#pragma unroll
                    for (int c = 0; c < 2; ++c) Y[c][tt] = mma_parts<XP, MP>(fx[c][ks], fm, Y[c][tt]);
                }
            // a lane stores four neighbouring columns of token 16 tt + l15
#pragma unroll
            for (int tt = 0; tt < TT; ++tt) {
                const int t = 16 * tt + l15;
                if (live && t < valid) {
                    const int64_t at = ((row0 + t) * p.H + h) * P + pc + 4 * lg;
#pragma unroll
                    for (int c = 0; c < 2; ++c) {
                        if constexpr (Cfg::BF) {
                            *reinterpret_cast<u32x2*>((__bf16*)p.y + at + 16 * c) =
                                u32x2{pack_bf2(Y[c][tt][0], Y[c][tt][1]), pack_bf2(Y[c][tt][2], Y[c][tt][3])};
                        } else {
                            *reinterpret_cast<f32x4*>((float*)p.y + at + 16 * c) = Y[c][tt];
                        }
                    }
                }
            }
        }

        // state update
        const float eL = d.eL;
#pragma unroll
        for (int c = 0; c < 2; ++c)
#pragma unroll
            for (int m = 0; m < NT; ++m) S[c][m] *= eL;
#pragma unroll
        for (int ks = 0; ks < L / 32; ++ks) {
            bf16x8 fw[2][WP];
#pragma unroll
            for (int c = 0; c < 2; ++c) {
                float v[8];
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    float x = (float)fx[c][ks][XP - 1][e];
#pragma unroll
                    for (int i = XP - 2; i >= 0; --i) x += (float)fx[c][ks][i][e];
                    v[e] = x * (REV ? d.eg : d.w)[32 * ks + 8 * lg + e];
                }
                parts8<WP>(v, fw[c]);
            }
#pragma unroll
            for (int j = 0; j < N / 32; ++j)
#pragma unroll
                for (int o = 0; o < 2; ++o) {
                    bf16x8 fb[XP];
#pragma unroll
                    for (int i = 0; i < XP; ++i)
                        fb[i] = OUT ? frag_col<N, 8>(tB + i * L * N, 32 * j + 4 * o, ks)
                                    : frag_col<N, 4>(tB + i * L * N, 32 * j + 16 * o, ks);
#pragma unroll
                    for (int c = 0; c < 2; ++c)
                        S[c][2 * j + o] = OUT ? mma_parts<XP, WP>(fb, fw[c], S[c][2 * j + o])
                                              : mma_parts<WP, XP>(fw[c], fb, S[c][2 * j + o]);
                }
        }
        __syncthreads();   // the tiles are consumed
    }

    if constexpr (MODE == kLocal) {
        save(p.seg + seg_at);
        if (wave < nh && lane == 0) p.seg_decay[slot * heads + h0 - hfirst + wave] = expf((float)total);
    } else {
        if (p.S_T && (REV ? s.r0 == s.start : s.r1 == s.end)) save(p.S_T + seq_at);
    }
}

// Incoming state of every segment from the segments' final states from zero,
// in place: S_0, then S_{j+1} = decay_j S_j + E_j (REV: from the last segment
// to the first).  The E of the segment at the far end is not read.  Empty
// sequences have no segment: their final state is their initial one.
template <bool REV>
__global__ __launch_bounds__(SS_THREADS) void ssm_merge_kernel(SsmScanParams p) {
    const int64_t np4 = (int64_t)p.N * p.P / 4, hpg = p.H / p.G, heads = p.gn * hpg;
    const int64_t i = (int64_t)blockIdx.x * SS_THREADS + threadIdx.x;
    if (i >= np4 * p.n_seqs * heads) return;
    const int64_t nhd = i / np4, e = i - nhd * np4;
    const int64_t n = nhd / heads, h = nhd - n * heads;
    const int64_t seq_at = (n * p.H + p.g0 * hpg + h) * np4 + e;
    const SsmRange r = ssm_range(p.cu, p.rows, p.T, n);
    const int64_t segs = (r.end - r.start + p.seg_len - 1) / p.seg_len;
    const int64_t base = p.cu ? r.start / p.seg_len + n : n * segs;
    f32x4 run = {0.f, 0.f, 0.f, 0.f};
    if (p.S0) run = reinterpret_cast<const f32x4*>(p.S0)[seq_at];
    if (segs == 0 && p.S_T) reinterpret_cast<f32x4*>(p.S_T)[seq_at] = run;
    f32x4* E = reinterpret_cast<f32x4*>(p.seg) + (base * heads + h) * np4 + e;
    const float* dec = p.seg_decay + base * heads + h;
    for (int64_t k = 0; k < segs; ++k) {
        const int64_t j = REV ? segs - 1 - k : k;
        f32x4 loc = {0.f, 0.f, 0.f, 0.f};
        float f = 0.f;
        if (k + 1 < segs) {
            loc = E[j * heads * np4];
            f = dec[j * heads];
        }
        E[j * heads * np4] = run;
        run = run * f + loc;
    }
}

// MODE kOut or kWalk, with the passes before it where sequences are cut.
template <typename InT, int N, int P, int MODE, bool REV>
static hipError_t run_scan(const SsmScanParams& p, hipStream_t stream) {
    constexpr int HPW = 128 / P;
    const int hpg = p.H / p.G;
    const int32_t hblocks = p.gn * ((hpg + HPW - 1) / HPW);
    const dim3 grid((unsigned)(p.slots * hblocks)), block(SS_THREADS);
    if (p.cut) {
        hipLaunchKernelGGL((ssm_scan_kernel<InT, N, P, kLocal, REV>), grid, block, 0, stream, p, hblocks);
        const int64_t n = (int64_t)p.n_seqs * p.gn * hpg * N * P / 4;
        hipLaunchKernelGGL((ssm_merge_kernel<REV>), dim3((unsigned)((n + SS_THREADS - 1) / SS_THREADS)), block, 0,
                           stream, p);
    }
    hipLaunchKernelGGL((ssm_scan_kernel<InT, N, P, MODE, REV>), grid, block, 0, stream, p, hblocks);
    return hipGetLastError();
}
template <typename InT, int MODE, bool REV>
static hipError_t run_scan(const SsmScanParams& p, hipStream_t stream) {
    if (p.N == 128)
        return p.P == 64 ? run_scan<InT, 128, 64, MODE, REV>(p, stream) : run_scan<InT, 128, 128, MODE, REV>(p, stream);
    return p.P == 64 ? run_scan<InT, 64, 64, MODE, REV>(p, stream) : run_scan<InT, 64, 128, MODE, REV>(p, stream);
}
hipError_t launch_ssm_chunk_fwd(const SsmScanParams& p, bool bf16_in, hipStream_t stream) {
    return bf16_in ? run_scan<__bf16, kOut, false>(p, stream) : run_scan<float, kOut, false>(p, stream);
}
hipError_t launch_ssm_walk(const SsmScanParams& p, bool bf16_in, bool reverse, hipStream_t stream) {
    if (reverse) return bf16_in ? run_scan<__bf16, kWalk, true>(p, stream) : run_scan<float, kWalk, true>(p, stream);
    return bf16_in ? run_scan<__bf16, kWalk, false>(p, stream) : run_scan<float, kWalk, false>(p, stream);
}

}  // namespace kda
