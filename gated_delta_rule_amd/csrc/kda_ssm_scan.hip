// Selective state space scan over whole sequences (gfx950).  Formulas:
// include/kda_ssm.h.
//
// Chunk form, with g_t the sum of a over the chunk's tokens up to t and S the
// state at its start:
//   y_t  = e^{g_t} S^T C_t + sum_{s<=t} (C_t . B_s) e^{g_t - g_s} dt_s x_s + D x_t
//   S'   = e^{g_end} S + sum_s B_s (e^{g_end - g_s} dt_s x_s)^T
// Every exponent is <= 0, so nothing overflows however strong the decay.
//
// A workgroup of eight waves runs one chain of chunks for 128 columns of x:
// two heads of 64 of one group, which share the B and C tiles and the products
// C . B, or one head of 128.  A wave owns 16 columns and keeps its part of the
// state in accumulator registers in an order in which it is, without any move,
// also the operand of the next chunk's S^T C.  Per chunk: the next chunk's rows
// are requested, the waves share out the 16 x 16 tiles of C . B up to the
// diagonal and put them, weighted, into LDS while each also computes its
// S^T C; after one barrier each adds M x and D x (in float32: D is no operand
// of the matrix cores), stores y and updates its state.
//
// Chains: one per (sequence, head pair) where those fill the GPU; otherwise
// each sequence is cut into segments.  A first pass computes each segment's
// final state from zero (state products only, no scores), the merge turns
// them into incoming states (the transition of a segment is one number per
// head), and the full pass runs all segments side by side.
//
// Measured (MI355X, bf16, N 128): 8192 tokens of 64 heads of 64 in 16 segments
// 123 to 131 us (local 42, merge 13, outputs 81); 16 packed sequences of 8192
// tokens, 96 heads of 128, one pass, 222 to 229 us.  Neither HBM (28 and 124 us) nor the
// matrix cores (0.33 busy): per chunk the compute unit's two workgroups take
// 14 000 cycles, with vector instructions in 0.63 and LDS in 0.38 of them, and
// three barriers between dependent products.
#include "kda_ssm_tile.h"

namespace kda {

template <typename InT, int N, int P>
struct ScanCfg {
    static constexpr bool BF = sizeof(InT) == 2;
    static constexpr int L = BF ? 64 : 32;     // tokens per chunk (float32: three planes per tile)
    static constexpr int XP = BF ? 1 : 3;      // bf16 parts of an input
    static constexpr int MP = BF ? 1 : 3;      // ... of M (bf16: two do not fit in LDS beside a second workgroup)
    // ... of S in S^T C.  With one for bf16, y was 1.4 times as far from 64
    // bits as its own rounding where the state's share is large (1.07 with
    // two), for 119 against 123.5 us (8192 tokens of 64 heads) and 206 against
    // 222 us (16 packed sequences, 96 heads of 128).
    static constexpr int SP = BF ? 2 : 3;
    static constexpr int WP = 3;               // ... of w x in the state update (two: S_T off by up to 2e-6, a tenth faster)
    static constexpr int HPW = 128 / P;        // heads per workgroup
};
// Eight waves of 16 columns each.
constexpr int SC_WAVES = 8, SC_THREADS = 64 * SC_WAVES, SC_COLS = 128 / SC_WAVES, SC_CT = SC_COLS / 16;

// What a launch computes along its chains.
enum ScanMode {
    kOut = 0,      // y and the final states
    kLocal = 1,    // each segment's final state from zero, and its decay
    kWalk = 2,     // the state before every chunk
};
// Second direction (blockIdx.y = 1): from the sequence's end to its start, for
// the state gradient
//   dS' = e^{g_end} dS + sum_t C_t (e^{g_t} dy_t)^T
// (C takes B's place, dy takes x's).
template <typename InT, int N, int P, int MODE>
__global__ __launch_bounds__(SC_THREADS, 4) void ssm_scan_kernel(SsmScanDirs dirs, int32_t hblocks) {
    constexpr bool OUT = MODE == kOut;
    const bool rev = !OUT && blockIdx.y;
    const SsmScanParams& p = dirs.dir[OUT ? 0 : blockIdx.y];
    using Cfg = ScanCfg<InT, N, P>;
    constexpr int L = Cfg::L, XP = Cfg::XP, MP = Cfg::MP, SP = Cfg::SP, WP = Cfg::WP, HPW = Cfg::HPW;
    constexpr int TT = L / 16, NT = N / 16;
    constexpr int TILES = TT * (TT + 1) / 2;   // 16 x 16 tiles of M up to the diagonal
    __shared__ __attribute__((aligned(16))) __bf16 tB[XP * L * N];
    __shared__ __attribute__((aligned(16))) __bf16 tC[OUT ? XP * L * N : 8];
    __shared__ __attribute__((aligned(16))) __bf16 tX[XP * L * 128];
    __shared__ __attribute__((aligned(16))) __bf16 tM[OUT ? HPW * MP * L * L : 8];
    // decay sums of DB chunks at a time, one chunk and head per wave
    constexpr int DB = SC_WAVES / HPW;
    __shared__ ChunkDecay<L> dec[DB][HPW];

    const int tid = threadIdx.x;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    int lane = tid & 63;
    int rN = lane_row<N>(lane), rL = lane_row<L>(lane);
    int2 cB = lane_col<N, OUT ? 8 : 4>(lane), cX = lane_col<128, 4>(lane);
    // this lane's four columns of x in row l & 15 (as it holds y)
    int oX = 16 * ss_unit<16>(lane & 15, wave * (SC_COLS / 8) + (lane >> 5)) + 8 * (lane >> 4 & 1);
    const int64_t slot = blockIdx.x / (uint32_t)hblocks;
    const int hb = (int)(blockIdx.x - (uint32_t)slot * hblocks);
    const int hpg = p.H / p.G, bpg = (hpg + HPW - 1) / HPW;
    const int gw = hb / bpg, grp = p.g0 + gw;
    const int h0 = grp * hpg + (hb - gw * bpg) * HPW;
    const int64_t heads = (int64_t)p.gn * hpg;    // of the seg, seg_decay and states arrays
    const int hfirst = p.g0 * hpg;
    const int nh = (grp + 1) * hpg - h0 < HPW ? (grp + 1) * hpg - h0 : HPW;
    const int wh = wave * SC_COLS / P;                 // this wave's head of the workgroup's
    const bool live = wh < nh;
    const int h = h0 + (live ? wh : 0);
    const int pc = (wave * SC_COLS) % P;               // first column within the head
    SsmPiece s;
    if (p.cut) {
        s = ssm_piece(p.cu, p.rows, p.T, p.n_seqs, p.seg_len, slot);
        if (s.piece < 0) return;
        // nothing follows the last segment (the full pass gives its final state)
        if (MODE == kLocal && (rev ? s.r0 == s.start : s.r1 == s.end)) return;
    } else {
        const int64_t n = p.cu && p.n_seqs <= 64 ? ssm_longest(p.cu, p.rows, p.n_seqs, (int)slot) : slot;
        const SsmRange r = ssm_range(p.cu, p.rows, p.T, n);
        s = SsmPiece{n, 0, r.start, r.end, r.start, r.end};
    }

    // The state changes its sign with every chunk (minus before odd ones): the
    // matrix cores round their sums a little towards minus infinity (a
    // hundredth of a unit in the last place), which in a state of one sign adds
    // up, all elements alike, and in dA, a sum over all tokens, comes to 2e-6 of
    // it (0.7e-6 with the signs, the same time).  The factors of chunk_decay
    // carry them, loads and stores of the state put them on and take them off.
    const int len = (int)(s.r1 - s.r0), chunks = (len + L - 1) / L;
    auto sign_of = [](int chunk) { return chunk & 1 ? -1.f : 1.f; };
    const float sign0 = sign_of(rev ? chunks - 1 : 0), sign1 = sign_of(rev ? -1 : chunks);

    // State in accumulator registers.  With outputs: element (tile m = 2 j + o,
    // register r) is row 32 j + 8 lg + 4 o + r, column pc + 16 c + l15, the
    // order in which it is an operand of S^T C.  Without: row 16 m + l15,
    // columns pc + 16 c + 4 lg + r, the order in which a lane's four registers
    // are neighbours in memory.
    auto state_at = [&](int c, int m, int r) {
        const int l15 = lane & 15, lg = lane >> 4;
        return OUT ? (32 * (m >> 1) + 8 * lg + 4 * (m & 1) + r) * P + pc + 16 * c + l15
                   : (16 * m + l15) * P + pc + 16 * c + 4 * lg + r;
    };
    f32x4 S[SC_CT][NT];
    const int64_t seg_at = (slot * heads + h - hfirst) * (N * P), seq_at = (s.n * p.H + h) * (N * P);
    const float* init = MODE == kLocal ? nullptr : p.cut ? p.seg + seg_at : p.S0 ? p.S0 + seq_at : nullptr;
#pragma unroll
    for (int c = 0; c < SC_CT; ++c)
#pragma unroll
        for (int m = 0; m < NT; ++m)
#pragma unroll
            for (int r = 0; r < 4; ++r) S[c][m][r] = init ? sign0 * init[state_at(c, m, r)] : 0.f;
    auto save = [&](float* to) {
        if (!live) return;
#pragma unroll
        for (int c = 0; c < SC_CT; ++c)
#pragma unroll
            for (int m = 0; m < NT; ++m) {
                if constexpr (OUT) {
#pragma unroll
                    for (int r = 0; r < 4; ++r) to[state_at(c, m, r)] = sign1 * S[c][m][r];
                } else {
                    *reinterpret_cast<f32x4*>(to + state_at(c, m, 0)) = sign1 * S[c][m];
                }
            }
    };

    if constexpr (OUT) {   // tiles above the diagonal that a 32-token slab reaches
        for (int i = tid; i < HPW * MP * L * L / 8; i += SC_THREADS)
            reinterpret_cast<u32x4*>(tM)[i] = u32x4{0, 0, 0, 0};
    }

    // From here on all counts are of this chain's tokens, in 32 bits, and the
    // pointers run along the chain: scalar registers that spill cost vector
    // instructions (24 of them: 121 against 118 us).
    const int way = rev ? -L : L;
    const int at0 = rev && chunks > 0 ? (chunks - 1) * L : 0;   // token of the first chunk
    // requests for a chunk's rows, one chunk ahead
    Stager<InT, L, N, SC_THREADS> gB, gC;
    Stager<InT, L, 128, SC_THREADS> gX;
    const int xs = (int)p.x_stride, bs = (int)p.B_stride, cs = (int)p.C_stride;
    const InT* nx = (const InT*)p.x + (s.r0 + at0) * p.x_stride + (int64_t)h0 * P;
    const InT* nb = (const InT*)p.B + (s.r0 + at0) * p.B_stride + grp * N;
    const InT* nc = OUT ? (const InT*)p.C + (s.r0 + at0) * p.C_stride + grp * N : nullptr;
    auto rows_at = [&](int at) { return at < 0 || at >= len ? 0 : len - at < L ? len - at : L; };
    const int dh = wave % HPW, dk = wave / HPW;   // the head and, within a block, the chunk
    const bool dec_live = dh < nh;
    const float bias = p.dt_bias && dec_live ? p.dt_bias[h0 + dh] : 0.f;
    const float Ah = dec_live ? p.A[h0 + dh] : 0.f;
    float gdt = 0.f;
    const float* dts = p.dt + s.r0 * p.H + h0 + dh;
    const int H = p.H;
    auto dt_there = [&](int k, int& at) {   // this lane's token of the k-th chunk of the walk
        at = at0 + k * way + lane;
        return dec_live && k < chunks && lane < L && at < len;
    };
    auto fetch_dt = [&](int k) {
        int at;
        gdt = dt_there(k, at) ? dts[(int64_t)at * H] : 0.f;
    };
    const float D = OUT && p.D ? p.D[h] : 0.f;
    double total = 0.0;
    // this chain's first chunk among the slots of the states array
    const int64_t chunk0 = (p.cu ? s.start / L + s.n : s.n * ((p.T + L - 1) / L)) + (s.r0 - s.start) / L;
    float* walk = MODE == kWalk ? p.states + ((chunk0 + at0 / L) * heads + h - hfirst) * (N * P) : nullptr;
    char* yrow = OUT ? (char*)p.y + (((s.r0 + at0) * p.H + h) * P + pc) * (int64_t)sizeof(InT) : nullptr;
    {
        const int valid = rows_at(at0);   // (an empty sequence: no row)
        gX.load(nx, xs, valid, nh * P);
        gB.load(nb, bs, valid, N);
        if constexpr (OUT) gC.load(nc, cs, valid, N);
    }
    fetch_dt(dk);

    for (int i = 0, at = at0; i < chunks; ++i, at += way) {
        const int valid = rows_at(at), next = rows_at(at + way);
        hide(lane), hide(rN), hide(rL), hide(cB), hide(cX), hide(oX);
        const int l15 = lane & 15, lg = lane >> 4;
        gB.put(tB);
        if constexpr (OUT) gC.put(tC);
        gX.put(tX);
        if (i % DB == 0) {
            int token;
            const bool there = dt_there(i + dk, token);
            const float sign = sign_of(at0 / L + (rev ? -(i + dk) : i + dk));   // of the state before that chunk
            total += chunk_decay<L>(dec[dk][dh], gdt, there, bias, p.softplus, Ah, rev ? -sign : sign, -sign, -1.f);
            fetch_dt(i + DB + dk);
        }
        const ChunkDecay<L>* dc = dec[i % DB];
        lds_barrier();
        // the next chunk's rows, a tile at a time between the products: a
        // wave would stand at a burst of requests
        nx += (int64_t)way * xs;
        gX.load(nx, xs, next, nh * P);
        const ChunkDecay<L>& d = dc[wh];
        if constexpr (MODE == kWalk) {   // whole tiles, see walk_at
            if (live) {
                f32x4* to = reinterpret_cast<f32x4*>(walk);
                const float sign = sign_of(at / L);
#pragma unroll
                for (int c = 0; c < SC_CT; ++c)
#pragma unroll
                    for (int m = 0; m < NT; ++m) __builtin_nontemporal_store(S[c][m] * sign, &to[walk_at<N>(pc / 16 + c, m, lane)]);
            }
        }

        f32x4 Y[SC_CT][TT];
        if constexpr (OUT) {
            // M tiles: rows s (B), columns t (C) of the transposed product, so
            // that a lane holds four neighbouring s of one t
            auto tile_of = [&](int idx, int& tt, int& st) {
                tt = (idx >= 1) + (idx >= 3) + (idx >= 6);
                st = idx - tt * (tt + 1) / 2;
            };
            auto raw_tile = [&](int tt, int st) {
                f32x4 acc = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
                for (int ks = 0; ks < N / 32; ++ks) {
                    bf16x8 fb[XP], fc[XP];
#pragma unroll
                    for (int i = 0; i < XP; ++i) {
                        fb[i] = frag_row<N>(tB + i * L * N, 16 * st, ks, rN);
                        fc[i] = frag_row<N>(tC + i * L * N, 16 * tt, ks, rN);
                    }
                    acc = mma_parts<XP, XP>(fb, fc, acc);
                }
                return acc;
            };
            // (The fast exponential's own error, |e| 2^-24, is that of its
            // argument's rounding: with expf the errors against 64 bits are the
            // same to 2 %, and 4096 float32 tokens of 32 heads take 85 us, not 81.)
            auto weigh = [&](const f32x4& acc, int tt, int st, int hh) {
                const int t = 16 * tt + l15, s0 = 16 * st + 4 * lg;
                const ChunkDecay<L>& dm = dc[hh];
                const float ht = dm.gh[t], lt = dm.gl[t];
                const f32x4 hs = *reinterpret_cast<const f32x4*>(&dm.gh[s0]);
                const f32x4 ls = *reinterpret_cast<const f32x4*>(&dm.gl[s0]);
                const f32x4 ds = *reinterpret_cast<const f32x4*>(&dm.dt[s0]);
                float m[4];
#pragma unroll
                for (int r = 0; r < 4; ++r) m[r] = acc[r] * (__expf((ht - hs[r]) + (lt - ls[r])) * ds[r]);
                if (tt == st) {   // the diagonal tile: nothing above the diagonal
#pragma unroll
                    for (int r = 0; r < 4; ++r) m[r] = s0 + r <= t ? m[r] : 0.f;
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
            };
            // a tile for both heads per wave, then the rest one head at a time
            int tt, st;
            if (wave < TILES) {
                tile_of(wave, tt, st);
                const f32x4 acc = raw_tile(tt, st);
#pragma unroll
                for (int hh = 0; hh < HPW; ++hh) weigh(acc, tt, st, hh);
            }
            if constexpr (TILES > SC_WAVES) {
                if (wave < (TILES - SC_WAVES) * HPW) {
                    tile_of(SC_WAVES + wave / HPW, tt, st);
                    weigh(raw_tile(tt, st), tt, st, wave % HPW);
                }
            }
            nb += (int64_t)way * bs;
            gB.load(nb, bs, next, N);
            // Y^T = S^T C^T, rows p, columns t
#pragma unroll
            for (int c = 0; c < SC_CT; ++c)
#pragma unroll
                for (int tt = 0; tt < TT; ++tt) Y[c][tt] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
            for (int j = 0; j < N / 32; ++j) {
                bf16x8 fs[SC_CT][SP];
#pragma unroll
                for (int c = 0; c < SC_CT; ++c) {
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
                    for (int i = 0; i < XP; ++i) fc[i] = frag_row<N>(tC + i * L * N, 16 * tt, j, rN);
#pragma unroll
                    for (int c = 0; c < SC_CT; ++c) Y[c][tt] = mma_parts<SP, XP>(fs[c], fc, Y[c][tt]);
                }
            }
#pragma unroll
            for (int tt = 0; tt < TT; ++tt) {
                const float e = d.eg[16 * tt + l15];
#pragma unroll
                for (int c = 0; c < SC_CT; ++c) Y[c][tt] *= e;
            }
            lds_barrier();   // M is whole
        }

        if constexpr (OUT) {
            nc += (int64_t)way * cs;
            gC.load(nc, cs, next, N);
        } else {
            nb += (int64_t)way * bs;
            gB.load(nb, bs, next, N);
        }
        // x columns as operands: k runs over the tokens
        bf16x8 fx[SC_CT][L / 32][XP];
#pragma unroll
        for (int c = 0; c < SC_CT; ++c)
#pragma unroll
            for (int ks = 0; ks < L / 32; ++ks)
#pragma unroll
                for (int i = 0; i < XP; ++i)
                    fx[c][ks][i] = frag_col<128>(tX + i * L * 128, SC_COLS * wave + 16 * c, ks, cX);

        if constexpr (OUT) {
            const __bf16* M = tM + wh * MP * L * L;
#pragma unroll
            for (int tt = 0; tt < TT; ++tt)
#pragma unroll
                for (int ks = 0; ks <= tt / 2; ++ks) {
                    bf16x8 fm[MP];
#pragma unroll
                    for (int i = 0; i < MP; ++i) fm[i] = frag_row<L>(M + i * L * L, 16 * tt, ks, rL);
#pragma unroll
                    for (int c = 0; c < SC_CT; ++c) Y[c][tt] = mma_parts<XP, MP>(fx[c][ks], fm, Y[c][tt]);
                }
            // D x, and a lane stores four neighbouring columns of token 16 tt + l15
            static_assert(SC_CT == 1, "one column tile per wave");
#pragma unroll
            for (int tt = 0; tt < TT; ++tt) {
                const int t = 16 * tt + l15;
                float x[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
                for (int i = XP - 1; i >= 0; --i) {
                    const u32x2 u = *reinterpret_cast<const u32x2*>(reinterpret_cast<const char*>(tX + (i * L + 16 * tt) * 128) + oX);
#pragma unroll
                    for (int k = 0; k < 2; ++k) {
                        x[2 * k] += bf2_first(u[k]);
                        x[2 * k + 1] += bf2_second(u[k]);
                    }
                }
#pragma unroll
                for (int k = 0; k < 4; ++k) Y[0][tt][k] = fmaf(D, x[k], Y[0][tt][k]);
                if (live && t < valid) {
                    char* to = yrow + (uint32_t)(t * H * P + 4 * lg) * (uint32_t)sizeof(InT);
#pragma unroll
                    for (int c = 0; c < SC_CT; ++c) {
                        if constexpr (Cfg::BF) {
                            reinterpret_cast<u32x2*>(to)[4 * c] =
                                u32x2{pack_bf2(Y[c][tt][0], Y[c][tt][1]), pack_bf2(Y[c][tt][2], Y[c][tt][3])};
                        } else {
                            reinterpret_cast<f32x4*>(to)[4 * c] = Y[c][tt];
                        }
                    }
                }
            }
        }

        // State update, four row tiles at a time: each part of w x runs over
        // the four before the next part, so that no product waits for its own
        // result.
        const float eL = d.eL;
#pragma unroll
        for (int c = 0; c < SC_CT; ++c)
#pragma unroll
            for (int m = 0; m < NT; ++m) S[c][m] *= eL;
#pragma unroll
        for (int ks = 0; ks < L / 32; ++ks) {
            bf16x8 fw[SC_CT][WP];
#pragma unroll
            for (int c = 0; c < SC_CT; ++c) {
                float v[8];
                const f32x4* ws = reinterpret_cast<const f32x4*>(&(rev ? d.eg : d.w)[32 * ks + 8 * lg]);
                const f32x4 w0 = ws[0], w1 = ws[1];
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    float x = (float)fx[c][ks][XP - 1][e];
#pragma unroll
                    for (int i = XP - 2; i >= 0; --i) x += (float)fx[c][ks][i][e];
                    v[e] = x * (e < 4 ? w0[e & 3] : w1[e & 3]);
                }
                parts8<WP>(v, fw[c]);
            }
#pragma unroll
            for (int m0 = 0; m0 < NT; m0 += 4) {
                bf16x8 fb[4][XP];
#pragma unroll
                for (int m = 0; m < 4; ++m)
#pragma unroll
                    for (int i = 0; i < XP; ++i)
                        fb[m][i] = frag_col<N>(tB + i * L * N,
                                               OUT ? 32 * ((m0 + m) >> 1) + 4 * (m & 1) : 16 * (m0 + m), ks, cB);
#pragma unroll
                for (int c = 0; c < SC_CT; ++c)
#pragma unroll
                    for (int k = 2; k >= 0; --k)   // parts i + j = k, smallest first
#pragma unroll
                        for (int i = 0; i < XP; ++i) {
                            const int j = k - i;
                            if (j < 0 || j >= WP) continue;
#pragma unroll
                            for (int m = 0; m < 4; ++m)
                                S[c][m0 + m] = OUT ? mfma32(fb[m][i], fw[c][j], S[c][m0 + m])
                                                   : mfma32(fw[c][j], fb[m][i], S[c][m0 + m]);
                        }
            }
        }
        if constexpr (MODE == kWalk) walk += (rev ? -1 : 1) * heads * (N * P);
        if constexpr (OUT) yrow += (int64_t)L * H * P * (int64_t)sizeof(InT);
        lds_barrier();   // the tiles are consumed (rows and stores stay in flight)
    }

    if constexpr (MODE == kLocal) {
        save(p.seg + seg_at);
        __shared__ double sums[SC_WAVES];
        if (lane == 0) sums[wave] = total;
        __syncthreads();
        if (tid < nh) {
            double g = 0.0;
            for (int k = 0; k < DB; ++k) g += sums[k * HPW + tid];
            p.seg_decay[slot * heads + h0 - hfirst + tid] = expf((float)g);
        }
    } else {
        if (p.S_T && (rev ? s.r0 == s.start : s.r1 == s.end)) save(p.S_T + seq_at);
    }
}

// Incoming state of every segment from the segments' final states from zero,
// in place: S_0, then S_{j+1} = decay_j S_j + E_j (second direction: from the
// last segment to the first).  The E of the segment at the far end is not read.  Empty
// sequences have no segment: their final state is their initial one.
__global__ __launch_bounds__(SS_THREADS) void ssm_merge_kernel(SsmScanDirs dirs) {
    const bool rev = blockIdx.y;
    const SsmScanParams& p = dirs.dir[blockIdx.y];
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
    constexpr int AHEAD = 8;   // segments read together
    for (int64_t k0 = 0; k0 < segs; k0 += AHEAD) {
        f32x4 loc[AHEAD];
        float f[AHEAD];
#pragma unroll
        for (int i = 0; i < AHEAD; ++i) {
            const int64_t j = rev ? segs - 1 - (k0 + i) : k0 + i;
            const bool there = k0 + i + 1 < segs;
            loc[i] = there ? E[j * heads * np4] : f32x4{0.f, 0.f, 0.f, 0.f};
            f[i] = there ? dec[j * heads] : 0.f;
        }
#pragma unroll
        for (int i = 0; i < AHEAD; ++i) {
            if (k0 + i >= segs) break;
            const int64_t j = rev ? segs - 1 - (k0 + i) : k0 + i;
            E[j * heads * np4] = run;
            run = run * f[i] + loc[i];
        }
    }
}

// MODE kOut (one direction) or kWalk (both), with the passes before it where
// sequences are cut.  Both directions of the backward pass share their
// launches: neither waits for the other.
template <typename InT, int N, int P, int MODE>
static hipError_t run_scan(const SsmScanDirs& d, hipStream_t stream) {
    constexpr int HPW = 128 / P;
    const SsmScanParams& p = d.dir[0];
    const int hpg = p.H / p.G;
    const int32_t hblocks = p.gn * ((hpg + HPW - 1) / HPW);
    const unsigned dirs = MODE == kOut ? 1 : 2;
    const dim3 grid((unsigned)(p.slots * hblocks), dirs), block(SC_THREADS);
    if (p.cut) {
        hipLaunchKernelGGL((ssm_scan_kernel<InT, N, P, kLocal>), grid, block, 0, stream, d, hblocks);
        const int64_t n = (int64_t)p.n_seqs * p.gn * hpg * N * P / 4;
        hipLaunchKernelGGL(ssm_merge_kernel, dim3((unsigned)((n + SS_THREADS - 1) / SS_THREADS), dirs),
                           dim3(SS_THREADS), 0, stream, d);
    }
    hipLaunchKernelGGL((ssm_scan_kernel<InT, N, P, MODE>), grid, block, 0, stream, d, hblocks);
    return hipGetLastError();
}
template <typename InT, int MODE>
static hipError_t run_scan(const SsmScanDirs& d, hipStream_t stream) {
    if (d.dir[0].N == 128)
        return d.dir[0].P == 64 ? run_scan<InT, 128, 64, MODE>(d, stream) : run_scan<InT, 128, 128, MODE>(d, stream);
    return d.dir[0].P == 64 ? run_scan<InT, 64, 64, MODE>(d, stream) : run_scan<InT, 64, 128, MODE>(d, stream);
}
hipError_t launch_ssm_chunk_fwd(const SsmScanParams& p, bool bf16_in, hipStream_t stream) {
    const SsmScanDirs d{{p, SsmScanParams{}}};
    return bf16_in ? run_scan<__bf16, kOut>(d, stream) : run_scan<float, kOut>(d, stream);
}
hipError_t launch_ssm_walks(const SsmScanDirs& d, bool bf16_in, hipStream_t stream) {
    return bf16_in ? run_scan<__bf16, kWalk>(d, stream) : run_scan<float, kWalk>(d, stream);
}

}  // namespace kda
