// Backward pass of the state space scan (gfx950): the gradients of every
// chunk, given the state S at its start and the state gradient R at its end
// (both from the walks in kda_ssm_scan.hip).
//
// With g_t the decay sums within the chunk, L_ts = e^{g_t - g_s} (s <= t),
// G_ts = C_t . B_s, E_ts = dy_t . x_s:
//   dC_t  = e^{g_t} S dy_t + sum_s L_ts E_ts dt_s B_s
//   dB_s  = e^{g_end - g_s} dt_s R x_s + sum_t L_ts E_ts dt_s C_t
//   dx_s  = e^{g_end - g_s} dt_s R^T B_s + sum_t L_ts G_ts dt_s dy_t + D dy_s
// The decay's gradient needs no difference of large sums: a_t scales exactly
// the terms that reach across token t,
//   da_t  = sum_{s<t<=u} W_us + sum_{u>=t} U_u + sum_{s<t} V_s + Z
//   W_us  = L_us G_us E_us dt_s,  U_u = e^{g_u} C_u . S dy_u,
//   V_s   = e^{g_end - g_s} dt_s B_s . R x_s,  Z = e^{g_end} <S, R>,
// (the first sum from row and column sums of W's 16 x 16 tiles; differences
// of them only within a tile), and
//   ddt_s = sum_u W_us / dt_s + V_s / dt_s + A da_s,  dA = sum_t dt_t da_t,
//   dD    = sum_t E_tt,
// with the divisions left out of the sums in the first place.
//
// A workgroup runs one chunk for several heads of a group in turn: B, C and
// the tiles of G stay on chip, and dB and dC are summed over the heads in
// registers, so that only one partial sum per workgroup goes through memory.
// S and R come straight from memory into operand registers, each row once and
// one head ahead; R's bf16 rounding for dx goes through LDS.
//
// Measured (MI355X, 2 x 4096 tokens, 64 heads of 64, N 128, bf16): 195 us for
// 0.74 GB, 0.54 GB of them S and R.  Bound by issue: 12 700 cycles per chunk
// and head, half of them vector instructions, a third in the two products with
// S and R (their float32 operands are split into three bf16 parts), 1 100 in
// requests; matrix cores 0.18 busy.  What is the same for all heads stays in
// registers (212 us without).
#include "kda_ssm_tile.h"

#include <type_traits>

namespace kda {

__device__ __forceinline__ float sum_lane_groups(float v) {   // over lanes with equal l & 15
    auto r = __builtin_amdgcn_permlane16_swap(__float_as_uint(v), __float_as_uint(v), false, false);
    v += __uint_as_float((threadIdx.x & 16) ? r[0] : r[1]);
    return v + swap_halves(v);
}

// The same for RT values (two or four) at once: a lane gets the sum of value
// (l >> 4) % RT, so that each exchange halves the values along with the groups.
template <int RT>
__device__ __forceinline__ float sum_lane_groups(const float (&v)[RT]) {
    static_assert(RT == 2 || RT == 4, "");
    auto swap32 = [](float a, float b) {
        const auto r = __builtin_amdgcn_permlane32_swap(__float_as_uint(a), __float_as_uint(b), false, false);
        return __uint_as_float(r[0]) + __uint_as_float(r[1]);
    };
    auto swap16 = [](float a, float b) {
        const auto r = __builtin_amdgcn_permlane16_swap(__float_as_uint(a), __float_as_uint(b), false, false);
        return __uint_as_float(r[0]) + __uint_as_float(r[1]);
    };
    if constexpr (RT == 4) return swap16(swap32(v[0], v[2]), swap32(v[1], v[3]));
    const float a = swap16(v[0], v[1]);   // rows 0, 2: the first value, rows 1, 3: the second
    return a + swap_halves(a);
}

// Eight waves.  For the products with S, R and the chunk matrices towards dB
// and dC a wave owns one 16-row tile of the state (and, with N = 64, every
// second 16-token tile); towards dx one 16-column tile of x (with P = 64,
// every second token tile).
constexpr int SG_WAVES = 8, SG_THREADS = 64 * SG_WAVES;

template <typename InT, int N, int P>
__global__ __launch_bounds__(SG_THREADS, 2) void ssm_grad_kernel(SsmGradParams q) {
    constexpr bool BF = sizeof(InT) == 2;
    constexpr int L = BF ? 64 : 32;
    constexpr int XP = BF ? 1 : 3;      // bf16 parts of an input
    // ... of the chunk matrices, and of R in dx.  With one for bf16, dx, dB and
    // dC are 1.94e-3 off 64 bits where rounding them alone is 1.66e-3 (the
    // case above); a second plane of R does not fit in LDS.
    constexpr int KP = BF ? 1 : 3, RP = BF ? 1 : 3;
    constexpr int SP = 3;               // ... of S and R where U and V come from (float32 results)
    constexpr int TT = L / 16, OFFD = TT * (TT - 1) / 2;   // 16 x 16 tiles below the diagonal
    constexpr int OW = SG_WAVES - TT, TPW = (OFFD + OW - 1) / OW;      // the waves that own them, tiles per wave
    constexpr int RW = N / 16, RS = SG_WAVES / RW, RT = TT / RS;   // row tiles; waves per row tile; its token tiles per wave
    constexpr int CW = P / 16, CS = SG_WAVES / CW, CT = TT / CS;   // column tiles of x, likewise
    // Heads whose decay sums are computed together, one per wave, and whose
    // decay gradients are, as many as LDS holds the sums of: a wave at a time
    // would keep the others waiting (a wave per head: 227 against 220 us).
    constexpr int HB = P == 64 ? SG_WAVES : SG_WAVES / 2;
    __shared__ __attribute__((aligned(16))) __bf16 tB[XP * L * N], tC[XP * L * N];
    __shared__ __attribute__((aligned(16))) __bf16 tX[XP * L * P], tY[XP * L * P];
    __shared__ __attribute__((aligned(16))) __bf16 tK[KP * L * L], tM[KP * L * L];
    __shared__ ChunkDecay<L> decs[HB];
    // R in bf16, for its columns (float32: they come from memory, three planes being too large)
    __shared__ __attribute__((aligned(16))) __bf16 tR[BF ? N * P : 8];
    struct __attribute__((aligned(16))) Sums {
        float R[TT][L], Q[TT][L], U[RW][L], V[RW][L], W[L], E[L], Z[RW];
    };
    __shared__ Sums sums[HB];

    const SsmScanParams& p = q.f;
    const int tid = threadIdx.x;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    int lane = tid & 63;
    int rN = lane_row<N>(lane), rP = lane_row<P>(lane), rL = lane_row<L>(lane);
    int2 cN = lane_col<N, 4>(lane), cP = lane_col<P, 4>(lane), cL = lane_col<L, 4>(lane);
    // this lane's four columns of dy in row l & 15 (as it holds dx)
    int oY = 16 * ss_unit<P / 8>(lane & 15, wave % (P / 16) * 2 + (lane >> 5)) + 8 * (lane >> 4 & 1);
    const int rt = wave % RW, rh = wave / RW;      // this wave's row tile and its share of the token tiles
    const int ct = wave % CW, ch = wave / CW;      // ... column tile ...
    const int n0 = 16 * rt, p0 = 16 * ct;
    const int hpg = p.H / p.G;
    const int64_t heads = (int64_t)p.gn * hpg;
    const int per_slot = p.gn * q.blocks;
    const int64_t slot = blockIdx.x / (uint32_t)per_slot;
    const int rest = (int)(blockIdx.x - (uint32_t)slot * per_slot);
    const int gw = rest / q.blocks, blk = rest - gw * q.blocks;
    const int grp = p.g0 + gw;
    const int hw0 = gw * hpg + blk * q.heads_per_block;    // first head, among this launch's
    const int hwn = (gw + 1) * hpg - hw0 < q.heads_per_block ? (gw + 1) * hpg - hw0 : q.heads_per_block;
    const int hfirst = p.g0 * hpg;
    const SsmPiece s = ssm_piece(p.cu, p.rows, p.T, p.n_seqs, L, slot);
    if (s.piece < 0) {
        for (int i = tid; i < 3 * hwn; i += SG_THREADS) q.sums[(slot * heads + hw0) * 3 + i] = 0.f;
        return;
    }
    const int64_t row0 = s.r0;
    const int valid = (int)(s.r1 - s.r0);

    for (int i = tid; i < KP * L * L / 8; i += SG_THREADS) {
        reinterpret_cast<u32x4*>(tK)[i] = u32x4{0, 0, 0, 0};
        reinterpret_cast<u32x4*>(tM)[i] = u32x4{0, 0, 0, 0};
    }
    Stager<InT, L, P, SG_THREADS> gX, gY;
    auto fetch = [&](int hw) {
        const int64_t h = hfirst + hw;
        gX.load((const InT*)p.x + row0 * p.x_stride + h * P, p.x_stride, valid, P);
        gY.load((const InT*)q.gy + (row0 * p.H + h) * P, (int64_t)p.H * P, valid, P);
    };
    // this lane's raw dt of head hw0 + k
    auto raw_dt = [&](int k) {
        const int64_t h = hfirst + hw0 + k;
        return k < hwn && lane < valid ? p.dt[(row0 + lane) * p.H + h] + (p.dt_bias ? p.dt_bias[h] : 0.f) : 0.f;
    };
    {
        Stager<InT, L, N, SG_THREADS> g, c;
        g.load((const InT*)p.B + row0 * p.B_stride + grp * N, p.B_stride, valid, N);
        c.load((const InT*)p.C + row0 * p.C_stride + grp * N, p.C_stride, valid, N);
        g.put(tB);
        c.put(tC);
    }
    // this wave's rows of a head's S and R, one head ahead
    f32x4 fS[P / 32][2], fR[P / 32][2];
    auto fetch_state = [&](f32x4 (&f)[P / 32][2], const float* states, int hw) {
        const f32x4* S = reinterpret_cast<const f32x4*>(states + (slot * heads + hw) * (N * P));
        const int l15 = lane & 15, lg = lane >> 4;
#pragma unroll
        for (int ks = 0; ks < P / 32; ++ks)
#pragma unroll
            for (int k = 0; k < 2; ++k)   // columns 32 ks + 8 lg + 4 k .. + 3 of row n0 + l15
                f[ks][k] = S[walk_at<N>(2 * ks + (lg >> 1), rt, l15 + 16 * (2 * (lg & 1) + k))];
    };
    fetch(hw0);
    fetch_state(fS, q.states, hw0);
    fetch_state(fR, q.dstates, hw0);
    float raw = 0.f, raw_next = wave < HB ? raw_dt(wave) : 0.f;   // of the head that this wave ends
    __syncthreads();

    // tiles of G^T (rows s, columns t), kept for all heads
    f32x4 G[TPW];
    // (the first TT waves own one on the diagonal each, the others the rest)
    const bool on_diag = wave < TT;
    auto tile_of = [&](int k, int& tt, int& st) {
        int idx = wave - TT + OW * k;
        idx = idx < OFFD ? idx : OFFD - 1;
        tt = on_diag ? wave : 1 + (idx >= 1) + (idx >= 3);
        st = on_diag ? wave : idx - tt * (tt - 1) / 2;
    };
#pragma unroll
    for (int k = 0; k < TPW; ++k) {
        int tt, st;
        tile_of(k, tt, st);
        G[k] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int ks = 0; ks < N / 32; ++ks) {
            bf16x8 fb[XP], fc[XP];
#pragma unroll
            for (int i = 0; i < XP; ++i) {
                fb[i] = frag_row<N>(tB + i * L * N, 16 * st, ks, rN);
                fc[i] = frag_row<N>(tC + i * L * N, 16 * tt, ks, rN);
            }
            G[k] = mma_parts<XP, XP>(fb, fc, G[k]);
        }
    }
    // four neighbouring values of a tile's row, as floats
    auto four = [&](const __bf16* tile, int plane, int row, int c, float (&f)[4]) {
        const __bf16* at = tile + 8 * ss_unit<N / 8>(row, c >> 3) + (c & 7);
#pragma unroll
        for (int k = 0; k < 4; ++k) f[k] = 0.f;
#pragma unroll
        for (int i = XP - 1; i >= 0; --i) {
            const u32x2 u = *reinterpret_cast<const u32x2*>(at + i * plane);
            f[0] += bf2_first(u[0]);
            f[1] += bf2_second(u[0]);
            f[2] += bf2_first(u[1]);
            f[3] += bf2_second(u[1]);
        }
    };

    // this wave's rows of C and B by token, for the sums against them: the
    // same for all heads (with P = 128 there are no registers left for them)
    constexpr bool KEEP = P == 64;
    float ownC[RT][4], ownB[RT][4];
    auto own_rows = [&](const __bf16* tile, float (&o)[RT][4]) {
#pragma unroll
        for (int k = 0; k < RT; ++k) four(tile, L * N, 16 * (rh + RS * k) + (lane & 15), n0 + 4 * (lane >> 4), o[k]);
    };
    bf16x8 colB[L / 32][XP], colC[L / 32][XP];   // and its columns of them by 32 tokens
    auto own_cols = [&](int ks) {
#pragma unroll
        for (int i = 0; i < XP; ++i) {
            colB[ks][i] = frag_col<N>(tB + i * L * N, n0, ks, cN);
            colC[ks][i] = frag_col<N>(tC + i * L * N, n0, ks, cN);
        }
    };
    if constexpr (KEEP) {
        own_rows(tC, ownC);
        own_rows(tB, ownB);
#pragma unroll
        for (int ks = 0; ks < L / 32; ++ks) own_cols(ks);
    }

    // gradients of the decay and of dt of head hk0 + wave, whose sums are
    // whole: one token per lane
    auto finish = [&](int hk0) {
        if (wave >= HB || hk0 + wave >= hwn) return;
        const int hw = hw0 + hk0 + wave, h = hfirst + hw;
        const Sums& o = sums[wave];
        const ChunkDecay<L>& dec = decs[wave];
        const int t = lane < L ? lane : L - 1;
        const bool on = lane < valid;
        const float A = p.A[h];
        // W across token t: tiles (u's tile a, s's tile b) around t's tile k.
        // Whole tiles and whole rows or columns of them only add up; just
        // within the tile on the diagonal do row and column sums cancel.
        const float dt = dec.dt[t];
        const int k = t / 16;
        float Q = 0.f, rows = 0.f, cols = 0.f;
        double whole = 0.0;
#pragma unroll
        for (int b = 0; b < TT; ++b) {
            const float r = o.R[b][t], c = o.Q[b][t];
            if (b < k) rows += r;         // (a = k, b < k)
            if (b > k) cols += c;         // (a = b > k, b = k)
            if (b >= k) Q += c;
        }
#pragma unroll
        for (int j = 1; j + 1 < TT; ++j) {   // tiles a > j, b < j
            float r = 0.f;
#pragma unroll
            for (int b = 0; b < j; ++b) r += o.R[b][t];
            const double all = wave_last_f64(wave_scan_f64(lane < L && k > j ? (double)r : 0.0));
            if (k == j) whole = all;
        }
        const double diag = (double)o.R[k][t] - (double)(o.Q[k][t] * dt);
        const double own = lane < L ? (double)(cols * dt) : 0.0;
        const double X = whole + row_suffix_f64(lane < L ? (double)rows + diag : 0.0) + (row_prefix_f64(own) - own);
        float U = 0.f, V = 0.f, Z = 0.f;
#pragma unroll
        for (int j = 0; j < RW; ++j) {
            U += o.U[j][t];
            V += o.V[j][t];
            Z += o.Z[j];
        }
        U *= dec.eg[t];
        V *= expf((dec.gh[L - 1] - dec.gh[t]) + (dec.gl[L - 1] - dec.gl[t]));   // without dt
        Z *= dec.eL;
        // U of this token and the later ones, V of the earlier ones
        const double x = lane < L ? (double)U : 0.0, y = lane < L ? (double)(V * dt) : 0.0;
        const double sx = wave_scan_f64(x), sy = wave_scan_f64(y);
        const double across = X + (wave_last_f64(sx) - sx + x) + (sy - y) + (double)Z;   // (by all lanes)
        // (rounding's remainder of the sums times a large dt is no gradient of A)
        const float da = dt * A < kDecayEnds ? 0.f : (float)across;
        float ddt = (Q + o.W[t]) + V + A * da;
        if (p.softplus) ddt *= 1.f / (1.f + expf(-raw));
        if (on) q.gdt[(row0 + lane) * p.H + h] = ddt;
        const float a = wave_sum_dpp(on ? dt * da : 0.f);
        const float d = wave_sum_dpp(on ? o.E[t] : 0.f);
        const float b = wave_sum_dpp(on ? ddt : 0.f);
        if (lane == 0) {
            float* to = q.sums + (slot * heads + hw) * 3;
            to[0] = a;
            to[1] = d;
            to[2] = b;
        }
    };

    f32x4 dB[RT], dC[RT];   // rows n, columns token, of all heads so far
#pragma unroll
    for (int k = 0; k < RT; ++k) dB[k] = dC[k] = f32x4{0.f, 0.f, 0.f, 0.f};

    for (int hk = 0; hk < hwn; ++hk) {
        const int hw = hw0 + hk, h = hfirst + hw;
        hide(lane), hide(rN), hide(rP), hide(rL), hide(cN), hide(cP), hide(cL), hide(oY);
        const int l15 = lane & 15, lg = lane >> 4;
        const float* R = q.dstates + (slot * heads + hw) * (N * P);
        const float D = p.D ? p.D[h] : 0.f;
        gX.put(tX);
        gY.put(tY);
        if (hk % HB == 0) {
            if (hk > 0) finish(hk - HB);
            if (wave < HB) {
                const int k = hk + wave;
                const float a = k < hwn ? p.A[hfirst + hw0 + k] : 0.f;
                raw = raw_next;
                chunk_decay<L>(decs[wave], raw, k < hwn && lane < valid, 0.f, p.softplus, a);
                raw_next = raw_dt(k + HB);
            }
        }
        const ChunkDecay<L>& dec = decs[hk % HB];
        Sums& now = sums[hk % HB];
        lds_barrier();
        // R by columns, for dx (float32): out of cache, its rows having come for fR
        float fRc[BF ? 1 : N / 32][8];
        if constexpr (!BF) {
#pragma unroll
            for (int ks = 0; ks < N / 32; ++ks)
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    const int n = 32 * ks + 8 * lg + e;
                    fRc[ks][e] = R[4 * walk_at<N>(ct, n >> 4, (n & 15) + 16 * (l15 >> 2)) + (l15 & 3)];
                }
            __builtin_amdgcn_sched_barrier(0);
        }
        // chunk matrices, a lane holding four neighbouring s of one t
        auto scores = [&](int k) {
            int tt, st;
            tile_of(k, tt, st);
            f32x4 E = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
            for (int ks = 0; ks < P / 32; ++ks) {
                bf16x8 fx[XP], fy[XP];
#pragma unroll
                for (int i = 0; i < XP; ++i) {
                    fx[i] = frag_row<P>(tX + i * L * P, 16 * st, ks, rP);
                    fy[i] = frag_row<P>(tY + i * L * P, 16 * tt, ks, rP);
                }
                E = mma_parts<XP, XP>(fx, fy, E);
            }
            return E;
        };
        auto weigh = [&](const f32x4& E, int k, auto diag) {
            int tt, st;
            tile_of(k, tt, st);
            const int t = 16 * tt + l15, s0 = 16 * st + 4 * lg;
            const float ht = dec.gh[t], lt = dec.gl[t];
            const f32x4 hs = *reinterpret_cast<const f32x4*>(&dec.gh[s0]);
            const f32x4 ls = *reinterpret_cast<const f32x4*>(&dec.gl[s0]);
            const f32x4 ds = *reinterpret_cast<const f32x4*>(&dec.dt[s0]);
            float K[4], M[4], row = 0.f, col[4];
#pragma unroll
            for (int r = 0; r < 4; ++r) {
                if constexpr (!diag) {
                    const float l = __expf((ht - hs[r]) + (lt - ls[r]));
                    K[r] = E[r] * l * ds[r];
                    M[r] = G[k][r] * l * ds[r];
                    col[r] = G[k][r] * l * E[r];
                    row = fmaf(col[r], ds[r], row);
                } else {   // nothing above the diagonal, and W's diagonal apart
                    const int sr = s0 + r;
                    const float l = sr <= t ? __expf((ht - hs[r]) + (lt - ls[r])) : 0.f;
                    K[r] = sr <= t ? E[r] * l * ds[r] : 0.f;
                    M[r] = sr <= t ? G[k][r] * l * ds[r] : 0.f;
                    const float w = sr <= t ? G[k][r] * l * E[r] : 0.f;
                    col[r] = sr < t ? w : 0.f;
                    row = fmaf(col[r], ds[r], row);
                    if (sr == t) {
                        now.W[t] = w;
                        now.E[t] = E[r];
                    }
                }
            }
            row = sum_lane_groups(row);
            if (lg == 0) now.R[st][t] = row;
#pragma unroll
            for (int r = 0; r < 4; ++r) {
                col[r] += dpp_mov<0xB1>(col[r]);
                col[r] += dpp_mov<0x4E>(col[r]);
                col[r] += dpp_mov<0x124>(col[r]);
                col[r] += dpp_mov<0x128>(col[r]);
            }
            if (l15 == 0) *reinterpret_cast<f32x4*>(&now.Q[tt][s0]) = f32x4{col[0], col[1], col[2], col[3]};
            const int at = 8 * ss_unit<L / 8>(t, s0 >> 3) + (s0 & 7);
#pragma unroll
            for (int i = 0; i < KP; ++i) {
                const u32x2 uk = {pack_bf2(K[0], K[1]), pack_bf2(K[2], K[3])};
                const u32x2 um = {pack_bf2(M[0], M[1]), pack_bf2(M[2], M[3])};
                *reinterpret_cast<u32x2*>(tK + i * L * L + at) = uk;
                *reinterpret_cast<u32x2*>(tM + i * L * L + at) = um;
                if (i + 1 < KP) {
#pragma unroll
                    for (int r = 0; r < 2; ++r) {
                        K[2 * r] -= bf2_first(uk[r]);
                        K[2 * r + 1] -= bf2_second(uk[r]);
                        M[2 * r] -= bf2_first(um[r]);
                        M[2 * r + 1] -= bf2_second(um[r]);
                    }
                }
            }
        };
        if (on_diag) {
            weigh(scores(0), 0, std::true_type{});
        } else if (TPW > 1 && wave - TT + OW < OFFD) {
            const f32x4 E0 = scores(0), E1 = scores(TPW - 1);
            weigh(E0, 0, std::false_type{});
            weigh(E1, TPW - 1, std::false_type{});
        } else if (wave - TT < OFFD) {
            weigh(scores(0), 0, std::false_type{});
        }

        // products with S and R: rows n0 .., columns token (tile rh + RS k)
        __builtin_amdgcn_sched_barrier(0);
        {
            float z = 0.f;
#pragma unroll
            for (int ks = 0; ks < P / 32; ++ks)
#pragma unroll
                for (int k = 0; k < 2; ++k)
#pragma unroll
                    for (int e = 0; e < 4; ++e) z = fmaf(fS[ks][k][e], fR[ks][k][e], z);
            z = wave_sum_dpp(z);
            if (lane == 0 && rh == 0) now.Z[rt] = z;
        }
        if constexpr (BF) {
            if (rh == 0) {
#pragma unroll
                for (int ks = 0; ks < P / 32; ++ks) {
                    u32x4 u;
#pragma unroll
                    for (int k = 0; k < 2; ++k) {
                        u[2 * k] = pack_bf2(fR[ks][k][0], fR[ks][k][1]);
                        u[2 * k + 1] = pack_bf2(fR[ks][k][2], fR[ks][k][3]);
                    }
                    *reinterpret_cast<u32x4*>(tR + 8 * ss_unit<P / 8>(n0 + l15, 4 * ks + lg)) = u;
                }
            }
        }
        // first S with dy, then R with x: acc, its sum against C or B by token, and its share of dC or dB
        auto with_state = [&](const f32x4 (&f)[P / 32][2], const __bf16* tok, const float (&own)[RT][4], const float* weight,
                              float* sums, f32x4 (&grad)[RT]) {
            f32x4 acc[RT];
#pragma unroll
            for (int k = 0; k < RT; ++k) acc[k] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
            for (int ks = 0; ks < P / 32; ++ks) {
                float v[8];
#pragma unroll
                for (int e = 0; e < 8; ++e) v[e] = f[ks][e / 4][e % 4];
                bf16x8 ps[SP];
                parts8<SP>(v, ps);
#pragma unroll
                for (int k = 0; k < RT; ++k) {
                    bf16x8 ft[XP];
#pragma unroll
                    for (int i = 0; i < XP; ++i) ft[i] = frag_row<P>(tok + i * L * P, 16 * (rh + RS * k), ks, rP);
                    acc[k] = mma_parts<SP, XP>(ps, ft, acc[k]);
                }
            }
            float u[RT];
#pragma unroll
            for (int k = 0; k < RT; ++k) {
                const int t = 16 * (rh + RS * k) + l15;
                const float w = weight[t];
                u[k] = 0.f;
#pragma unroll
                for (int r = 0; r < 4; ++r) {
                    u[k] = fmaf(own[k][r], acc[k][r], u[k]);
                    grad[k][r] = fmaf(w, acc[k][r], grad[k][r]);
                }
            }
            if constexpr (RT == 1) {
                const float v = sum_lane_groups(u[0]);
                if (lg == 0) sums[16 * rh + l15] = v;
            } else {
                const float v = sum_lane_groups<RT>(u);
                if (lg < RT) sums[16 * (rh + RS * lg) + l15] = v;
            }
        };
        if constexpr (!KEEP) own_rows(tC, ownC);
        with_state(fS, tY, ownC, dec.eg, now.U[rt], dC);
        // (the next head's requests apart: a wave would stand at a burst)
        __builtin_amdgcn_sched_barrier(0);
        if (hk + 1 < hwn) fetch_state(fS, q.states, hw + 1);
        __builtin_amdgcn_sched_barrier(0);
        if constexpr (!KEEP) own_rows(tB, ownB);
        with_state(fR, tX, ownB, dec.w, now.V[rt], dB);
        __builtin_amdgcn_sched_barrier(0);
        if (hk + 1 < hwn) fetch_state(fR, q.dstates, hw + 1);
        lds_barrier();   // the chunk matrices and the partial sums are whole
        if (hk + 1 < hwn) fetch(hw + 1);

        // products with the chunk matrices
#pragma unroll
        for (int ks = 0; ks < L / 32; ++ks) {
            if constexpr (!KEEP) own_cols(ks);
            const auto &fb = colB[ks], &fc = colC[ks];
#pragma unroll
            for (int k = 0; k < RT; ++k) {
                const int t = rh + RS * k;
                constexpr bool even = RS == 2;
                const int last = even ? k : k / 2;   // = t / 2, the slab with the diagonal
                if (ks <= last) {
                    bf16x8 fk[KP];
#pragma unroll
                    for (int i = 0; i < KP; ++i) fk[i] = frag_row<L>(tK + i * L * L, 16 * t, ks, rL);
                    dC[k] = mma_parts<XP, KP>(fb, fk, dC[k]);
                }
                if (ks >= last) {
                    bf16x8 fk[KP];
#pragma unroll
                    for (int i = 0; i < KP; ++i) fk[i] = frag_col<L>(tK + i * L * L, 16 * t, ks, cL);
                    dB[k] = mma_parts<XP, KP>(fc, fk, dB[k]);
                }
            }
        }
        __builtin_amdgcn_sched_barrier(0);
        {
            f32x4 dX[CT];
#pragma unroll
            for (int k = 0; k < CT; ++k) dX[k] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
            for (int ks = 0; ks < N / 32; ++ks) {
                bf16x8 pR[RP];
                if constexpr (BF) pR[0] = frag_col<P>(tR, p0, ks, cP);
                else parts8<RP>(fRc[ks], pR);
#pragma unroll
                for (int k = 0; k < CT; ++k) {
                    bf16x8 fb[XP];
#pragma unroll
                    for (int i = 0; i < XP; ++i) fb[i] = frag_row<N>(tB + i * L * N, 16 * (ch + CS * k), ks, rN);
                    dX[k] = mma_parts<RP, XP>(pR, fb, dX[k]);
                }
            }
#pragma unroll
            for (int k = 0; k < CT; ++k) dX[k] *= dec.w[16 * (ch + CS * k) + l15];
#pragma unroll
            for (int ks = 0; ks < L / 32; ++ks) {
                bf16x8 fy[XP];
#pragma unroll
                for (int i = 0; i < XP; ++i) fy[i] = frag_col<P>(tY + i * L * P, p0, ks, cP);
#pragma unroll
                for (int k = 0; k < CT; ++k) {
                    if (ks < (CS == 2 ? k : k / 2)) continue;
                    bf16x8 fm[KP];
#pragma unroll
                    for (int i = 0; i < KP; ++i) fm[i] = frag_col<L>(tM + i * L * L, 16 * (ch + CS * k), ks, cL);
                    dX[k] = mma_parts<XP, KP>(fy, fm, dX[k]);
                }
            }
#pragma unroll
            for (int k = 0; k < CT; ++k) {
                const int row = 16 * (ch + CS * k) + l15;
                float y[4] = {0.f, 0.f, 0.f, 0.f};   // D dy, in float32
#pragma unroll
                for (int i = XP - 1; i >= 0; --i) {
                    const u32x2 u = *reinterpret_cast<const u32x2*>(
                        reinterpret_cast<const char*>(tY + (i * L + 16 * (ch + CS * k)) * P) + oY);
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        y[2 * e] += bf2_first(u[e]);
                        y[2 * e + 1] += bf2_second(u[e]);
                    }
                }
#pragma unroll
                for (int e = 0; e < 4; ++e) dX[k][e] = fmaf(D, y[e], dX[k][e]);
                if (row < valid) {
                    const int64_t at = (row0 + row) * q.gx_stride + (int64_t)h * P + p0 + 4 * lg;
                    if constexpr (BF)
                        *reinterpret_cast<u32x2*>((__bf16*)q.gx + at) =
                            u32x2{pack_bf2(dX[k][0], dX[k][1]), pack_bf2(dX[k][2], dX[k][3])};
                    else
                        *reinterpret_cast<f32x4*>((float*)q.gx + at) = dX[k];
                }
            }
        }

        lds_barrier();   // the tiles are consumed (rows and stores stay in flight)
    }

    finish((hwn - 1) / HB * HB);

    // dB and dC of these heads: the gradients themselves, or a partial sum
    const int l15 = lane & 15, lg = lane >> 4;
#pragma unroll
    for (int k = 0; k < RT; ++k) {
        const int row = 16 * (rh + RS * k) + l15, n = n0 + 4 * lg;
        if (row >= valid) continue;
        if (q.blocks == 1) {
            const int64_t b = (row0 + row) * q.gB_stride + grp * N + n, c = (row0 + row) * q.gC_stride + grp * N + n;
            if constexpr (BF) {
                *reinterpret_cast<u32x2*>((__bf16*)q.gB + b) =
                    u32x2{pack_bf2(dB[k][0], dB[k][1]), pack_bf2(dB[k][2], dB[k][3])};
                *reinterpret_cast<u32x2*>((__bf16*)q.gC + c) =
                    u32x2{pack_bf2(dC[k][0], dC[k][1]), pack_bf2(dC[k][2], dC[k][3])};
            } else {
                *reinterpret_cast<f32x4*>((float*)q.gB + b) = dB[k];
                *reinterpret_cast<f32x4*>((float*)q.gC + c) = dC[k];
            }
        } else {
            const int64_t at = (((int64_t)blk * p.gn + gw) * p.rows + row0 + row) * N + n;
            *reinterpret_cast<f32x4*>(q.part + at) = dB[k];
            *reinterpret_cast<f32x4*>(q.part + (int64_t)q.blocks * p.gn * p.rows * N + at) = dC[k];
        }
    }
}

// Adds up the head blocks' partial sums of dB and dC, four channels per lane.
template <typename InT>
__device__ __forceinline__ void ssm_grad_bc(const SsmGradParams& q) {
    const SsmScanParams& p = q.f;
    const int64_t n4 = p.N / 4, per = (int64_t)p.gn * p.rows * n4;   // pieces of one block's array
    const int64_t i = (int64_t)blockIdx.x * SS_THREADS + threadIdx.x;
    if (i >= 2 * per) return;
    const int which = i >= per;
    const int64_t e = i - which * per;
    const int64_t n = e % n4, gr = e / n4, row = gr % p.rows, gw = gr / p.rows;
    if (p.cu && (row < p.cu[0] || row >= p.cu[p.n_seqs])) return;   // rows of no sequence
    f32x4 a = {0.f, 0.f, 0.f, 0.f};
    const f32x4* src = reinterpret_cast<const f32x4*>(q.part) + which * q.blocks * per + e;
    for (int b = 0; b < q.blocks; ++b) a += src[b * per];
    const int64_t at = row * (which ? q.gC_stride : q.gB_stride) + (p.g0 + gw) * p.N + 4 * n;
    void* to = which ? q.gC : q.gB;
    if constexpr (sizeof(InT) == 2)
        *reinterpret_cast<u32x2*>((__bf16*)to + at) = u32x2{pack_bf2(a[0], a[1]), pack_bf2(a[2], a[3])};
    else
        *reinterpret_cast<f32x4*>((float*)to + at) = a;
}

// Per head: the chunks' sums for A, D and dt_bias, in slot order per lane.
__device__ __forceinline__ void ssm_grad_sums(const SsmGradParams& q, int64_t hw) {
    const SsmScanParams& p = q.f;
    const int64_t heads = (int64_t)p.gn * (p.H / p.G);
    double a[3] = {0.0, 0.0, 0.0};
    for (int64_t s = threadIdx.x; s < q.slots; s += SS_THREADS)
#pragma unroll
        for (int k = 0; k < 3; ++k) a[k] += (double)q.sums[(s * heads + hw) * 3 + k];
    __shared__ double lds[3][SS_THREADS / 64];
#pragma unroll
    for (int k = 0; k < 3; ++k) {
#pragma unroll
        for (int o = 32; o > 0; o >>= 1) a[k] += __shfl_xor(a[k], o);
        if ((threadIdx.x & 63) == 0) lds[k][threadIdx.x >> 6] = a[k];
    }
    __syncthreads();
    if (threadIdx.x < 3) {
        const int k = threadIdx.x;
        const float v = (float)((lds[k][0] + lds[k][1]) + (lds[k][2] + lds[k][3]));
        float* to = k == 0 ? q.gA : k == 1 ? q.gD : q.gbias;
        if (to) to[p.g0 * (p.H / p.G) + hw] = v;
    }
}

// Zeros in the rows of no sequence (packed batches), a row per workgroup at a
// time; all columns, of every group of heads.
template <typename InT>
__device__ __forceinline__ void ssm_grad_rest(const SsmGradParams& q, int64_t first, int64_t step) {
    const SsmScanParams& p = q.f;
    const int64_t begin = ssm_range(p.cu, p.rows, p.T, 0).start;
    const int64_t end = ssm_range(p.cu, p.rows, p.T, p.n_seqs - 1).end;
    auto clear = [&](void* to, int64_t at, int64_t n) {   // n elements from `at`, whole 16-byte pieces
        u32x4* t = reinterpret_cast<u32x4*>((InT*)to + at);
        for (int64_t i = threadIdx.x; i < n * (int64_t)sizeof(InT) / 16; i += SS_THREADS) t[i] = u32x4{0, 0, 0, 0};
    };
    for (int64_t i = first; i < begin + (p.rows - end); i += step) {
        const int64_t row = i < begin ? i : end + (i - begin);
        if (q.zero_rest & KDA_FRESH_X) clear(q.gx, row * q.gx_stride, (int64_t)p.H * p.P);
        if (q.zero_rest & KDA_FRESH_B) clear(q.gB, row * q.gB_stride, (int64_t)p.G * p.N);
        if (q.zero_rest & KDA_FRESH_C) clear(q.gC, row * q.gC_stride, (int64_t)p.G * p.N);
        if (q.zero_rest & KDA_FRESH_DT)
            for (int h = threadIdx.x; h < p.H; h += SS_THREADS) q.gdt[row * p.H + h] = 0.f;
    }
}

// All in one launch: `bc` workgroups for dB and dC, then one per head, then
// those for the rows of no sequence.
template <typename InT>
__global__ __launch_bounds__(SS_THREADS) void ssm_grad_tail_kernel(SsmGradParams q, int64_t bc) {
    const int64_t heads = (int64_t)q.f.gn * (q.f.H / q.f.G), i = (int64_t)blockIdx.x - bc;
    if (i < 0) ssm_grad_bc<InT>(q);
    else if (i < heads) ssm_grad_sums(q, i);
    else ssm_grad_rest<InT>(q, i - heads, (int64_t)gridDim.x - bc - heads);
}

template <typename InT>
static hipError_t run_grad(const SsmGradParams& q, hipStream_t stream) {
    const SsmScanParams& p = q.f;
    if (q.slots > 0) {
        const dim3 grid((unsigned)(q.slots * p.gn * q.blocks)), wide(SG_THREADS);
        if (p.N == 128 && p.P == 64) hipLaunchKernelGGL((ssm_grad_kernel<InT, 128, 64>), grid, wide, 0, stream, q);
        else if (p.N == 128) hipLaunchKernelGGL((ssm_grad_kernel<InT, 128, 128>), grid, wide, 0, stream, q);
        else if (p.P == 64) hipLaunchKernelGGL((ssm_grad_kernel<InT, 64, 64>), grid, wide, 0, stream, q);
        else hipLaunchKernelGGL((ssm_grad_kernel<InT, 64, 128>), grid, wide, 0, stream, q);
    }
    const int64_t n = q.blocks > 1 ? 2 * (int64_t)p.gn * p.rows * (p.N / 4) : 0, bc = (n + SS_THREADS - 1) / SS_THREADS;
    const int64_t rest = q.zero_rest && p.n_seqs > 0 ? (p.rows < kGradRest ? p.rows : kGradRest) : 0;
    hipLaunchKernelGGL(ssm_grad_tail_kernel<InT>, dim3((unsigned)(bc + p.gn * (p.H / p.G) + rest)), dim3(SS_THREADS), 0,
                       stream, q, bc);
    return hipGetLastError();
}
hipError_t launch_ssm_grad(const SsmGradParams& q, bool bf16_in, hipStream_t stream) {
    return bf16_in ? run_grad<__bf16>(q, stream) : run_grad<float>(q, stream);
}

}  // namespace kda
