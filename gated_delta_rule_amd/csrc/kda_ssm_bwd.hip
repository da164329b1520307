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
// (the first sum by differences of row and column sums of W without its
// diagonal, over one chunk only), and
//   ddt_s = sum_u W_us / dt_s + V_s / dt_s + A da_s,  dA = sum_t dt_t da_t,
//   dD    = sum_t E_tt,
// with the divisions left out of the sums in the first place.
//
// A workgroup runs one chunk for several heads of a group in turn: B, C and
// the tiles of G stay on chip, and dB and dC are summed over the heads in
// registers, so that only one partial sum per workgroup goes through memory.
// Wave w owns a quarter of the state's rows (for dB, dC, U, V, Z) and of x's
// columns (for dx).  S and R come straight from memory into operand
// registers, each row once.  Bound by the traffic of S and R, which the walks
// wrote: 16 N P bytes per chunk and head against 6 L P of x, dy and dx.
#include "kda_ssm_tile.h"

namespace kda {

__device__ __forceinline__ float sum_lane_groups(float v) {   // over lanes with equal l & 15
    v += __shfl_xor(v, 16);
    v += __shfl_xor(v, 32);
    return v;
}

template <typename InT, int N, int P>
__global__ __launch_bounds__(SS_THREADS, sizeof(InT) == 2 && P == 64 ? 2 : 1) void ssm_grad_kernel(SsmGradParams q) {
    constexpr bool BF = sizeof(InT) == 2;
    constexpr int L = BF ? 64 : 32;
    constexpr int XP = BF ? 1 : 3;      // bf16 parts of an input
    constexpr int KP = BF ? 1 : 3;      // ... of the chunk matrices (their products are rounded to the input type)
    constexpr int RP = BF ? 1 : 3;      // ... of R in dx
    constexpr int SP = 3;               // ... of S and R where U and V come from (float32 results)
    constexpr int TT = L / 16, NTILE = TT * (TT + 1) / 2, TPW = (NTILE + 3) / 4;
    constexpr int MT = N / 64, PT = P / 64;   // row tiles of the state, column tiles of x per wave
    __shared__ __attribute__((aligned(16))) __bf16 tB[XP * L * N], tC[XP * L * N];
    __shared__ __attribute__((aligned(16))) __bf16 tX[XP * L * P], tY[XP * L * P];
    __shared__ __attribute__((aligned(16))) __bf16 tK[KP * L * L], tM[KP * L * L];
    __shared__ ChunkDecay<L> dec;
    __shared__ float sR[TT][L], sQ[TT][L], sU[4][L], sV[4][L], sW[L], sE[L], sZ[4];

    const SsmScanParams& p = q.f;
    const int tid = threadIdx.x;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    int lane = tid & 63;
    int rN = lane_row<N>(lane), rP = lane_row<P>(lane), rL = lane_row<L>(lane);
    int2 cN = lane_col<N, 4>(lane), cP = lane_col<P, 4>(lane), cL = lane_col<L, 4>(lane);
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
        for (int i = tid; i < 3 * hwn; i += SS_THREADS) q.sums[(slot * heads + hw0) * 3 + i] = 0.f;
        return;
    }
    const int64_t row0 = s.r0;
    const int valid = (int)(s.r1 - s.r0);

    for (int i = tid; i < KP * L * L / 8; i += SS_THREADS) {
        reinterpret_cast<u32x4*>(tK)[i] = u32x4{0, 0, 0, 0};
        reinterpret_cast<u32x4*>(tM)[i] = u32x4{0, 0, 0, 0};
    }
    Stager<InT, L, P, SS_THREADS> gX, gY;
    float gdt = 0.f;
    auto fetch = [&](int hw) {
        const int64_t h = hfirst + hw;
        gX.load((const InT*)p.x + row0 * p.x_stride + h * P, p.x_stride, valid, P);
        gY.load((const InT*)q.gy + (row0 * p.H + h) * P, (int64_t)p.H * P, valid, P);
        if (wave == 0) gdt = lane < valid ? p.dt[(row0 + lane) * p.H + h] : 0.f;
    };
    {
        Stager<InT, L, N, SS_THREADS> g;
        g.load((const InT*)p.B + row0 * p.B_stride + grp * N, p.B_stride, valid, N);
        g.put(tB);
        g.load((const InT*)p.C + row0 * p.C_stride + grp * N, p.C_stride, valid, N);
        g.put(tC);
    }
    fetch(hw0);
    __syncthreads();

    // tiles of G^T (rows s, columns t), kept for all heads
    f32x4 G[TPW];
    int g_tt[TPW], g_st[TPW];
#pragma unroll
    for (int k = 0; k < TPW; ++k) {
        const int idx = wave + 4 * k < NTILE ? wave + 4 * k : NTILE - 1;
        int tt = 0;
        while ((tt + 1) * (tt + 2) / 2 <= idx) ++tt;
        g_tt[k] = tt;
        g_st[k] = idx - tt * (tt + 1) / 2;
        G[k] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int ks = 0; ks < N / 32; ++ks) {
            bf16x8 fb[XP], fc[XP];
#pragma unroll
            for (int i = 0; i < XP; ++i) {
                fb[i] = frag_row<N>(tB + i * L * N, 16 * g_st[k], ks, rN);
                fc[i] = frag_row<N>(tC + i * L * N, 16 * g_tt[k], ks, rN);
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

    f32x4 dB[MT][TT], dC[MT][TT];   // rows n, columns token, of all heads so far
#pragma unroll
    for (int m = 0; m < MT; ++m)
#pragma unroll
        for (int t = 0; t < TT; ++t) dB[m][t] = dC[m][t] = f32x4{0.f, 0.f, 0.f, 0.f};

    for (int hw = hw0; hw < hw0 + hwn; ++hw) {
        const int h = hfirst + hw;
        hide(lane), hide(rN), hide(rP), hide(rL), hide(cN), hide(cP), hide(cL);
        const int l15 = lane & 15, lg = lane >> 4;
        const float* S = q.states + (slot * heads + hw) * (N * P);
        const float* R = q.dstates + (slot * heads + hw) * (N * P);
        const float bias = p.dt_bias ? p.dt_bias[h] : 0.f;
        const float raw = gdt + bias;          // wave 0
        const float A = p.A[h], D = p.D ? p.D[h] : 0.f;
        gX.put(tX);
        gY.put(tY);
        if (wave == 0) chunk_decay<L>(dec, gdt, lane < valid, bias, p.softplus, A);
        lds_barrier();
        // S and R rows of this wave, in flight during the chunk matrices
        f32x4 fS[MT][P / 32][2], fR[MT][P / 32][2];
#pragma unroll
        for (int m = 0; m < MT; ++m)
#pragma unroll
            for (int ks = 0; ks < P / 32; ++ks) {
                const int at = ((N / 4) * wave + 16 * m + l15) * P + 32 * ks + 8 * lg;
#pragma unroll
                for (int k = 0; k < 2; ++k) {
                    fS[m][ks][k] = *reinterpret_cast<const f32x4*>(S + at + 4 * k);
                    fR[m][ks][k] = *reinterpret_cast<const f32x4*>(R + at + 4 * k);
                }
            }
        __builtin_amdgcn_sched_barrier(0);

        // chunk matrices, a lane holding four neighbouring s of one t
#pragma unroll
        for (int k = 0; k < TPW; ++k) {
            if (wave + 4 * k >= NTILE) break;
            const int tt = g_tt[k], st = g_st[k];
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
            const int t = 16 * tt + l15, s0 = 16 * st + 4 * lg;
            const float ht = dec.gh[t], lt = dec.gl[t];
            const f32x4 hs = *reinterpret_cast<const f32x4*>(&dec.gh[s0]);
            const f32x4 ls = *reinterpret_cast<const f32x4*>(&dec.gl[s0]);
            const f32x4 ds = *reinterpret_cast<const f32x4*>(&dec.dt[s0]);
            float K[4], M[4], row = 0.f, col[4];
#pragma unroll
            for (int r = 0; r < 4; ++r) {
                const int sr = s0 + r;
                const float l = sr <= t ? __expf((ht - hs[r]) + (lt - ls[r])) : 0.f;
                K[r] = sr <= t ? E[r] * l * ds[r] : 0.f;
                M[r] = sr <= t ? G[k][r] * l * ds[r] : 0.f;
                const float w = sr <= t ? G[k][r] * l * E[r] : 0.f;
                col[r] = sr < t ? w : 0.f;
                row += col[r] * ds[r];
                if (tt == st && sr == t) {
                    M[r] += D;
                    sW[t] = w;
                    sE[t] = E[r];
                }
            }
            row = sum_lane_groups(row);
            if (lg == 0) sR[st][t] = row;
#pragma unroll
            for (int r = 0; r < 4; ++r) {
                float v = col[r];
                v += dpp_mov<0xB1>(v);
                v += dpp_mov<0x4E>(v);
                v += dpp_mov<0x124>(v);
                v += dpp_mov<0x128>(v);
                if (l15 == 0) sQ[tt][s0 + r] = v;
            }
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
        }

        // products with S and R: rows n = (N / 4) wave + 16 m + .., columns token
        __builtin_amdgcn_sched_barrier(0);
        float z = 0.f, u[TT], v[TT];
#pragma unroll
        for (int t = 0; t < TT; ++t) u[t] = v[t] = 0.f;
#pragma unroll
        for (int m = 0; m < MT; ++m) {
            const int n0 = (N / 4) * wave + 16 * m;
            f32x4 aC[TT], aB[TT];
#pragma unroll
            for (int t = 0; t < TT; ++t) aC[t] = aB[t] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
            for (int ks = 0; ks < P / 32; ++ks) {
                float vS[8], vR[8];
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    vS[e] = fS[m][ks][e / 4][e % 4];
                    vR[e] = fR[m][ks][e / 4][e % 4];
                    z = fmaf(vS[e], vR[e], z);
                }
                bf16x8 pS[SP], pR[SP];
                parts8<SP>(vS, pS);
                parts8<SP>(vR, pR);
#pragma unroll
                for (int t = 0; t < TT; ++t) {
                    bf16x8 fy[XP], fx[XP];
#pragma unroll
                    for (int i = 0; i < XP; ++i) {
                        fy[i] = frag_row<P>(tY + i * L * P, 16 * t, ks, rP);
                        fx[i] = frag_row<P>(tX + i * L * P, 16 * t, ks, rP);
                    }
                    aC[t] = mma_parts<SP, XP>(pS, fy, aC[t]);
                    aB[t] = mma_parts<SP, XP>(pR, fx, aB[t]);
                }
                __builtin_amdgcn_sched_barrier(0);
            }
#pragma unroll
            for (int t = 0; t < TT; ++t) {
                float c[4], b[4];
                four(tC, L * N, 16 * t + l15, n0 + 4 * lg, c);
                four(tB, L * N, 16 * t + l15, n0 + 4 * lg, b);
                const float eg = dec.eg[16 * t + l15], w = dec.w[16 * t + l15];
#pragma unroll
                for (int r = 0; r < 4; ++r) {
                    u[t] = fmaf(c[r], aC[t][r], u[t]);
                    v[t] = fmaf(b[r], aB[t][r], v[t]);
                    dC[m][t][r] = fmaf(eg, aC[t][r], dC[m][t][r]);
                    dB[m][t][r] = fmaf(w, aB[t][r], dB[m][t][r]);
                }
            }
            __builtin_amdgcn_sched_barrier(0);
        }
        z = wave_sum_dpp(z);
        if (lane == 0) sZ[wave] = z;
#pragma unroll
        for (int t = 0; t < TT; ++t) {
            const float a = sum_lane_groups(u[t]), b = sum_lane_groups(v[t]);
            if (lg == 0) {
                sU[wave][16 * t + l15] = a;
                sV[wave][16 * t + l15] = b;
            }
        }
        lds_barrier();   // the chunk matrices and the partial sums are whole
        if (hw + 1 < hw0 + hwn) fetch(hw + 1);

        // products with the chunk matrices
#pragma unroll
        for (int m = 0; m < MT; ++m) {
            const int n0 = (N / 4) * wave + 16 * m;
#pragma unroll
            for (int ks = 0; ks < L / 32; ++ks) {
                bf16x8 fb[XP], fc[XP];
#pragma unroll
                for (int i = 0; i < XP; ++i) {
                    fb[i] = frag_col<N>(tB + i * L * N, n0, ks, cN);
                    fc[i] = frag_col<N>(tC + i * L * N, n0, ks, cN);
                }
#pragma unroll
                for (int t = 0; t < TT; ++t) {
                    if (ks <= t / 2) {
                        bf16x8 fk[KP];
#pragma unroll
                        for (int i = 0; i < KP; ++i) fk[i] = frag_row<L>(tK + i * L * L, 16 * t, ks, rL);
                        dC[m][t] = mma_parts<XP, KP>(fb, fk, dC[m][t]);
                    }
                    if (ks >= t / 2) {
                        bf16x8 fk[KP];
#pragma unroll
                        for (int i = 0; i < KP; ++i) fk[i] = frag_col<L>(tK + i * L * L, 16 * t, ks, cL);
                        dB[m][t] = mma_parts<XP, KP>(fc, fk, dB[m][t]);
                    }
                }
            }
            __builtin_amdgcn_sched_barrier(0);
        }
#pragma unroll
        for (int c = 0; c < PT; ++c) {
            const int p0 = (P / 4) * wave + 16 * c;
            f32x4 dX[TT];
#pragma unroll
            for (int t = 0; t < TT; ++t) dX[t] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
            for (int ks = 0; ks < N / 32; ++ks) {
                float f[8];
#pragma unroll
                for (int e = 0; e < 8; ++e) f[e] = R[(32 * ks + 8 * lg + e) * P + p0 + l15];
                bf16x8 pR[RP];
                parts8<RP>(f, pR);
#pragma unroll
                for (int t = 0; t < TT; ++t) {
                    bf16x8 fb[XP];
#pragma unroll
                    for (int i = 0; i < XP; ++i) fb[i] = frag_row<N>(tB + i * L * N, 16 * t, ks, rN);
                    dX[t] = mma_parts<RP, XP>(pR, fb, dX[t]);
                }
            }
#pragma unroll
            for (int t = 0; t < TT; ++t) dX[t] *= dec.w[16 * t + l15];
#pragma unroll
            for (int ks = 0; ks < L / 32; ++ks) {
                bf16x8 fy[XP];
#pragma unroll
                for (int i = 0; i < XP; ++i) fy[i] = frag_col<P>(tY + i * L * P, p0, ks, cP);
#pragma unroll
                for (int t = 0; t < TT; ++t) {
                    if (ks < t / 2) continue;
                    bf16x8 fm[KP];
#pragma unroll
                    for (int i = 0; i < KP; ++i) fm[i] = frag_col<L>(tM + i * L * L, 16 * t, ks, cL);
                    dX[t] = mma_parts<XP, KP>(fy, fm, dX[t]);
                }
            }
#pragma unroll
            for (int t = 0; t < TT; ++t) {
                const int row = 16 * t + l15;
                if (row < valid) {
                    const int64_t at = (row0 + row) * q.gx_stride + (int64_t)h * P + p0 + 4 * lg;
                    if constexpr (BF)
                        *reinterpret_cast<u32x2*>((__bf16*)q.gx + at) =
                            u32x2{pack_bf2(dX[t][0], dX[t][1]), pack_bf2(dX[t][2], dX[t][3])};
                    else
                        *reinterpret_cast<f32x4*>((float*)q.gx + at) = dX[t];
                }
            }
        }

        // gradients of the decay and of dt: one token per lane of wave 0
        if (wave == 0) {
            const int t = lane < L ? lane : L - 1;
            float R_ = 0.f, Q = 0.f;
#pragma unroll
            for (int k = 0; k < TT; ++k) {
                if (k <= t / 16) R_ += sR[k][t];
                if (k >= t / 16) Q += sQ[k][t];
            }
            const float dt = dec.dt[t];
            const float er = expf((dec.gh[L - 1] - dec.gh[t]) + (dec.gl[L - 1] - dec.gl[t]));
            const float U = dec.eg[t] * ((sU[0][t] + sU[1][t]) + (sU[2][t] + sU[3][t]));
            const float V = er * ((sV[0][t] + sV[1][t]) + (sV[2][t] + sV[3][t]));   // without dt
            const float Z = dec.eL * ((sZ[0] + sZ[1]) + (sZ[2] + sZ[3]));
            double suf = lane < L ? (double)R_ - (double)(Q * dt) + (double)U : 0.0;
            double pre = lane < L ? (double)(V * dt) : 0.0;
            const double own = pre;
#pragma unroll
            for (int o = 1; o < L; o <<= 1) {
                const double a = __shfl_down(suf, o), b = __shfl_up(pre, o);
                if (lane + o < L) suf += a;
                if (lane >= o) pre += b;
            }
            const float da = (float)(suf + (pre - own) + (double)Z);
            float ddt = (Q + sW[t]) + V + A * da;
            if (p.softplus) ddt *= 1.f / (1.f + expf(-raw));
            const bool on = lane < valid;
            if (on) q.gdt[(row0 + lane) * p.H + h] = ddt;
            const float a = wave_sum_dpp(on ? dt * da : 0.f);
            const float d = wave_sum_dpp(on ? sE[t] : 0.f);
            const float b = wave_sum_dpp(on ? ddt : 0.f);
            if (lane == 0) {
                float* to = q.sums + (slot * heads + hw) * 3;
                to[0] = a;
                to[1] = d;
                to[2] = b;
            }
        }
        lds_barrier();   // the tiles are consumed (rows and stores stay in flight)
    }

    // dB and dC of these heads: the gradients themselves, or a partial sum
    const int l15 = lane & 15, lg = lane >> 4;
#pragma unroll
    for (int m = 0; m < MT; ++m)
#pragma unroll
        for (int t = 0; t < TT; ++t) {
            const int row = 16 * t + l15, n = (N / 4) * wave + 16 * m + 4 * lg;
            if (row >= valid) continue;
            if (q.blocks == 1) {
                const int64_t b = (row0 + row) * q.gB_stride + grp * N + n, c = (row0 + row) * q.gC_stride + grp * N + n;
                if constexpr (BF) {
                    *reinterpret_cast<u32x2*>((__bf16*)q.gB + b) =
                        u32x2{pack_bf2(dB[m][t][0], dB[m][t][1]), pack_bf2(dB[m][t][2], dB[m][t][3])};
                    *reinterpret_cast<u32x2*>((__bf16*)q.gC + c) =
                        u32x2{pack_bf2(dC[m][t][0], dC[m][t][1]), pack_bf2(dC[m][t][2], dC[m][t][3])};
                } else {
                    *reinterpret_cast<f32x4*>((float*)q.gB + b) = dB[m][t];
                    *reinterpret_cast<f32x4*>((float*)q.gC + c) = dC[m][t];
                }
            } else {
                const int64_t at = (((int64_t)blk * p.gn + gw) * p.rows + row0 + row) * N + n;
                *reinterpret_cast<f32x4*>(q.part + at) = dB[m][t];
                *reinterpret_cast<f32x4*>(q.part + (int64_t)q.blocks * p.gn * p.rows * N + at) = dC[m][t];
            }
        }
}

// Adds up the head blocks' partial sums of dB and dC, four channels per lane.
template <typename InT>
__global__ __launch_bounds__(SS_THREADS) void ssm_grad_bc_kernel(SsmGradParams q) {
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
__global__ __launch_bounds__(SS_THREADS) void ssm_grad_sums_kernel(SsmGradParams q) {
    const SsmScanParams& p = q.f;
    const int64_t hw = blockIdx.x, heads = (int64_t)p.gn * (p.H / p.G);
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

template <typename InT>
static hipError_t run_grad(const SsmGradParams& q, hipStream_t stream) {
    const SsmScanParams& p = q.f;
    const dim3 block(SS_THREADS);
    if (q.slots > 0) {
        const dim3 grid((unsigned)(q.slots * p.gn * q.blocks));
        if (p.N == 128 && p.P == 64) hipLaunchKernelGGL((ssm_grad_kernel<InT, 128, 64>), grid, block, 0, stream, q);
        else if (p.N == 128) hipLaunchKernelGGL((ssm_grad_kernel<InT, 128, 128>), grid, block, 0, stream, q);
        else if (p.P == 64) hipLaunchKernelGGL((ssm_grad_kernel<InT, 64, 64>), grid, block, 0, stream, q);
        else hipLaunchKernelGGL((ssm_grad_kernel<InT, 64, 128>), grid, block, 0, stream, q);
    }
    if (q.blocks > 1 && p.rows > 0) {
        const int64_t n = 2 * (int64_t)p.gn * p.rows * (p.N / 4);
        hipLaunchKernelGGL(ssm_grad_bc_kernel<InT>, dim3((unsigned)((n + SS_THREADS - 1) / SS_THREADS)), block, 0, stream, q);
    }
    hipLaunchKernelGGL(ssm_grad_sums_kernel, dim3((unsigned)(p.gn * (p.H / p.G))), block, 0, stream, q);
    return hipGetLastError();
}
hipError_t launch_ssm_grad(const SsmGradParams& q, bool bf16_in, hipStream_t stream) {
    return bf16_in ? run_grad<__bf16>(q, stream) : run_grad<float>(q, stream);
}

}  // namespace kda
