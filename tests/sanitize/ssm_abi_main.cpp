// Sanitizer driver for the host code of kda_ssm.h and kda_spec.h
// (gated_delta_rule_amd/csrc/kda_ssm_abi.hip compiled as plain C++ with g++
// and -fsanitize=address,undefined by tests/test_ssm_sanitizers.py; CPU only).
// The kernel launchers are replaced by stubs that check what they are asked to
// launch: every array of a plan lies within the workspace of the call, no
// launch has 2^32 threads, segments and head blocks cover everything.  Sizes
// are drawn from small, odd and extreme values, so that the arithmetic of the
// validation runs at its limits.  The pointers are fake device addresses that
// are never dereferenced.
#include <stdint.h>
#include <stdio.h>

#include "kda_spec.h"
#include "kda_ssm.h"
#include "kda_ssm_launch.h"

namespace {
int fails = 0;
long launched = 0;
uintptr_t ws_lo = 0, ws_hi = 0;   // the running call's workspace
#define CHECK(c)                                                               \
    do {                                                                       \
        if (!(c)) {                                                            \
            if (fails < 20) fprintf(stderr, "check failed: %s (line %d)\n", #c, __LINE__); \
            ++fails;                                                           \
        }                                                                      \
    } while (0)
typedef __int128 big;
void in_ws(const void* p, big bytes) {
    const big at = (big)(uintptr_t)p;
    CHECK(at >= (big)ws_lo && at + bytes <= (big)ws_hi && at % 4 == 0);
}
void threads(big workgroups, int per) { CHECK(workgroups >= 0 && workgroups * per < ((big)1 << 32)); }
big cdiv(big a, big b) { return (a + b - 1) / b; }

uint64_t seed = 12345;
uint32_t rnd(uint32_t n) {
    seed = seed * 6364136223846793005ull + 1442695040888963407ull;
    return (uint32_t)(seed >> 33) % n;
}
template <typename T, int N>
T pick(const T (&a)[N]) {
    return a[rnd(N)];
}

void check_scan(const kda::SsmScanParams& p, int dirs) {
    const big heads = (big)p.gn * (p.H / p.G), np = (big)p.N * p.P;
    const big rows = p.cu ? p.T : (big)p.n_seqs * p.T;
    CHECK(p.rows == rows && p.g0 >= 0 && p.gn >= 1 && p.g0 + p.gn <= p.G);
    const int hpw = 128 / p.P;
    threads((big)p.slots * p.gn * cdiv(p.H / p.G, hpw), 512);
    if (p.cut) {
        CHECK(p.seg_len > 0 && p.seg_len % 64 == 0);
        CHECK((big)p.slots == (p.cu ? rows / p.seg_len + p.n_seqs : p.n_seqs * cdiv(p.T, p.seg_len)));
        in_ws(p.seg, (big)p.slots * heads * np * 4);
        CHECK((uintptr_t)p.seg % 16 == 0);
        in_ws(p.seg_decay, (big)p.slots * heads * 4);
        threads(cdiv(np / 4 * p.n_seqs * heads, 256), 256);
    } else {
        CHECK(p.slots == p.n_seqs);
    }
    (void)dirs;
    ++launched;
}
}  // namespace

namespace kda {
hipError_t launch_conv_fwd(const ConvParams& p, bool, hipStream_t) {
    CHECK(p.channels % 8 == 0 && p.width >= 2 && p.width <= 4);
    const big strips = cdiv(p.channels, 256), rpw = conv_rows_per_wave(p.rows, p.channels);
    threads(strips * cdiv(p.rows, kConvWaves * rpw), 64 * (int)kConvWaves);
    threads(cdiv((big)p.n_seqs * (p.channels / 4), 64), 64);
    ++launched;
    return hipSuccess;
}
hipError_t launch_conv_step(const ConvParams& p, bool, hipStream_t) {
    CHECK(p.cache && p.T >= 0 && p.T <= 64 && p.Tr >= 0 && p.Tr <= 64);
    threads(cdiv((big)p.n_seqs * (p.channels / 4), 64), 64);
    ++launched;
    return hipSuccess;
}
hipError_t launch_conv_bwd(const ConvBwdParams& q, bool, hipStream_t) {
    const ConvParams& p = q.f;
    const big parts = conv_bwd_parts(p.rows, p.channels);
    CHECK(q.rows_per_wave == conv_rows_per_wave(p.rows, p.channels) && q.rows_per_wave >= 4);
    CHECK((big)parts * kConvWaves * q.rows_per_wave >= p.rows);
    if (p.rows > 0) in_ws(q.partial, parts * (p.width + 1) * p.channels * 4);
    threads(cdiv(p.channels, 256) * parts, 64 * (int)kConvWaves);
    threads(cdiv((big)(p.width + 1) * p.channels, 64) + cdiv((big)p.n_seqs * (p.channels / 4), 256), 256);
    ++launched;
    return hipSuccess;
}
hipError_t launch_ssm_chunk_fwd(const SsmScanParams& p, bool, hipStream_t) {
    check_scan(p, 1);
    CHECK(p.g0 == 0 && p.gn == p.G);
    return hipSuccess;
}
hipError_t launch_ssm_walks(const SsmScanDirs& d, bool bf16_in, hipStream_t) {
    const int64_t L = ssm_chunk_tokens(bf16_in);
    for (const SsmScanParams& p : d.dir) {
        check_scan(p, 2);
        const big chunks = p.cu ? p.rows / L + p.n_seqs : p.n_seqs * cdiv(p.T, L);
        in_ws(p.states, chunks * p.gn * (p.H / p.G) * p.N * p.P * 4);
        CHECK((uintptr_t)p.states % 16 == 0);
    }
    CHECK(d.dir[0].slots == d.dir[1].slots && d.dir[0].seg_len == d.dir[1].seg_len);
    CHECK(!d.dir[0].cut || d.dir[0].seg + (int64_t)d.dir[0].slots * d.dir[0].gn * (d.dir[0].H / d.dir[0].G) *
                                              d.dir[0].N * d.dir[0].P <= d.dir[1].seg);
    CHECK(!d.dir[0].S_T);
    return hipSuccess;
}
hipError_t launch_ssm_grad(const SsmGradParams& q, bool bf16_in, hipStream_t) {
    const SsmScanParams& p = q.f;
    const int64_t L = ssm_chunk_tokens(bf16_in);
    const big hpg = p.H / p.G, heads = p.gn * hpg;
    CHECK(p.n_seqs == 0 || (big)q.slots == (p.cu ? p.rows / L + p.n_seqs : p.n_seqs * cdiv(p.T, L)));
    CHECK(q.heads_per_block >= 1 && (big)q.blocks * q.heads_per_block >= hpg &&
          (big)(q.blocks - 1) * q.heads_per_block < hpg);
    threads((big)q.slots * p.gn * q.blocks, 512);
    threads((q.blocks > 1 ? cdiv(2 * (big)p.gn * p.rows * (p.N / 4), 256) : 0) + heads, 256);
    if (q.blocks > 1) {
        in_ws(q.part, 2 * (big)q.blocks * p.gn * p.rows * p.N * 4);
        CHECK((uintptr_t)q.part % 16 == 0);
    }
    if (q.slots > 0) {
        in_ws(q.sums, (big)q.slots * heads * 3 * 4);
        in_ws(q.states, (big)q.slots * heads * p.N * p.P * 4);
        in_ws(q.dstates, (big)q.slots * heads * p.N * p.P * 4);
        CHECK(q.dstates - q.states >= (int64_t)((big)q.slots * heads * p.N * p.P));
    }
    ++launched;
    return hipSuccess;
}
hipError_t launch_ssm_recurrent(const SsmRecParams& p, bool, hipStream_t) {
    CHECK(p.S && p.rep.T >= 0 && p.rep.T <= 64 && p.out.T >= 0 && p.out.T <= 64);
    threads((big)p.B * p.H, 256);
    ++launched;
    return hipSuccess;
}
hipError_t launch_verify(const VerifyParams& p, bool, hipStream_t) {
    CHECK(p.n_parts == cdiv(p.V, kVerifyPart) && p.run >= 1);
    in_ws(p.partial, (big)p.B * p.n_parts * 16);
    threads((big)p.B * cdiv(p.n_parts, p.run), kVerifyThreads);
    ++launched;
    return hipSuccess;
}
}  // namespace kda

int main() {
    // distinct fake addresses, 2^55 bytes apart: no tensor reaches the next
    auto at = [](int i) { return (float*)((uintptr_t)(i + 1) << 55); };
    const int32_t counts[] = {0, 1, 2, 3, 17, 128, 4097, 65536, 1 << 20, INT32_MAX, -1, INT32_MIN};
    const int64_t lens[] = {0, 1, 5, 63, 64, 65, 517, 4096, 100000, 1 << 24, (int64_t)1 << 31, (int64_t)1 << 40, INT64_MAX, -1};
    const int32_t heads[] = {1, 2, 6, 7, 64, 96, 1024, 65536, 65537, 0};
    const int32_t dims[] = {64, 128, 64, 128, 32};
    const int32_t chans[] = {8, 64, 264, 4352, 65536, 1 << 28, INT32_MAX - 7, 12, 0};
    const int32_t toks[] = {0, 1, 4, 64, 65};
    hipStream_t st = nullptr;
    for (int i = 0; i < 400000; ++i) {
        const int dt = rnd(20) ? (int)rnd(2) : 2;
        const int32_t n = pick(counts), H = pick(heads), N = pick(dims), P = pick(dims), c = pick(chans);
        const int32_t G = rnd(3) ? 1 : H > 1 && H % 2 == 0 ? (rnd(2) ? 2 : H) : H, W = 1 + (int32_t)rnd(4);
        const int64_t T = pick(lens);
        const int32_t* cu = rnd(2) ? (const int32_t*)at(30) : nullptr;
        const int64_t es = dt == KDA_BF16 ? 2 : 4;
        auto stride = [&](int64_t width) { return rnd(8) ? width : (int64_t)(rnd(2) ? width + 16 : (1 << 23) + (int)rnd(2) * 8); };
        const int64_t xw = (int64_t)H * P, bw = (int64_t)G * N;
        auto ws = [&](size_t bytes) {
            ws_lo = (uintptr_t)at(40);
            ws_hi = ws_lo + bytes;
            return (void*)ws_lo;
        };
        const int64_t rows = cu ? T : T > 0 && n > 0 && T <= INT64_MAX / n ? n * T : 0;
        (void)es;
        switch (rnd(7)) {
        case 0:
            kda_ssm_conv_fwd(at(1), stride(c), dt, at(2), rnd(2) ? at(3) : nullptr, rnd(2) ? at(4) : nullptr, cu, n, T, c, W,
                             1, at(5), st);
            break;
        case 1:
            kda_ssm_conv_step(at(1), stride(c), dt, at(2), nullptr, at(4), at(6), stride(c), rnd(2) ? (int32_t*)at(7) : nullptr,
                              n, pick(toks), pick(toks), c, W, 1, (int)rnd(2), at(5), st);
            break;
        case 2: {
            const size_t need = kda_ssm_conv_bwd_workspace_bytes(rows, c, W);
            const size_t have = rnd(8) ? need : need / 2;
            kda_ssm_conv_bwd(at(1), stride(c), dt, at(2), at(3), rnd(2) ? at(4) : nullptr, cu, n, T, c, W, 1, at(8), stride(c),
                             at(9), at(10), at(11), rnd(2) ? at(12) : nullptr, ws(have), have, st);
            break;
        }
        case 3: {
            const size_t need = kda_ssm_chunk_fwd_workspace_bytes(n, T, H, G, N, P, cu != nullptr);
            const size_t have = rnd(4) ? need : need / 2;
            kda_ssm_chunk_fwd(at(1), stride(xw), at(2), stride(bw), at(3), stride(bw), dt, at(4), at(5), 1, at(6), at(7),
                              rnd(2) ? at(8) : nullptr, cu, n, T, H, G, N, P, at(9), rnd(2) ? at(10) : nullptr, ws(have), have, st);
            break;
        }
        case 4: {
            const size_t need = kda_ssm_chunk_bwd_workspace_bytes(dt, n, T, H, G, N, P, cu != nullptr, rnd(2) ? G : 1);
            const size_t have = rnd(8) ? need : need / 2;
            kda_ssm_chunk_bwd(at(1), stride(xw), at(2), stride(bw), at(3), stride(bw), dt, at(4), at(5), 1, at(6), at(7),
                              rnd(2) ? at(8) : nullptr, cu, n, T, H, G, N, P, at(9), rnd(2) ? at(10) : nullptr, at(11), stride(xw),
                              at(12), stride(bw), at(13), stride(bw), at(14), at(15), at(16), at(17), rnd(2) ? at(18) : nullptr,
                              ws(have), have, st);
            break;
        }
        case 5:
            kda_ssm_recurrent_fwd(at(1), stride(xw), at(2), stride(bw), at(3), stride(bw), dt, at(4), at(5), 1, at(6), at(7),
                                  at(8), stride(xw), at(9), stride(bw), at(10), (int32_t*)at(11), at(12), n, pick(toks),
                                  pick(toks), H, G, N, P, (int)rnd(2), at(13), st);
            break;
        default: {
            const int32_t K = pick(toks);
            const size_t need = kda_verify_drafts_workspace_bytes(n, K, T);
            const size_t have = rnd(8) ? need : need / 2;
            kda_verify_drafts(at(1), rnd(2) ? at(2) : nullptr, dt, (int32_t*)at(3), rnd(2) ? (int32_t*)at(4) : nullptr, at(5),
                              at(6), n, K, T, (int32_t*)at(7), (int32_t*)at(8), ws(have), have, st);
        }
        }
    }
    CHECK(launched > 20000);
    if (fails) return 1;
    printf("%ld launches, all checks passed\n", launched);
    return 0;
}
