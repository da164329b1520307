// Sanitizer driver for the backward pass's workspaces between one group of
// heads at a time and all of them (kda_ssm_chunk_bwd): with the launch stubs
// of ssm_abi_main.cpp, which check that every array of a launch lies within
// the call's workspace.  The number of groups that a workspace holds rarely
// divides G, so that the last pass has fewer groups than the others: its
// arrays have to fit, too, whatever fewer heads would let a plan of their own
// choose (segments where the others need none, more blocks of heads).
#define main ssm_abi_driver
#include "ssm_abi_main.cpp"
#undef main

int main() {
    (void)&ssm_abi_driver;
    auto at = [](int i) { return (float*)((uintptr_t)(i + 1) << 55); };
    const int64_t lens[] = {64, 192, 320, 512, 640, 2000, 8000};
    const int32_t per_group[] = {1, 2, 3, 5, 16, 32, 64};
    const int32_t seqs[] = {1, 2, 3, 16, 100};
    long rests = 0;
    for (int i = 0; i < 40000; ++i) {
        const int dt = (int)rnd(2);
        const int32_t G = 3 + (int32_t)rnd(7), hpg = pick(per_group), H = G * hpg, N = rnd(2) ? 64 : 128, P = rnd(2) ? 64 : 128;
        const int32_t n = pick(seqs);
        const int64_t T = pick(lens);
        const int32_t* cu = rnd(2) ? (const int32_t*)at(30) : nullptr;
        const int64_t xw = (int64_t)H * P, bw = (int64_t)G * N;
        const int32_t g = 1 + (int32_t)rnd(G);
        auto bytes = [&](int32_t k) { return kda_ssm_chunk_bwd_workspace_bytes(dt, n, T, H, G, N, P, cu != nullptr, k); };
        const size_t have = bytes(g) + (rnd(2) ? 0 : rnd(4096));
        ws_lo = (uintptr_t)at(40);
        ws_hi = ws_lo + have;
        const int rc = kda_ssm_chunk_bwd(at(1), xw, at(2), bw, at(3), bw, dt, at(4), at(5), 1, at(6), at(7), rnd(2) ? at(8) : nullptr, cu, n,
                                         T, H, G, N, P, at(9), rnd(2) ? at(10) : nullptr, at(11), xw, at(12), bw, at(13), bw, at(14),
                                         at(15), at(16), at(17), rnd(2) ? at(18) : nullptr, (void*)ws_lo, have, nullptr);
        CHECK(rc == KDA_OK);
        int32_t fits = G;
        while (fits > 1 && bytes(fits) > have) --fits;
        rests += rc == KDA_OK && G % fits != 0;
    }
    CHECK(rests > 10000);
    if (fails) {
        fprintf(stderr, "%d checks failed\n", fails);
        return 1;
    }
    printf("%ld launches, %ld calls with a smaller last pass, all checks passed\n", launched, rests);
    return 0;
}
