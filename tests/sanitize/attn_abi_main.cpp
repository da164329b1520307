// Sanitizer driver for the host code of kda_attn.h and kda_pages.h
// (gated_delta_rule_amd/csrc/kda_attn_abi.hip compiled as plain C++ with g++
// and -fsanitize=address,undefined by tests/test_attn_sanitizers.py; CPU only).
// The kernel launchers are replaced by stubs that check what they are asked to
// launch: every array of a plan lies within the workspace of the call, no
// launch has 2^32 threads, blocks cover all rows, pieces and parts are at least
// one.  Sizes are drawn from small, odd and extreme values, so that the
// arithmetic of the validation runs at its limits.  The pointers are fake
// device addresses that are never dereferenced.
#include <stdint.h>
#include <stdio.h>

#include "kda_attn.h"
#include "kda_attn_launch.h"
#include "kda_pages.h"

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

uint64_t seed = 999;
uint32_t rnd(uint32_t n) {
    seed = seed * 6364136223846793005ull + 1442695040888963407ull;
    return (uint32_t)(seed >> 33) % n;
}
template <typename T, int N>
T pick(const T (&a)[N]) {
    return a[rnd(N)];
}

// Blocks of `block` rows, `per` rows to a token, cover every sequence.
void blocks(const kda::AttnParams& p, big slots, big per, big block) {
    CHECK(p.rows == (p.cu ? p.T : (int64_t)p.n_seqs * p.T) && p.H == p.G * p.hpg);
    CHECK(slots == (p.cu ? (big)p.rows * per / block + p.n_seqs : (big)p.n_seqs * cdiv((big)p.T * per, block)));
    CHECK((big)p.T * per + block < ((big)1 << 31));   // rows are counted in 32 bits
}
void forward(const kda::AttnParams& p, bool bf16) {
    const big block = bf16 ? kda::kAttnBlockBf16 : kda::kAttnBlockF32, units = (big)p.slots * p.G;
    blocks(p, p.slots, p.hpg, block);
    CHECK(p.splits >= 1);
    if (bf16) {
        CHECK(p.splits == 1);
        if (p.workgroups > 0) {
            CHECK(p.lengths && p.workgroups % 8 == 0 && units > 0);
            const big info = (2 * units + 3) / 4 * 4 * 4;
            in_ws(p.part, info + 2 * (big)p.workgroups * block * (p.D + 4) * 4);
            CHECK(((uintptr_t)p.part + (uintptr_t)info) % 16 == 0);
            threads(p.workgroups, 256);
            threads(units * block / 4, 256);
        } else {
            threads(units, 256);
        }
    } else {
        threads(units * p.splits, 256);
        if (p.splits > 1) {
            in_ws(p.part, units * p.splits * block * (p.D + 2) * 4);
            threads(units * block / 4, 256);
        }
    }
    ++launched;
}
}  // namespace

namespace kda {
hipError_t launch_attn_fwd_f32(const AttnParams& p, hipStream_t) {
    forward(p, false);
    return hipSuccess;
}
hipError_t launch_attn_fwd_bf16(const AttnParams& p, hipStream_t) {
    forward(p, true);
    return hipSuccess;
}
hipError_t launch_attn_step(const AttnParams& p, bool bf16, int32_t max_rows, hipStream_t) {
    const big units = (big)p.n_seqs * p.G;
    CHECK(max_rows >= 1 && max_rows <= kAttnStepRows && max_rows == p.T * p.hpg && p.lengths);
    CHECK(p.workgroups == (bf16 || p.D == 64 ? 512 : 256));
    const big info = (2 * units + 3) / 4 * 4 * 4;
    in_ws(p.part, info + (p.workgroups + units) * step_row_tiles(max_rows) * 16 * (p.D + 4) * 4);
    CHECK(((uintptr_t)p.part + (uintptr_t)info) % 16 == 0);
    threads(p.workgroups, 256);
    threads(units * max_rows, 256);   // joining: at most a workgroup of 1024 per row where there are few
    CHECK(p.workgroups / units < 64 || units * max_rows * 1024 < ((big)1 << 32));
    ++launched;
    return hipSuccess;
}
static void backward(const AttnBwdParams& a, bool bf16) {
    const AttnParams& p = a.f;
    const big block = bf16 ? kAttnBlockBf16 : kAttnBwdBlockF32;
    blocks(p, p.slots, p.hpg, block);
    blocks(p, a.key_slots, 1, block);
    CHECK(a.parts >= 1);
    in_ws(a.delta, (big)p.rows * p.H * 4);
    threads((big)p.slots * p.G, 256);
    threads((big)a.key_slots * p.G * a.parts, 256);
    if (a.parts > 1) {
        in_ws(a.part, (big)a.parts * p.rows * p.G * 2 * p.D * 4);
        CHECK((uintptr_t)a.part % 16 == 0);
        threads(cdiv((big)p.rows * p.G * p.D / 2, 256), 256);
    }
    ++launched;
}
hipError_t launch_attn_bwd_f32(const AttnBwdParams& a, hipStream_t) {
    backward(a, false);
    return hipSuccess;
}
hipError_t launch_attn_bwd_bf16(const AttnBwdParams& a, hipStream_t) {
    backward(a, true);
    return hipSuccess;
}
hipError_t launch_kv_append(const AppendParams& p, bool bf16, hipStream_t) {
    threads(cdiv((big)p.rows * p.G * p.D / (bf16 ? 8 : 4), 256), 256);
    CHECK(p.page_shift >= 4 && p.page_shift <= 8);
    ++launched;
    return hipSuccess;
}
static void pages(const PagesParams& p) {
    CHECK(p.page_shift >= 4 && p.page_shift <= 8 && (big)p.n_slots * p.max_pages < ((big)1 << 31));
    CHECK(((big)p.max_pages << p.page_shift) < ((big)1 << 31));
    for (int t = 0; t < p.data.n; ++t) CHECK(p.data.bytes[t] % 16 == 0 && (p.n_pages < 2 || p.data.stride[t] >= p.data.bytes[t]));
    ++launched;
}
hipError_t launch_kv_resize(const PagesParams& p, hipStream_t) {
    pages(p);
    return hipSuccess;
}
hipError_t launch_kv_fork(const PagesParams& p, hipStream_t) {
    pages(p);
    in_ws(p.ws, (((big)p.n_slots + 3) / 4 * 4 + (big)p.n * 5 + (big)p.n * p.max_pages) * 4);
    threads((big)p.n * (cdiv(p.max_pages, 256) + 64), 256);
    return hipSuccess;
}
hipError_t launch_kv_compact(const PagesParams& p, hipStream_t) {
    pages(p);
    in_ws(p.ws, 16 + 12 * (big)p.n_pages);
    return hipSuccess;
}
}  // namespace kda

int main() {
    const uintptr_t base = (uintptr_t)1 << 52, gap = (uintptr_t)1 << 56;
    auto at = [&](int i) { return (void*)(base + (uintptr_t)i * gap); };
    const int32_t heads[] = {1, 2, 3, 8, 32, 96, 1000, 16384, 65536}, groups[] = {1, 2, 3, 8, 96, 65536}, dims[] = {64, 128, 96};
    const int32_t seqs[] = {0, 1, 2, 5, 64, 1000, 65536, INT32_MAX};
    const int64_t lens[] = {0, 1, 2, 5, 63, 64, 65, 1000, 4097, 1 << 20, (int64_t)1 << 30, (int64_t)1 << 36, INT64_MAX};
    const int32_t page[] = {16, 32, 64, 128, 256, 17}, many[] = {0, 1, 3, 100, 5000, 1 << 20, INT32_MAX};
    long refused = 0;
    for (int i = 0; i < 200000; ++i) {
        const int32_t G = pick(groups), H = rnd(3) ? G * (1 + (int32_t)rnd(8)) : pick(heads), D = rnd(9) ? dims[rnd(2)] : pick(dims);
        const int32_t n = pick(seqs), pg = rnd(9) ? page[rnd(5)] : pick(page), mp = pick(many), np = pick(many);
        const int64_t T = pick(lens), HD = (int64_t)H * D, GD = (int64_t)G * D, stride = HD + 2 * GD;
        const int dt = rnd(20) ? (int)rnd(2) : 2;
        const bool packed = rnd(2);
        const int32_t* cu = packed ? (const int32_t*)at(20) : nullptr;
        ws_lo = (uintptr_t)at(30);
        auto q = [&](int k) { return at(k); };
        size_t bytes = kda_attn_bwd_workspace_bytes(dt, n, T, H, G, D, packed);
        ws_hi = ws_lo + bytes;
        int rc = kda_attn_fwd(q(1), stride, q(2), stride, q(3), stride, dt, cu, n, T, H, G, D, 0.1f, 1, q(4), (float*)q(5), nullptr);
        refused += rc != KDA_OK;
        rc = kda_attn_bwd(q(1), stride, q(2), stride, q(3), stride, dt, cu, n, T, H, G, D, 0.1f, 0, q(4), (const float*)q(5), q(6), q(7), stride,
                          q(8), stride, q(9), stride, (void*)ws_lo, bytes, nullptr);
        refused += rc != KDA_OK;
        CHECK(rc != KDA_ERR_WORKSPACE);
        bytes = kda_attn_paged_workspace_bytes(dt, n, T, H, G, D, pg, mp, packed);
        ws_hi = ws_lo + bytes;
        rc = kda_attn_paged_fwd(q(1), stride, dt, q(2), q(3), GD * pg, np, pg, (const int32_t*)q(10), mp, (const int32_t*)q(11), cu, n, T, H, G,
                                D, 0.1f, q(4), (float*)q(5), (void*)ws_lo, bytes, nullptr);
        refused += rc != KDA_OK;
        CHECK(rc != KDA_ERR_WORKSPACE);
        rc = kda_kv_append(q(1), stride, q(2), stride, dt, q(3), q(4), GD * pg, np, pg, (const int32_t*)q(10), mp, (const int32_t*)q(11), cu, n, T,
                           G, D, nullptr);
        refused += rc != KDA_OK;
        int32_t* ints[8];
        for (int k = 0; k < 8; ++k) ints[k] = (int32_t*)at(10 + k);
        rc = kda_kv_resize(ints[0], ints[1], ints[2], ints[3], rnd(2) ? ints[4] : nullptr, n, mp, np, pg, nullptr);
        refused += rc != KDA_OK;
        void* data[17];
        int64_t size[17], step[17];
        const int32_t tensors = (int32_t)rnd(18);
        for (int k = 0; k < 17; ++k) {
            data[k] = (void*)(base + (uintptr_t)(40 + k) * gap);
            size[k] = 16 * (1 + rnd(100000));
            step[k] = size[k] + 16 * rnd(3);
        }
        const int32_t pairs = pick(seqs);
        bytes = kda_kv_fork_workspace_bytes(pairs, n, mp);
        ws_hi = ws_lo + bytes;
        rc = kda_kv_fork(ints[0], ints[1], ints[2], ints[3], ints[4], ints[5], pairs, n, mp, np, pg, data, size, step, tensors, (void*)ws_lo, bytes,
                         nullptr);
        refused += rc != KDA_OK;
        bytes = kda_kv_compact_workspace_bytes(np);
        ws_hi = ws_lo + bytes;
        const bool in_place = rnd(2);
        rc = kda_kv_compact(ints[0], ints[1], ints[2], in_place ? ints[0] : ints[3], in_place ? ints[2] : ints[4], ints[5], n, mp, np, pg, data, size,
                            step, tensors, (void*)ws_lo, bytes, nullptr);
        refused += rc != KDA_OK;
    }
    if (fails || launched < 100000 || refused < 100000) {
        fprintf(stderr, "%d checks failed, %ld launches, %ld refusals\n", fails, launched, refused);
        return 1;
    }
    printf("%ld launches, %ld refusals: all checks passed\n", launched, refused);
    return 0;
}
