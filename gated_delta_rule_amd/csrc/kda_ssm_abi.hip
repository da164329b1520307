// C ABI of the state space scan, its short convolution (include/kda_ssm.h)
// and the draft verification (include/kda_spec.h): argument validation and
// launch planning.  Everything here runs on the host; nothing is enqueued
// unless every check passes.
#include <stdint.h>

#include "../../include/kda_spec.h"
#include "../../include/kda_ssm.h"
#include "kda_host.h"
#include "kda_ssm_launch.h"

namespace {

using namespace kda::host;

constexpr int64_t kMaxWide = kMaxWorkgroups / 2;    // of 512
constexpr int32_t kMaxTokens = 64;        // tokens per request in the step forms
constexpr int64_t kScanUnits = 256;       // compute units
constexpr int64_t kScanFill = 2 * kScanUnits;   // chains that fill them
constexpr int64_t kScanLongSeg = 512, kScanMinSeg = 128, kScanMinSegF32 = 64;   // see scan_plan
constexpr int64_t kScanMinCut = 4;        // segments from which two passes are shorter than one chain
constexpr int64_t kScanAlign = 64;
constexpr int64_t kVerifyFill = 2048;     // workgroups of the verification (512 to 2048: the same time)
// Workgroups of the gradient kernel that fill the GPU (its LDS leaves room for
// one per compute unit): 256 against 512 is 90 / 103 us for a backward pass of
// 1024 tokens of 64 heads, 432 / 445 for 2 x 4096.
constexpr int64_t kGradFill = 256;

// A row stride: at least the row, whole 16-byte pieces, small enough for
// 32-bit offsets within a chunk.
int check_stride(int64_t stride, int64_t width, int64_t es) {
    if (stride < width) return KDA_ERR_BAD_SHAPE;
    if (stride > KDA_SSM_MAX_STRIDE) return KDA_ERR_TOO_LARGE;
    return (stride * es) % 16 == 0 ? KDA_OK : KDA_ERR_MISALIGNED;
}

// Token rows of a batch, bounded so that no product of sizes below can wrap.
constexpr int64_t kMaxChain = (int64_t)1 << 30;   // tokens of a scan's sequence, counted in 32 bits with room for whole chunks
constexpr int64_t kMaxRows = (int64_t)1 << 36, kMaxState = (int64_t)1 << 56;
int count_rows(bool varlen, int32_t n_seqs, int64_t T, int64_t* rows) {
    if (T > kMaxRows) return KDA_ERR_TOO_LARGE;
    if (varlen) *rows = T;
    else if (!mul_ok((int64_t)n_seqs, T, rows)) return KDA_ERR_TOO_LARGE;
    return *rows <= kMaxRows ? KDA_OK : KDA_ERR_TOO_LARGE;
}

int conv_shape(int in_dtype, int32_t n_seqs, int64_t T, int32_t channels, int32_t width) {
    if (!dtype_ok(in_dtype)) return KDA_ERR_BAD_DTYPE;
    if (n_seqs < 0 || T < 0 || channels < 8 || channels % 8 != 0 || width < 2 || width > 4)
        return KDA_ERR_BAD_SHAPE;
    return channels <= KDA_SSM_MAX_STRIDE ? KDA_OK : KDA_ERR_TOO_LARGE;
}

int scan_shape(int in_dtype, int32_t n_seqs, int64_t T, int32_t H, int32_t G, int32_t N, int32_t P) {
    if (!dtype_ok(in_dtype)) return KDA_ERR_BAD_DTYPE;
    if (n_seqs < 0 || T < 0 || H < 1 || G < 1 || H % G != 0 || (N != 64 && N != 128) ||
        (P != 64 && P != 128))
        return KDA_ERR_BAD_SHAPE;
    if (H > KDA_MAX_HEADS || (int64_t)H * P > KDA_SSM_MAX_STRIDE || T > kMaxChain) return KDA_ERR_TOO_LARGE;
    return (int64_t)n_seqs * H <= kMaxState / ((int64_t)N * P) ? KDA_OK : KDA_ERR_TOO_LARGE;
}

// Workgroups per chain set: two heads of 64 of one group, or one of 128.
int64_t scan_blocks(int32_t H, int32_t G, int32_t P) { return (int64_t)G * ceil_div(H / G, 128 / P); }

// How sequences are cut into segments.  A chain alone on a compute unit takes
// 4.3 us per chunk, two take 6.3 us together, and a segment costs its state's
// traffic (two reads and writes of N x P floats per head): long segments for
// two chains per unit, shorter ones for one, none below 128 tokens.  Measured
// (64 heads of 64, one group, N 128, bf16, one sequence, cut against one
// chain): 512 tokens 32.4 against 38.4 us, 1024 36 / 71, 2048 49 / 138, 4096
// 71 / 270; segments of 64 tokens at 256 tokens 25.7 / 20.8.  Other lengths
// (against 48, 35 and 117 us at that time): segments of 128 at 2048 tokens 54
// us, of 256 at 1024 tokens 42, of 1024 at 8192 tokens 122.  A packed batch is
// planned by the number of its sequences, whatever their lengths: one long
// one beside so many short ones that there are 512 chains runs as one chain.
// Float32 chains take four times as long per token, so their
// segments go down to 64 (16 heads of 64, N 128: 256 tokens 26 against 37 us
// with 128, 1024 tokens 32 against 40; 16 of 128, N 64: 20.5 against 24 and 29
// against 31, but 4 x 256 tokens 27 against 25).
//
// Three segments leave the two passes as long as one chain.  Cut / whole, us:
// bf16 300 tokens of 64 heads 29 / 26, 6 x 400 of 32 heads 54 / 36, 6 x 4096 of
// 64 heads 325 / 280, float32 6 x 2048 of 64 heads 373 / 281; four, bf16 400 tokens of 64 heads 31 / 34, 4 x 2048 122 / 140,
// float32 2 x 512 48 / 74 (but 4 x 400 of 16 heads of 128 27 / 23).
//
// The backward pass's two directions fill the GPU twice as far, so it cuts
// from four segments of twice the least length, or five.  Cut / whole, us: three
// segments, bf16, 3 x 512 tokens of 32 heads of 64 99 / 76, 3 x 4096 of 64 heads
// 644 / 624, float32 3 x 1024 of 32 heads 252 / 220; four short ones, bf16 512
// tokens of 64 heads 71 / 64, float32 256 tokens 70 / 62; four longer ones, bf16
// 1024 tokens 88 / 89, 1536 134 / 142, 2 x 4096 409 / 420 (but 2 x 2048 228 /
// 216), float32 512 tokens 90 / 91, 1024 131 / 148; five and more, bf16 640
// tokens of 16 heads 53 / 58, 4096 of 64 heads 229 / 283, float32 300 tokens of
// 16 heads 54 / 56, 2048 of 32 heads 132 / 224.
struct ScanPlan {
    bool cut;
    int64_t seg_len, slots;
};
// `dirs` directions (the backward pass: two) run side by side.
ScanPlan scan_plan(bool bf16_in, int32_t n_seqs, int64_t T, int64_t blocks, bool varlen, int64_t dirs) {
    const int64_t rows = varlen ? T : n_seqs * T;
    const ScanPlan whole{false, T > 0 ? T : 1, n_seqs};
    if (n_seqs * blocks * dirs >= kScanFill) return whole;
    const int64_t work = rows * blocks * dirs;
    const int64_t least = bf16_in ? kScanMinSeg : kScanMinSegF32;
    int64_t len = ceil_div(work, kScanUnits);
    len = len < least ? least : len > kScanLongSeg ? kScanLongSeg : len;
    if (len < ceil_div(work, kScanFill)) len = ceil_div(work, kScanFill);
    const int64_t segs = ceil_div(T, len);
    if (segs < (dirs == 1 || len >= 2 * least ? kScanMinCut : kScanMinCut + 1)) return whole;
    if (!varlen) len = ceil_div(T, segs);
    len = ceil_div(len, kScanAlign) * kScanAlign;
    return ScanPlan{true, len, varlen ? T / len + n_seqs : n_seqs * ceil_div(T, len)};
}

// Segments' states and decays.
size_t scan_bytes(const ScanPlan& s, int32_t H, int32_t N, int32_t P) {
    return s.cut ? (size_t)s.slots * H * ((size_t)N * P + 1) * 4 : 0;
}

// Backward: arrays (offsets in floats) for `groups` groups of heads at a time.
struct BwdPlan {
    ScanPlan scan;
    int64_t slots;           // chunks
    int32_t heads_per_block, blocks;
    int64_t states, dstates, seg[2], seg_decay[2], part, sums, total;   // seg: of each direction
};
bool bwd_plan(int in_dtype, int32_t n_seqs, int64_t T, int64_t rows, int32_t H, int32_t G, int32_t N,
              int32_t P, bool varlen, int32_t groups, BwdPlan* b) {
    const int64_t len = kda::ssm_chunk_tokens(in_dtype == KDA_BF16);
    const int64_t hpg = H / G, heads = groups * hpg;
    b->slots = varlen ? rows / len + n_seqs : n_seqs * ceil_div(T, len);
    b->scan = scan_plan(in_dtype == KDA_BF16, n_seqs, T, scan_blocks((int32_t)heads, groups, P), varlen, 2);
    // as many heads of a group in one workgroup (fewer partial sums) as leave
    // enough workgroups to fill the GPU
    const int64_t want = ceil_div(kGradFill, b->slots * groups > 0 ? b->slots * groups : 1);
    b->heads_per_block = (int32_t)(want >= hpg ? 1 : hpg / want);
    b->blocks = (int32_t)ceil_div(hpg, b->heads_per_block);
    int64_t st = 0, seg = 0, part = 0;
    if (!mul_ok(b->slots * heads, (int64_t)N * P, &st) || !mul_ok(b->scan.slots * heads, (int64_t)N * P, &seg) ||
        !mul_ok(2 * (int64_t)b->blocks * groups * N, rows, &part))
        return false;
    if (st > INT64_MAX / 64 || seg > INT64_MAX / 64 || part > INT64_MAX / 64) return false;
    if (!b->scan.cut) seg = 0;
    if (b->blocks == 1) part = 0;
    const int64_t four = 3;   // every array starts on 16 bytes
    b->states = 0;
    b->dstates = b->states + st;
    b->seg[0] = b->dstates + st;
    b->seg[1] = b->seg[0] + seg;
    b->part = b->seg[1] + seg;
    b->seg_decay[0] = b->part + part;
    b->seg_decay[1] = b->seg_decay[0] + (b->scan.cut ? b->scan.slots * heads : 0);
    b->sums = (b->seg_decay[1] + (b->scan.cut ? b->scan.slots * heads : 0) + four) & ~four;
    b->total = b->sums + ((b->slots * heads * 3 + 4 + four) & ~four);
    return b->total <= INT64_MAX / 8;
}

}  // namespace

extern "C" {

int kda_ssm_conv_fwd(const void* x, int64_t x_stride, int in_dtype, const float* w,
                     const float* bias, float* cache, const int32_t* cu_seqlens, int32_t n_seqs,
                     int64_t T, int32_t channels, int32_t width, int activation, void* y,
                     hipStream_t stream) {
    int rc = conv_shape(in_dtype, n_seqs, T, channels, width);
    if (rc) return rc;
    int64_t rows = 0;
    if ((rc = count_rows(cu_seqlens != nullptr, n_seqs, T, &rows))) return rc;
    if (n_seqs == 0) return KDA_OK;
    if (ceil_div(rows, 32) * ceil_div(channels, 256) > kMaxWorkgroups ||
        ceil_div((int64_t)n_seqs * channels, 256) > kMaxWorkgroups)
        return KDA_ERR_TOO_LARGE;
    if (rows > 0 && (!x || !w || !y)) return KDA_ERR_NULL_POINTER;
    const int64_t es = elem_size(in_dtype);
    if (rows > 0 && (rc = check_stride(x_stride, channels, es))) return rc;
    if (!aligned(x, 16) || !aligned(w, 16) || !aligned(y, 16) || !aligned(cache, 16) ||
        !aligned(bias, 4) || !aligned(cu_seqlens, 4))
        return KDA_ERR_MISALIGNED;
    const Span ry = span(y, rows * channels * es);
    const Span rc_ = span(cache, (int64_t)n_seqs * (width - 1) * channels * 4);
    const Span ins[] = {rows_span(x, rows, x_stride, channels, es), span(w, (int64_t)channels * width * 4),
                        span(bias, (int64_t)channels * 4),
                        span(cu_seqlens, ((int64_t)n_seqs + 1) * 4)};
    for (const Span& r : ins)
        if (overlaps(ry, r) || overlaps(rc_, r)) return KDA_ERR_ALIASING;
    if (overlaps(ry, rc_)) return KDA_ERR_ALIASING;
    kda::ConvParams p{};
    p.x = x;
    p.w = w;
    p.bias = bias;
    p.cache = cache;
    p.cu = cu_seqlens;
    p.y = y;
    p.x_stride = x_stride;
    p.rows = rows;
    p.T = T;
    p.n_seqs = n_seqs;
    p.channels = channels;
    p.width = width;
    p.activation = activation != 0;
    return kda::launch_conv_fwd(p, in_dtype == KDA_BF16, stream) == hipSuccess ? KDA_OK : KDA_ERR_HIP;
}

int kda_ssm_conv_step(const void* x, int64_t x_stride, int in_dtype, const float* w,
                      const float* bias, float* cache, const void* rx, int64_t rx_stride,
                      const int32_t* n_replay, int32_t B, int32_t T, int32_t Tr, int32_t channels,
                      int32_t width, int activation, int commit, void* y, hipStream_t stream) {
    int rc = conv_shape(in_dtype, B, T, channels, width);
    if (rc) return rc;
    if (T > kMaxTokens || Tr < 0 || Tr > kMaxTokens) return KDA_ERR_BAD_SHAPE;
    if (B == 0) return KDA_OK;
    if (ceil_div((int64_t)B * (channels / 4), 64) > kMaxWorkgroups) return KDA_ERR_TOO_LARGE;
    if (!cache || (T > 0 && (!x || !w || !y)) || (Tr > 0 && !rx)) return KDA_ERR_NULL_POINTER;
    if (!w) return KDA_ERR_NULL_POINTER;
    const int64_t es = elem_size(in_dtype);
    if (T > 0 && (rc = check_stride(x_stride, channels, es))) return rc;
    if (Tr > 0 && (rc = check_stride(rx_stride, channels, es))) return rc;
    if (!aligned(cache, 16) || !aligned(w, 16) || !aligned(bias, 4) || !aligned(n_replay, 4) ||
        (T > 0 && (!aligned(x, 16) || !aligned(y, 16))) || (Tr > 0 && !aligned(rx, 16)))
        return KDA_ERR_MISALIGNED;
    const int64_t rows = (int64_t)B * T;
    const Span ry = span(y, rows * channels * es);
    const Span rc_ = span(cache, (int64_t)B * (width - 1) * channels * 4);
    const Span ins[] = {rows_span(x, rows, x_stride, channels, es),
                        rows_span(rx, (int64_t)B * Tr, rx_stride, channels, es),
                        span(w, (int64_t)channels * width * 4), span(bias, (int64_t)channels * 4),
                        span(n_replay, (int64_t)B * 4)};
    for (const Span& r : ins)
        if (overlaps(ry, r) || overlaps(rc_, r)) return KDA_ERR_ALIASING;
    if (overlaps(ry, rc_)) return KDA_ERR_ALIASING;
    kda::ConvParams p{};
    p.x = x;
    p.rx = rx;
    p.w = w;
    p.bias = bias;
    p.cache = cache;
    p.n_replay = Tr > 0 ? n_replay : nullptr;
    p.y = y;
    p.x_stride = x_stride;
    p.rx_stride = rx_stride;
    p.rows = rows;
    p.T = T;
    p.n_seqs = B;
    p.channels = channels;
    p.width = width;
    p.activation = activation != 0;
    p.Tr = Tr;
    p.commit = commit != 0;
    return kda::launch_conv_step(p, in_dtype == KDA_BF16, stream) == hipSuccess ? KDA_OK : KDA_ERR_HIP;
}

size_t kda_ssm_conv_bwd_workspace_bytes(int64_t rows, int32_t channels, int32_t width) {
    if (rows < 0 || rows > kMaxRows || conv_shape(KDA_BF16, 0, 0, channels, width)) return 0;
    const int64_t parts = kda::conv_bwd_parts(rows, channels);
    int64_t n = 0;
    if (!mul_ok(parts, (int64_t)(width + 1) * channels * 4, &n)) return 0;
    return (size_t)(n < 16 ? 16 : n);
}

int kda_ssm_conv_bwd_fresh(const void* x, int64_t x_stride, int in_dtype, const float* w,
                           const float* bias, const float* cache, const int32_t* cu_seqlens,
                           int32_t n_seqs, int64_t T, int32_t channels, int32_t width, int activation,
                           const void* grad_y, int64_t grad_y_stride, void* grad_x, float* grad_w,
                           float* grad_bias, float* grad_cache, void* workspace, size_t workspace_bytes,
                           hipStream_t stream, int fresh) {
    int rc = conv_shape(in_dtype, n_seqs, T, channels, width);
    if (rc) return rc;
    int64_t rows = 0;
    if ((rc = count_rows(cu_seqlens != nullptr, n_seqs, T, &rows))) return rc;
    if (n_seqs == 0) rows = 0;
    if (ceil_div(rows, 32) * ceil_div(channels, 256) > kMaxWorkgroups ||
        ceil_div((int64_t)n_seqs * channels, 256) > kMaxWorkgroups)
        return KDA_ERR_TOO_LARGE;
    if (!w || !grad_w || (rows > 0 && (!x || !grad_y || !grad_x))) return KDA_ERR_NULL_POINTER;
    const int64_t es = elem_size(in_dtype);
    if (rows > 0 && ((rc = check_stride(x_stride, channels, es)) ||
                     (rc = check_stride(grad_y_stride, channels, es))))
        return rc;
    if (!aligned(x, 16) || !aligned(w, 16) || !aligned(cache, 16) || !aligned(grad_y, 16) ||
        !aligned(grad_x, 16) || !aligned(grad_cache, 16) || !aligned(workspace, 16) ||
        !aligned(bias, 4) || !aligned(cu_seqlens, 4) || !aligned(grad_w, 4) || !aligned(grad_bias, 4))
        return KDA_ERR_MISALIGNED;
    const size_t need = kda_ssm_conv_bwd_workspace_bytes(rows, channels, width);
    if (rows > 0 && (!workspace || workspace_bytes < need)) return KDA_ERR_WORKSPACE;
    const int64_t cache_bytes = (int64_t)n_seqs * (width - 1) * channels * 4;
    const Span ins[] = {rows_span(x, rows, x_stride, channels, es),
                        rows_span(grad_y, rows, grad_y_stride, channels, es),
                        span(w, (int64_t)channels * width * 4), span(bias, (int64_t)channels * 4),
                        span(cache, cache_bytes), span(cu_seqlens, ((int64_t)n_seqs + 1) * 4)};
    const Span outs[] = {span(grad_x, rows * channels * es), span(grad_w, (int64_t)channels * width * 4),
                         span(grad_bias, (int64_t)channels * 4), span(grad_cache, cache_bytes),
                         span(workspace, rows > 0 ? (int64_t)need : 0)};
    for (int a = 0; a < 5; ++a) {
        for (const Span& r : ins)
            if (overlaps(outs[a], r)) return KDA_ERR_ALIASING;
        for (int b = a + 1; b < 5; ++b)
            if (overlaps(outs[a], outs[b])) return KDA_ERR_ALIASING;
    }
    kda::ConvBwdParams q{};
    q.f.x = x;
    q.f.w = w;
    q.f.bias = bias;
    q.f.cache = const_cast<float*>(cache);   // read only here
    q.f.cu = cu_seqlens;
    q.f.x_stride = x_stride;
    q.f.rows = rows;
    q.f.T = T;
    q.f.n_seqs = n_seqs;
    q.f.channels = channels;
    q.f.width = width;
    q.f.activation = activation != 0;
    q.gy = grad_y;
    q.gx = grad_x;
    q.gw = grad_w;
    q.gbias = grad_bias;
    q.gcache = grad_cache;
    q.partial = (float*)workspace;
    q.gy_stride = grad_y_stride;
    q.rows_per_wave = (int32_t)kda::conv_rows_per_wave(rows, channels);
    q.zero_rest = cu_seqlens && (fresh & KDA_FRESH_X);
    return kda::launch_conv_bwd(q, in_dtype == KDA_BF16, stream) == hipSuccess ? KDA_OK : KDA_ERR_HIP;
}
int kda_ssm_conv_bwd(const void* x, int64_t x_stride, int in_dtype, const float* w,
                     const float* bias, const float* cache, const int32_t* cu_seqlens,
                     int32_t n_seqs, int64_t T, int32_t channels, int32_t width, int activation,
                     const void* grad_y, int64_t grad_y_stride, void* grad_x, float* grad_w,
                     float* grad_bias, float* grad_cache, void* workspace, size_t workspace_bytes,
                     hipStream_t stream) {
    return kda_ssm_conv_bwd_fresh(x, x_stride, in_dtype, w, bias, cache, cu_seqlens, n_seqs, T, channels, width,
                                  activation, grad_y, grad_y_stride, grad_x, grad_w, grad_bias, grad_cache,
                                  workspace, workspace_bytes, stream, 0);
}

size_t kda_ssm_chunk_fwd_workspace_bytes(int32_t n_seqs, int64_t T, int32_t H, int32_t G,
                                         int32_t N, int32_t P, int varlen) {
    if (scan_shape(KDA_BF16, n_seqs, T, H, G, N, P)) return 0;
    int64_t rows = 0;
    if (count_rows(varlen != 0, n_seqs, T, &rows)) return 0;
    size_t need = 0;   // of either type
    for (int bf16_in = 0; bf16_in < 2; ++bf16_in) {
        const size_t n = scan_bytes(scan_plan(bf16_in != 0, n_seqs, T, scan_blocks(H, G, P), varlen != 0, 1), H, N, P);
        if (n > need) need = n;
    }
    return need;
}

int kda_ssm_chunk_fwd(const void* x, int64_t x_stride, const void* B, int64_t B_stride,
                      const void* C, int64_t C_stride, int in_dtype, const float* dt,
                      const float* dt_bias, int softplus, const float* A, const float* D,
                      const float* S0, const int32_t* cu_seqlens, int32_t n_seqs, int64_t T,
                      int32_t H, int32_t G, int32_t N, int32_t P, void* y, float* S_T,
                      void* workspace, size_t workspace_bytes, hipStream_t stream) {
    int rc = scan_shape(in_dtype, n_seqs, T, H, G, N, P);
    if (rc) return rc;
    int64_t rows = 0;
    if ((rc = count_rows(cu_seqlens != nullptr, n_seqs, T, &rows))) return rc;
    if (n_seqs == 0) return KDA_OK;
    if ((int64_t)n_seqs * H > INT32_MAX) return KDA_ERR_TOO_LARGE;
    if (!A || (rows > 0 && (!x || !B || !C || !dt || !y))) return KDA_ERR_NULL_POINTER;
    const int64_t es = elem_size(in_dtype);
    if (rows > 0 && ((rc = check_stride(x_stride, (int64_t)H * P, es)) ||
                     (rc = check_stride(B_stride, (int64_t)G * N, es)) ||
                     (rc = check_stride(C_stride, (int64_t)G * N, es))))
        return rc;
    if (!aligned(x, 16) || !aligned(B, 16) || !aligned(C, 16) || !aligned(y, 16) || !aligned(S0, 16) ||
        !aligned(S_T, 16) || !aligned(dt, 4) || !aligned(dt_bias, 4) || !aligned(A, 4) ||
        !aligned(D, 4) || !aligned(cu_seqlens, 4))
        return KDA_ERR_MISALIGNED;
    const int64_t st_bytes = (int64_t)n_seqs * H * N * P * 4;
    const Span rs0 = span(S0, st_bytes), rst = span(S_T, st_bytes), ry = span(y, rows * H * P * es);
    const Span ins[] = {rows_span(x, rows, x_stride, (int64_t)H * P, es),
                        rows_span(B, rows, B_stride, (int64_t)G * N, es),
                        rows_span(C, rows, C_stride, (int64_t)G * N, es), span(dt, rows * H * 4),
                        span(dt_bias, (int64_t)H * 4), span(A, (int64_t)H * 4), span(D, (int64_t)H * 4),
                        span(cu_seqlens, ((int64_t)n_seqs + 1) * 4)};
    for (const Span& r : ins)
        if (overlaps(ry, r) || overlaps(rst, r)) return KDA_ERR_ALIASING;
    if (overlaps(ry, rs0) || overlaps(ry, rst)) return KDA_ERR_ALIASING;
    if (S0 != (const float*)S_T && overlaps(rs0, rst)) return KDA_ERR_ALIASING;

    ScanPlan s = scan_plan(in_dtype == KDA_BF16, n_seqs, T, scan_blocks(H, G, P), cu_seqlens != nullptr, 1);
    const size_t need = scan_bytes(s, H, N, P);
    if (s.cut && (!workspace || workspace_bytes < need))
        s = ScanPlan{false, T, n_seqs};
    if (s.cut) {
        if (!aligned(workspace, 16)) return KDA_ERR_MISALIGNED;
        const Span rw = span(workspace, (int64_t)need);
        for (const Span& r : ins)
            if (overlaps(rw, r)) return KDA_ERR_ALIASING;
        if (overlaps(rw, ry) || overlaps(rw, rs0) || overlaps(rw, rst)) return KDA_ERR_ALIASING;
    }
    if (s.slots * scan_blocks(H, G, P) > kMaxWide ||
        ceil_div((int64_t)n_seqs * H * N * P, 1024) > kMaxWorkgroups)
        return KDA_ERR_TOO_LARGE;
    kda::SsmScanParams p{};
    p.x = x;
    p.B = B;
    p.C = C;
    p.dt = dt;
    p.dt_bias = dt_bias;
    p.A = A;
    p.D = D;
    p.S0 = S0;
    p.cu = cu_seqlens;
    p.y = y;
    p.S_T = S_T;
    p.seg = s.cut ? (float*)workspace : nullptr;
    p.seg_decay = s.cut ? (float*)workspace + s.slots * H * N * P : nullptr;
    p.x_stride = x_stride;
    p.B_stride = B_stride;
    p.C_stride = C_stride;
    p.rows = rows;
    p.T = T;
    p.seg_len = s.seg_len;
    p.slots = s.slots;
    p.cut = s.cut;
    p.n_seqs = n_seqs;
    p.H = H;
    p.G = G;
    p.N = N;
    p.P = P;
    p.softplus = softplus != 0;
    p.g0 = 0;
    p.gn = G;
    return kda::launch_ssm_chunk_fwd(p, in_dtype == KDA_BF16, stream) == hipSuccess ? KDA_OK : KDA_ERR_HIP;
}

size_t kda_ssm_chunk_bwd_workspace_bytes(int in_dtype, int32_t n_seqs, int64_t T, int32_t H,
                                         int32_t G, int32_t N, int32_t P, int varlen,
                                         int32_t groups) {
    if (scan_shape(in_dtype, n_seqs, T, H, G, N, P) || groups < 1) return 0;
    int64_t rows = 0;
    if (count_rows(varlen != 0, n_seqs, T, &rows)) return 0;
    BwdPlan b;
    if (!bwd_plan(in_dtype, n_seqs, T, rows, H, G, N, P, varlen != 0, groups < G ? groups : G, &b)) return 0;
    return (size_t)b.total * 4;
}

int kda_ssm_chunk_bwd_fresh(const void* x, int64_t x_stride, const void* B, int64_t B_stride,
                            const void* C, int64_t C_stride, int in_dtype, const float* dt,
                            const float* dt_bias, int softplus, const float* A, const float* D,
                            const float* S0, const int32_t* cu_seqlens, int32_t n_seqs, int64_t T,
                            int32_t H, int32_t G, int32_t N, int32_t P, const void* grad_y,
                            const float* grad_S_T, void* grad_x, int64_t grad_x_stride, void* grad_B,
                            int64_t grad_B_stride, void* grad_C, int64_t grad_C_stride, float* grad_dt,
                            float* grad_A, float* grad_D, float* grad_dt_bias, float* grad_S0,
                            void* workspace, size_t workspace_bytes, hipStream_t stream, int fresh) {
    int rc = scan_shape(in_dtype, n_seqs, T, H, G, N, P);
    if (rc) return rc;
    int64_t rows = 0;
    if ((rc = count_rows(cu_seqlens != nullptr, n_seqs, T, &rows))) return rc;
    if (n_seqs == 0) rows = 0;
    if ((int64_t)n_seqs * H > INT32_MAX) return KDA_ERR_TOO_LARGE;
    if (!A || !grad_A || (rows > 0 && (!x || !B || !C || !dt || !grad_y || !grad_x || !grad_B || !grad_C || !grad_dt)))
        return KDA_ERR_NULL_POINTER;
    const bool varlen = cu_seqlens != nullptr;
    const int64_t es = elem_size(in_dtype), xw = (int64_t)H * P, bw = (int64_t)G * N;
    if (rows > 0 && ((rc = check_stride(x_stride, xw, es)) || (rc = check_stride(B_stride, bw, es)) ||
                     (rc = check_stride(C_stride, bw, es)) || (rc = check_stride(grad_x_stride, xw, es)) ||
                     (rc = check_stride(grad_B_stride, bw, es)) || (rc = check_stride(grad_C_stride, bw, es))))
        return rc;
    if (!aligned(x, 16) || !aligned(B, 16) || !aligned(C, 16) || !aligned(grad_y, 16) || !aligned(grad_x, 16) ||
        !aligned(grad_B, 16) || !aligned(grad_C, 16) || !aligned(S0, 16) || !aligned(grad_S_T, 16) ||
        !aligned(grad_S0, 16) || !aligned(workspace, 16) || !aligned(dt, 4) || !aligned(dt_bias, 4) ||
        !aligned(A, 4) || !aligned(D, 4) || !aligned(cu_seqlens, 4) || !aligned(grad_dt, 4) ||
        !aligned(grad_A, 4) || !aligned(grad_D, 4) || !aligned(grad_dt_bias, 4))
        return KDA_ERR_MISALIGNED;
    // as many groups at a time as the workspace holds
    BwdPlan b;
    int32_t groups = G;
    for (; groups >= 1; --groups) {
        if (!bwd_plan(in_dtype, n_seqs, T, rows, H, G, N, P, varlen, groups, &b)) {
            if (groups == 1) return KDA_ERR_TOO_LARGE;
            continue;
        }
        if ((size_t)b.total * 4 <= workspace_bytes) break;
    }
    if (!workspace || groups < 1) return KDA_ERR_WORKSPACE;
    const int64_t per = scan_blocks(groups * (H / G), groups, P);
    if (b.scan.slots * per > kMaxWide || b.slots * groups * b.blocks > kMaxWide ||
        ceil_div((int64_t)n_seqs * H * N * P, 1024) > kMaxWorkgroups ||
        ceil_div(rows * groups * N, 512) + groups * (int64_t)(H / G) + kda::kGradRest > kMaxWorkgroups)
        return KDA_ERR_TOO_LARGE;

    // outputs overlap nothing, except that grad_x, grad_B and grad_C may
    // share wider rows and grad_S0 may be grad_S_T
    const int64_t st_bytes = (int64_t)n_seqs * H * N * P * 4, hb = (int64_t)H * 4;
    const Span rgst = span(grad_S_T, st_bytes);
    const Span ins[] = {rows_span(x, rows, x_stride, xw, es), rows_span(B, rows, B_stride, bw, es),
                        rows_span(C, rows, C_stride, bw, es), span(dt, rows * H * 4), span(dt_bias, hb),
                        span(A, hb), span(D, hb), span(S0, st_bytes), span(grad_y, rows * xw * es),
                        span(cu_seqlens, ((int64_t)n_seqs + 1) * 4)};
    const Span outs[] = {rows_span(grad_x, rows, grad_x_stride, xw, es), rows_span(grad_B, rows, grad_B_stride, bw, es),
                         rows_span(grad_C, rows, grad_C_stride, bw, es), span(grad_dt, rows * H * 4),
                         span(grad_A, hb), span(grad_D, hb), span(grad_dt_bias, hb), span(workspace, b.total * 4),
                         span(grad_S0, st_bytes)};
    for (int i = 0; i < 9; ++i) {
        for (const Span& r : ins)
            if (overlaps(outs[i], r)) return KDA_ERR_ALIASING;
        if (!(i == 8 && grad_S0 == grad_S_T) && overlaps(outs[i], rgst)) return KDA_ERR_ALIASING;
        for (int j = i + 1; j < 9; ++j)
            if (i < 3 && j < 3 ? overlaps_rows(outs[i], outs[j]) : overlaps(outs[i], outs[j])) return KDA_ERR_ALIASING;
    }

    float* ws = (float*)workspace;
    const bool bf16_in = in_dtype == KDA_BF16;
    kda::SsmScanParams f{};
    f.x = x;
    f.B = B;
    f.C = C;
    f.dt = dt;
    f.dt_bias = dt_bias;
    f.A = A;
    f.D = D;
    f.S0 = S0;
    f.cu = cu_seqlens;
    f.x_stride = x_stride;
    f.B_stride = B_stride;
    f.C_stride = C_stride;
    f.rows = rows;
    f.T = T;
    f.n_seqs = n_seqs;
    f.H = H;
    f.G = G;
    f.N = N;
    f.P = P;
    f.softplus = softplus != 0;
    // One plan for all passes.  A last pass of fewer groups keeps the segments
    // and head blocks of the others, so that each of its arrays is a smaller
    // one in the same place: a plan of its own could need more than they do
    // (segments where `groups` groups fill the GPU without, more head blocks).
    f.cut = b.scan.cut;
    f.seg_len = b.scan.seg_len;
    f.slots = b.scan.slots;
    for (int32_t g0 = 0; g0 < G; g0 += groups) {
        const int32_t gn = G - g0 < groups ? G - g0 : groups;
        f.g0 = g0;
        f.gn = gn;
        if (n_seqs > 0) {
            kda::SsmScanDirs walks{{f, f}};
            for (int i = 0; b.scan.cut && i < 2; ++i) {
                walks.dir[i].seg = ws + b.seg[i];
                walks.dir[i].seg_decay = ws + b.seg_decay[i];
            }
            walks.dir[0].states = ws + b.states;   // S at every chunk's start
            kda::SsmScanParams& w = walks.dir[1];  // the state gradient at every chunk's end
            w.x = grad_y;
            w.x_stride = xw;
            w.B = C;
            w.B_stride = C_stride;
            w.S0 = grad_S_T;
            w.S_T = grad_S0;
            w.states = ws + b.dstates;
            if (kda::launch_ssm_walks(walks, bf16_in, stream) != hipSuccess) return KDA_ERR_HIP;
        }
        kda::SsmGradParams q{};
        q.f = f;
        q.gy = grad_y;
        q.states = ws + b.states;
        q.dstates = ws + b.dstates;
        q.gx = grad_x;
        q.gB = grad_B;
        q.gC = grad_C;
        q.gdt = grad_dt;
        q.gA = grad_A;
        q.gD = grad_D;
        q.gbias = grad_dt_bias;
        q.part = ws + b.part;
        q.sums = ws + b.sums;
        q.gx_stride = grad_x_stride;
        q.gB_stride = grad_B_stride;
        q.gC_stride = grad_C_stride;
        q.slots = n_seqs > 0 ? b.slots : 0;
        q.heads_per_block = b.heads_per_block;
        q.blocks = b.blocks;
        q.zero_rest = varlen && g0 == 0 ? fresh : 0;
        if (kda::launch_ssm_grad(q, bf16_in, stream) != hipSuccess) return KDA_ERR_HIP;
    }
    return KDA_OK;
}
int kda_ssm_chunk_bwd(const void* x, int64_t x_stride, const void* B, int64_t B_stride,
                      const void* C, int64_t C_stride, int in_dtype, const float* dt,
                      const float* dt_bias, int softplus, const float* A, const float* D,
                      const float* S0, const int32_t* cu_seqlens, int32_t n_seqs, int64_t T,
                      int32_t H, int32_t G, int32_t N, int32_t P, const void* grad_y,
                      const float* grad_S_T, void* grad_x, int64_t grad_x_stride, void* grad_B,
                      int64_t grad_B_stride, void* grad_C, int64_t grad_C_stride, float* grad_dt,
                      float* grad_A, float* grad_D, float* grad_dt_bias, float* grad_S0,
                      void* workspace, size_t workspace_bytes, hipStream_t stream) {
    return kda_ssm_chunk_bwd_fresh(x, x_stride, B, B_stride, C, C_stride, in_dtype, dt, dt_bias, softplus, A, D, S0,
                                   cu_seqlens, n_seqs, T, H, G, N, P, grad_y, grad_S_T, grad_x, grad_x_stride,
                                   grad_B, grad_B_stride, grad_C, grad_C_stride, grad_dt, grad_A, grad_D,
                                   grad_dt_bias, grad_S0, workspace, workspace_bytes, stream, 0);
}

int kda_ssm_recurrent_fwd(const void* x, int64_t x_stride, const void* Bm, int64_t B_stride,
                          const void* C, int64_t C_stride, int in_dtype, const float* dt,
                          const float* dt_bias, int softplus, const float* A, const float* D,
                          const void* rx, int64_t rx_stride, const void* rB, int64_t rB_stride,
                          const float* rdt, const int32_t* n_replay, float* S, int32_t B,
                          int32_t T, int32_t Tr, int32_t H, int32_t G, int32_t N, int32_t P,
                          int commit, void* y, hipStream_t stream) {
    int rc = scan_shape(in_dtype, B, T, H, G, N, P);
    if (rc) return rc;
    if (T > kMaxTokens || Tr < 0 || Tr > kMaxTokens) return KDA_ERR_BAD_SHAPE;
    if (B == 0) return KDA_OK;
    if ((int64_t)B * H > kMaxWorkgroups) return KDA_ERR_TOO_LARGE;
    if (!S || !A || (T > 0 && (!x || !Bm || !C || !dt || !y)) || (Tr > 0 && (!rx || !rB || !rdt)))
        return KDA_ERR_NULL_POINTER;
    const int64_t es = elem_size(in_dtype), xw = (int64_t)H * P, bw = (int64_t)G * N;
    if (T > 0 && ((rc = check_stride(x_stride, xw, es)) || (rc = check_stride(B_stride, bw, es)) ||
                  (rc = check_stride(C_stride, bw, es))))
        return rc;
    if (Tr > 0 && ((rc = check_stride(rx_stride, xw, es)) || (rc = check_stride(rB_stride, bw, es))))
        return rc;
    if (!aligned(S, 16) || !aligned(A, 4) || !aligned(D, 4) || !aligned(dt_bias, 4) || !aligned(n_replay, 4) ||
        (T > 0 && (!aligned(x, 16) || !aligned(Bm, 16) || !aligned(C, 16) || !aligned(dt, 4) || !aligned(y, 16))) ||
        (Tr > 0 && (!aligned(rx, 16) || !aligned(rB, 16) || !aligned(rdt, 4))))
        return KDA_ERR_MISALIGNED;
    const int64_t rn = (int64_t)B * T, rr = (int64_t)B * Tr;
    const Span rs = span(S, (int64_t)B * H * N * P * 4), ry = span(y, rn * xw * es);
    const Span ins[] = {rows_span(x, rn, x_stride, xw, es), rows_span(Bm, rn, B_stride, bw, es),
                        rows_span(C, rn, C_stride, bw, es), span(dt, rn * H * 4),
                        rows_span(rx, rr, rx_stride, xw, es), rows_span(rB, rr, rB_stride, bw, es),
                        span(rdt, rr * H * 4), span(n_replay, Tr > 0 ? (int64_t)B * 4 : 0),
                        span(A, (int64_t)H * 4), span(D, (int64_t)H * 4), span(dt_bias, (int64_t)H * 4)};
    for (const Span& r : ins)
        if (overlaps(ry, r) || overlaps(rs, r)) return KDA_ERR_ALIASING;
    if (overlaps(ry, rs)) return KDA_ERR_ALIASING;
    kda::SsmRecParams p{};
    p.rep = kda::SsmTokens{rx, rB, nullptr, rdt, rx_stride, rB_stride, 0, Tr};
    p.out = kda::SsmTokens{x, Bm, C, dt, x_stride, B_stride, C_stride, T};
    p.n_replay = Tr > 0 ? n_replay : nullptr;
    p.dt_bias = dt_bias;
    p.A = A;
    p.D = D;
    p.S = S;
    p.y = y;
    p.B = B;
    p.H = H;
    p.G = G;
    p.N = N;
    p.P = P;
    p.softplus = softplus != 0;
    p.commit = commit != 0;
    return kda::launch_ssm_recurrent(p, in_dtype == KDA_BF16, stream) == hipSuccess ? KDA_OK : KDA_ERR_HIP;
}

size_t kda_verify_drafts_workspace_bytes(int32_t B, int32_t K, int64_t V) {
    if (B < 0 || K < 0 || K > KDA_SPEC_MAX_DRAFTS || V < 1 || V > INT32_MAX) return 0;
    const int64_t n = B * ceil_div(V, kda::kVerifyPart) * 16;
    return (size_t)(n < 16 ? 16 : n);
}

int kda_verify_drafts(const void* p_target, const void* p_draft, int in_dtype,
                      const int32_t* drafts, const int32_t* n_draft, const float* u,
                      const float* u_next, int32_t B, int32_t K, int64_t V, int32_t* n_accepted,
                      int32_t* tokens, void* workspace, size_t workspace_bytes,
                      hipStream_t stream) {
    if (!dtype_ok(in_dtype)) return KDA_ERR_BAD_DTYPE;
    if (B < 0 || K < 0 || K > KDA_SPEC_MAX_DRAFTS || V < 1) return KDA_ERR_BAD_SHAPE;
    if (V > INT32_MAX) return KDA_ERR_TOO_LARGE;
    if (B == 0) return KDA_OK;
    const int64_t parts = ceil_div(V, kda::kVerifyPart);
    if (B * parts > kMaxWorkgroups) return KDA_ERR_TOO_LARGE;
    if (!p_target || !u_next || !n_accepted || !tokens || (K > 0 && (!drafts || !u)))
        return KDA_ERR_NULL_POINTER;
    if (!aligned(p_target, 16) || !aligned(p_draft, 16) || !aligned(workspace, 16) || !aligned(drafts, 4) ||
        !aligned(n_draft, 4) || !aligned(u, 4) || !aligned(u_next, 4) || !aligned(n_accepted, 4) ||
        !aligned(tokens, 4))
        return KDA_ERR_MISALIGNED;
    const size_t need = kda_verify_drafts_workspace_bytes(B, K, V);
    if (!workspace || workspace_bytes < need) return KDA_ERR_WORKSPACE;
    const int64_t es = elem_size(in_dtype);
    const Span ins[] = {span(p_target, (int64_t)B * (K + 1) * V * es), span(p_draft, (int64_t)B * K * V * es),
                        span(drafts, (int64_t)B * K * 4), span(n_draft, (int64_t)B * 4),
                        span(u, (int64_t)B * K * 4), span(u_next, (int64_t)B * 4)};
    const Span outs[] = {span(n_accepted, (int64_t)B * 4), span(tokens, (int64_t)B * (K + 1) * 4),
                         span(workspace, (int64_t)need)};
    for (int a = 0; a < 3; ++a) {
        for (const Span& r : ins)
            if (overlaps(outs[a], r)) return KDA_ERR_ALIASING;
        for (int b = a + 1; b < 3; ++b)
            if (overlaps(outs[a], outs[b])) return KDA_ERR_ALIASING;
    }
    kda::VerifyParams v{};
    v.p = p_target;
    v.q = K > 0 ? p_draft : nullptr;
    v.drafts = drafts;
    v.n_draft = n_draft;
    v.u = u;
    v.u_next = u_next;
    v.n_accepted = n_accepted;
    v.tokens = tokens;
    v.partial = (double*)workspace;
    v.V = V;
    v.B = B;
    v.K = K;
    v.n_parts = (int32_t)parts;
    v.run = (int32_t)(B * parts / kVerifyFill > 1 ? ceil_div(B * parts, kVerifyFill) : 1);
    return kda::launch_verify(v, in_dtype == KDA_BF16, stream) == hipSuccess ? KDA_OK : KDA_ERR_HIP;
}

}  // extern "C"
