// C ABI of softmax attention (include/kda_attn.h) and of the pages of its
// cache (include/kda_pages.h): argument validation and launch planning.
// Everything here runs on the host; nothing is enqueued unless every check
// passes.
#include <stdint.h>

#include "../../include/kda_attn.h"
#include "../../include/kda_pages.h"
#include "kda_attn_launch.h"
#include "kda_host.h"

namespace {

using namespace kda::host;

constexpr int64_t kMaxWideGroups = kMaxWorkgroups / 4;   // workgroups of up to 1024 threads
constexpr int64_t kMaxRows = (int64_t)1 << 36;
constexpr int64_t kMaxSeqRows = (int64_t)1 << 30;        // tokens * heads of a group, counted in 32 bits
constexpr int64_t kUnits = 256;                          // compute units
constexpr int64_t kFill = 512;                           // workgroups that fill the GPU (two per compute unit)
constexpr int64_t kMinPartRows = 256;                    // rows of a part of the backward pass
constexpr int64_t kMinSplitKeys = 256;                   // keys of a part, at least

int attn_shape(int in_dtype, int32_t n_seqs, int64_t T, int32_t H, int32_t G, int32_t D, bool varlen, int64_t* rows) {
    if (!dtype_ok(in_dtype)) return KDA_ERR_BAD_DTYPE;
    if (n_seqs < 0 || T < 0 || H < 1 || G < 1 || H % G != 0 || (D != 64 && D != 128)) return KDA_ERR_BAD_SHAPE;
    if (H > KDA_MAX_HEADS || T > kMaxSeqRows / (H / G)) return KDA_ERR_TOO_LARGE;
    if (varlen) *rows = T;
    else if (!mul_ok((int64_t)n_seqs, T, rows)) return KDA_ERR_TOO_LARGE;
    if (n_seqs == 0) *rows = 0;
    return *rows <= kMaxRows / H ? KDA_OK : KDA_ERR_TOO_LARGE;
}

// The kernels take scores in base 2: scale log2 e has to be a number, too.
bool scale_ok(float x) {
    const float c = x * 1.44269504f;
    return c - c == 0.f;
}

// A row stride: at least the row, whole 16-byte pieces, small enough for
// 32-bit offsets within a tile of rows.
int check_stride(int64_t stride, int64_t width, int64_t es) {
    if (stride < width) return KDA_ERR_BAD_SHAPE;
    if (stride > KDA_ATTN_MAX_STRIDE) return KDA_ERR_TOO_LARGE;
    return (stride * es) % 16 == 0 ? KDA_OK : KDA_ERR_MISALIGNED;
}

int page_shift(int32_t page_size) {
    for (int s = 4; s <= 8; ++s)
        if (page_size == 1 << s) return s;
    return -1;
}

// Blocks of `block` rows, `per` rows to a token (see AttnParams).
int64_t block_slots(int64_t rows, int32_t n_seqs, int64_t T, int64_t per, int64_t block, bool varlen) {
    return varlen ? rows * per / block + n_seqs : n_seqs * ceil_div(T * per, block);
}

kda::AttnParams attn_params(const void* q, int64_t q_stride, const void* k, int64_t k_stride, const void* v,
                            int64_t v_stride, const int32_t* cu, int32_t n_seqs, int64_t T, int64_t rows, int32_t H,
                            int32_t G, int32_t D, float scale, int causal, void* o, float* lse) {
    kda::AttnParams p{};
    p.q = q;
    p.k = k;
    p.v = v;
    p.q_stride = q_stride;
    p.k_stride = k_stride;
    p.v_stride = v_stride;
    p.cu = cu;
    p.n_seqs = n_seqs;
    p.T = T;
    p.rows = rows;
    p.H = H;
    p.G = G;
    p.D = D;
    p.hpg = H / G;
    p.scale = scale;
    p.causal = causal != 0;
    p.o = o;
    p.lse = lse;
    p.splits = 1;
    return p;
}

// Paged attention: a few rows per (request, group) go to the step kernel, whose
// workgroups share all requests' keys equally; more of them to the block
// kernels, where blocks that do not fill the GPU share their keys, too (bf16:
// equal pieces of all blocks; float32: so many parts per block that the GPU is
// full, with kMinSplitKeys keys each where a request holds all it can).
struct PagedPlan {
    bool step;
    int64_t slots, splits, workgroups, max_rows, bytes;
    int block;
};
int block_rows(bool bf16) { return bf16 ? kda::kAttnBlockBf16 : kda::kAttnBlockF32; }
PagedPlan paged_plan(bool bf16, int32_t n_seqs, int64_t T, int64_t rows, int32_t H, int32_t G, int32_t D,
                     int64_t max_tokens, bool varlen) {
    PagedPlan a{};
    a.max_rows = T * (H / G);   // of a request (packed: T is all of them)
    a.step = a.max_rows <= kda::kAttnStepRows;
    if (a.step) {
        // two workgroups per compute unit, or one where its LDS (128 KB with float32 and D 128) leaves no room
        a.workgroups = bf16 || D == 64 ? 2 * kUnits : kUnits;
        const int64_t units = (int64_t)n_seqs * G;
        a.bytes = ((2 * units + 3) / 4 * 4 + (a.workgroups + units) * kda::step_row_tiles(a.max_rows) * 16 * (D + 4)) * 4;
        a.splits = 1;
        return a;
    }
    a.block = block_rows(bf16);
    a.slots = block_slots(rows, n_seqs, T, H / G, a.block, varlen);
    a.splits = 1;
    const int64_t units = a.slots * G;
    if (bf16) {
        // (from four blocks per workgroup on, the order of the blocks evens them out)
        a.workgroups = units > 0 && units < 4 * kFill ? kFill : 0;
        a.bytes = a.workgroups > 0 ? ((2 * units + 3) / 4 * 4 + 2 * a.workgroups * a.block * (D + 4)) * 4 : 0;
        return a;
    }
    // A packed batch's requests may differ by much, so it gets four times the parts.  A chunk of 512 tokens and 7 single
    // ones over 16384 keys, 32 heads of 128 on 8: 1642 us instead of 2606 (63 single ones over 4096: 961 and 976, 64 single
    // ones: 601 and 838); 64 tokens of each of 16 requests over 1024 the other way round: 227 us, 172 with the fewer parts.
    const int64_t want = units > 0 ? (varlen ? 4 : 1) * kFill / units : 1, most = max_tokens / kMinSplitKeys;
    a.splits = want < most ? want : most;
    if (a.splits < 1) a.splits = 1;
    a.bytes = a.splits > 1 ? units * a.splits * a.block * (D + 2) * 4 : 0;
    return a;
}

// The backward pass cuts the rows that a block of keys walks into parts, so
// that there are about 1024 workgroups (twice as many as run at once: the
// first keys' blocks walk the most rows) of at least 256 rows of an average
// sequence each (4 x 200 tokens 43 us, 53 with 256 of the whole batch); the parts'
// sums are added by another launch.  32 heads of 128 on 8, with 1 / 2 / 4 / 8 / 16
// parts, us: 512 tokens 112 / 77 / 60 / 51 / 51, 2048 tokens 407 / 256 / 189 / 186 / 246,
// 4096 tokens 878 / 611 / 542 / 585 / 681, 2 x 4096 1150 / 1013 / 1034 / 1138 / 1352.
// In float32, whose blocks have 16 keys, about 512 workgroups of at least 512
// rows (a launch more costs as much as it saves below): 1024 tokens, 16
// heads of 128 on 4, 196 us, 206 and 232 with twice and four times as many; 385
// of each of 2, 32 heads on 4, 158, 162 and 183; before blocks were cut 279 and
// 224 (operands read one product ahead included).
struct BwdPlan {
    int64_t slots, key_slots, parts, delta, bytes;   // delta: bytes before the parts' sums
};
BwdPlan bwd_plan(bool bf16, int32_t n_seqs, int64_t T, int64_t rows, int32_t H, int32_t G, int32_t D, bool varlen) {
    BwdPlan b{};
    const int block = bf16 ? kda::kAttnBlockBf16 : kda::kAttnBwdBlockF32;
    b.slots = block_slots(rows, n_seqs, T, H / G, block, varlen);
    b.key_slots = block_slots(rows, n_seqs, T, 1, block, varlen);
    b.delta = (rows * H * 4 + 15) / 16 * 16;
    b.parts = 1;
    // (the same for a packed batch of equal lengths)
    const int64_t least = (bf16 ? 1 : 2) * kMinPartRows, most = rows * (H / G) / (least * (n_seqs > 0 ? n_seqs : 1));
    const int64_t blocks = block_slots(rows, n_seqs, T, 1, block, true) * G;
    b.parts = blocks > 0 ? ((bf16 ? 2 : 1) * kFill + blocks / 2) / blocks : 1;
    if (b.parts > most) b.parts = most;
    if (b.parts < 1) b.parts = 1;
    b.bytes = b.delta + (b.parts > 1 ? b.parts * rows * G * 2 * D * 4 : 0);
    return b;
}

int status(hipError_t e) { return e == hipSuccess ? KDA_OK : KDA_ERR_HIP; }

}  // namespace

extern "C" {

int kda_attn_fwd(const void* q, int64_t q_stride, const void* k, int64_t k_stride, const void* v, int64_t v_stride,
                 int in_dtype, const int32_t* cu_seqlens, int32_t n_seqs, int64_t T, int32_t H, int32_t G, int32_t D,
                 float scale, int causal, void* o, float* lse, hipStream_t stream) {
    int64_t rows = 0;
    int rc = attn_shape(in_dtype, n_seqs, T, H, G, D, cu_seqlens != nullptr, &rows);
    if (rc) return rc;
    if (!scale_ok(scale)) return KDA_ERR_BAD_SHAPE;
    if (rows == 0) return KDA_OK;
    if (!q || !k || !v || !o) return KDA_ERR_NULL_POINTER;
    const int64_t es = elem_size(in_dtype), HD = (int64_t)H * D, GD = (int64_t)G * D;
    if ((rc = check_stride(q_stride, HD, es)) || (rc = check_stride(k_stride, GD, es)) ||
        (rc = check_stride(v_stride, GD, es)))
        return rc;
    if (!aligned(q, 16) || !aligned(k, 16) || !aligned(v, 16) || !aligned(o, 16) || !aligned(lse, 4) ||
        !aligned(cu_seqlens, 4))
        return KDA_ERR_MISALIGNED;
    const Span outs[] = {span(o, rows * HD * es), span(lse, rows * H * 4)};
    const Span ins[] = {rows_span(q, rows, q_stride, HD, es), rows_span(k, rows, k_stride, GD, es),
                        rows_span(v, rows, v_stride, GD, es), span(cu_seqlens, ((int64_t)n_seqs + 1) * 4)};
    for (const Span& a : outs)
        for (const Span& b : ins)
            if (overlaps(a, b)) return KDA_ERR_ALIASING;
    if (overlaps(outs[0], outs[1])) return KDA_ERR_ALIASING;
    kda::AttnParams p = attn_params(q, q_stride, k, k_stride, v, v_stride, cu_seqlens, n_seqs, T, rows, H, G, D,
                                    scale, causal, o, lse);
    const bool bf16 = in_dtype == KDA_BF16;
    p.slots = block_slots(rows, n_seqs, T, p.hpg, block_rows(bf16), cu_seqlens != nullptr);
    if (p.slots > kMaxWideGroups / G) return KDA_ERR_TOO_LARGE;
    return status(bf16 ? kda::launch_attn_fwd_bf16(p, stream) : kda::launch_attn_fwd_f32(p, stream));
}

size_t kda_attn_bwd_workspace_bytes(int in_dtype, int32_t n_seqs, int64_t T, int32_t H, int32_t G, int32_t D,
                                    int varlen) {
    int64_t rows = 0;
    if (attn_shape(in_dtype, n_seqs, T, H, G, D, varlen != 0, &rows) || rows == 0) return 0;
    return (size_t)bwd_plan(in_dtype == KDA_BF16, n_seqs, T, rows, H, G, D, varlen != 0).bytes;
}

int kda_attn_bwd_fresh(const void* q, int64_t q_stride, const void* k, int64_t k_stride, const void* v,
                       int64_t v_stride, int in_dtype, const int32_t* cu_seqlens, int32_t n_seqs, int64_t T, int32_t H,
                       int32_t G, int32_t D, float scale, int causal, const void* o, const float* lse,
                       const void* grad_o, void* grad_q, int64_t grad_q_stride, void* grad_k, int64_t grad_k_stride,
                       void* grad_v, int64_t grad_v_stride, void* workspace, size_t workspace_bytes,
                       hipStream_t stream, int fresh) {
    const bool varlen = cu_seqlens != nullptr;
    int64_t rows = 0;
    int rc = attn_shape(in_dtype, n_seqs, T, H, G, D, varlen, &rows);
    if (rc) return rc;
    if (!scale_ok(scale)) return KDA_ERR_BAD_SHAPE;
    if (rows == 0) return KDA_OK;
    if (!q || !k || !v || !o || !lse || !grad_o || !grad_q || !grad_k || !grad_v) return KDA_ERR_NULL_POINTER;
    const int64_t es = elem_size(in_dtype), HD = (int64_t)H * D, GD = (int64_t)G * D;
    const int64_t strides[] = {q_stride, k_stride, v_stride, grad_q_stride, grad_k_stride, grad_v_stride};
    for (int i = 0; i < 6; ++i)
        if ((rc = check_stride(strides[i], i % 3 == 0 ? HD : GD, es))) return rc;
    const void* wide[] = {q, k, v, o, grad_o, grad_q, grad_k, grad_v, workspace};
    for (const void* a : wide)
        if (!aligned(a, 16)) return KDA_ERR_MISALIGNED;
    if (!aligned(lse, 4) || !aligned(cu_seqlens, 4)) return KDA_ERR_MISALIGNED;
    const BwdPlan plan = bwd_plan(in_dtype == KDA_BF16, n_seqs, T, rows, H, G, D, varlen);
    if (plan.slots > kMaxWideGroups / G || plan.key_slots * plan.parts > kMaxWideGroups / G ||
        rows * G / 4 >= kMaxWorkgroups)
        return KDA_ERR_TOO_LARGE;
    if (!workspace || workspace_bytes < (size_t)plan.bytes) return KDA_ERR_WORKSPACE;
    const Span outs[] = {rows_span(grad_q, rows, grad_q_stride, HD, es), rows_span(grad_k, rows, grad_k_stride, GD, es),
                         rows_span(grad_v, rows, grad_v_stride, GD, es), span(workspace, plan.bytes)};
    const Span ins[] = {rows_span(q, rows, q_stride, HD, es), rows_span(k, rows, k_stride, GD, es),
                        rows_span(v, rows, v_stride, GD, es), span(o, rows * HD * es), span(grad_o, rows * HD * es),
                        span(lse, rows * H * 4), span(cu_seqlens, ((int64_t)n_seqs + 1) * 4)};
    for (const Span& a : outs)
        for (const Span& b : ins)
            if (overlaps(a, b)) return KDA_ERR_ALIASING;
    for (int i = 0; i < 4; ++i)
        for (int j = 0; j < i; ++j)
            if (i == 3 ? overlaps(outs[i], outs[j]) : overlaps_rows(outs[i], outs[j])) return KDA_ERR_ALIASING;
    kda::AttnBwdParams a{};
    a.f = attn_params(q, q_stride, k, k_stride, v, v_stride, cu_seqlens, n_seqs, T, rows, H, G, D, scale, causal,
                      const_cast<void*>(o), const_cast<float*>(lse));
    a.f.slots = plan.slots;
    a.key_slots = plan.key_slots;
    a.go = grad_o;
    a.gq = grad_q;
    a.gk = grad_k;
    a.gv = grad_v;
    a.gq_stride = grad_q_stride;
    a.gk_stride = grad_k_stride;
    a.gv_stride = grad_v_stride;
    a.delta = (float*)workspace;
    a.part = (float*)((char*)workspace + plan.delta);
    a.parts = (int32_t)plan.parts;
    a.zero_rest = fresh;
    return status(in_dtype == KDA_BF16 ? kda::launch_attn_bwd_bf16(a, stream) : kda::launch_attn_bwd_f32(a, stream));
}

int kda_attn_bwd(const void* q, int64_t q_stride, const void* k, int64_t k_stride, const void* v, int64_t v_stride,
                 int in_dtype, const int32_t* cu_seqlens, int32_t n_seqs, int64_t T, int32_t H, int32_t G, int32_t D,
                 float scale, int causal, const void* o, const float* lse, const void* grad_o, void* grad_q,
                 int64_t grad_q_stride, void* grad_k, int64_t grad_k_stride, void* grad_v, int64_t grad_v_stride,
                 void* workspace, size_t workspace_bytes, hipStream_t stream) {
    return kda_attn_bwd_fresh(q, q_stride, k, k_stride, v, v_stride, in_dtype, cu_seqlens, n_seqs, T, H, G, D, scale,
                              causal, o, lse, grad_o, grad_q, grad_q_stride, grad_k, grad_k_stride, grad_v,
                              grad_v_stride, workspace, workspace_bytes, stream, 0);
}

// What kda_kv_append and kda_attn_paged_fwd share.
static int check_cache(const void* k_pages, const void* v_pages, int64_t page_stride, int32_t n_pages,
                       int32_t page_size, const int32_t* table, int32_t max_pages, const int32_t* lengths,
                       const int32_t* cu, int64_t GD, int64_t es) {
    if (n_pages < 0 || max_pages < 0 || page_shift(page_size) < 0) return KDA_ERR_BAD_SHAPE;
    if (max_pages > INT32_MAX / page_size / 2) return KDA_ERR_TOO_LARGE;
    if (!lengths || (max_pages > 0 && !table) || (n_pages > 0 && (!k_pages || !v_pages))) return KDA_ERR_NULL_POINTER;
    if (n_pages > 1) {
        if (page_stride < GD * page_size) return KDA_ERR_BAD_SHAPE;
        if (page_stride > ((int64_t)1 << 40)) return KDA_ERR_TOO_LARGE;
        if ((page_stride * es) % 16 != 0) return KDA_ERR_MISALIGNED;
    }
    return aligned(k_pages, 16) && aligned(v_pages, 16) && aligned(table, 4) && aligned(lengths, 4) && aligned(cu, 4)
               ? KDA_OK : KDA_ERR_MISALIGNED;
}

int kda_kv_append(const void* k, int64_t k_stride, const void* v, int64_t v_stride, int in_dtype, void* k_pages,
                  void* v_pages, int64_t page_stride, int32_t n_pages, int32_t page_size, const int32_t* table,
                  int32_t max_pages, const int32_t* lengths, const int32_t* cu_seqlens, int32_t n_seqs, int64_t T,
                  int32_t G, int32_t D, hipStream_t stream) {
    int64_t rows = 0;
    int rc = attn_shape(in_dtype, n_seqs, T, G, G, D, cu_seqlens != nullptr, &rows);
    if (rc) return rc;
    const int64_t es = elem_size(in_dtype), GD = (int64_t)G * D;
    if (n_seqs > 0 && (rc = check_cache(k_pages, v_pages, page_stride, n_pages, page_size, table, max_pages, lengths,
                                        cu_seqlens, GD, es)))
        return rc;
    if (rows == 0 || n_pages == 0 || max_pages == 0) return KDA_OK;
    if (!k || !v) return KDA_ERR_NULL_POINTER;
    if ((rc = check_stride(k_stride, GD, es)) || (rc = check_stride(v_stride, GD, es))) return rc;
    if (!aligned(k, 16) || !aligned(v, 16)) return KDA_ERR_MISALIGNED;
    if (rows * GD * es / 16 / 256 >= kMaxWorkgroups) return KDA_ERR_TOO_LARGE;
    const Span outs[] = {rows_span(k_pages, n_pages, page_stride, GD * page_size, es),
                         rows_span(v_pages, n_pages, page_stride, GD * page_size, es)};
    const Span ins[] = {rows_span(k, rows, k_stride, GD, es), rows_span(v, rows, v_stride, GD, es),
                        span(table, (int64_t)n_seqs * max_pages * 4), span(lengths, (int64_t)n_seqs * 4),
                        span(cu_seqlens, ((int64_t)n_seqs + 1) * 4)};
    for (const Span& a : outs)
        for (const Span& b : ins)
            if (overlaps(a, b)) return KDA_ERR_ALIASING;
    if (overlaps_rows(outs[0], outs[1])) return KDA_ERR_ALIASING;
    kda::AppendParams p{};
    p.k = k;
    p.v = v;
    p.k_pages = k_pages;
    p.v_pages = v_pages;
    p.table = table;
    p.lengths = lengths;
    p.cu = cu_seqlens;
    p.k_stride = k_stride;
    p.v_stride = v_stride;
    p.page_stride = page_stride;
    p.rows = rows;
    p.T = T;
    p.n_seqs = n_seqs;
    p.G = G;
    p.D = D;
    p.n_pages = n_pages;
    p.max_pages = max_pages;
    p.page_shift = page_shift(page_size);
    return status(kda::launch_kv_append(p, in_dtype == KDA_BF16, stream));
}

size_t kda_attn_paged_workspace_bytes(int in_dtype, int32_t n_seqs, int64_t T, int32_t H, int32_t G, int32_t D,
                                      int32_t page_size, int32_t max_pages, int varlen) {
    int64_t rows = 0;
    if (attn_shape(in_dtype, n_seqs, T, H, G, D, varlen != 0, &rows) || page_shift(page_size) < 0 || max_pages < 0 ||
        rows == 0)
        return 0;
    return (size_t)paged_plan(in_dtype == KDA_BF16, n_seqs, T, rows, H, G, D, (int64_t)max_pages * page_size, varlen != 0).bytes;
}

int kda_attn_paged_fwd(const void* q, int64_t q_stride, int in_dtype, const void* k_pages, const void* v_pages,
                       int64_t page_stride, int32_t n_pages, int32_t page_size, const int32_t* table,
                       int32_t max_pages, const int32_t* lengths, const int32_t* cu_seqlens, int32_t n_seqs, int64_t T,
                       int32_t H, int32_t G, int32_t D, float scale, void* o, float* lse, void* workspace,
                       size_t workspace_bytes, hipStream_t stream) {
    const bool varlen = cu_seqlens != nullptr;
    int64_t rows = 0;
    int rc = attn_shape(in_dtype, n_seqs, T, H, G, D, varlen, &rows);
    if (rc) return rc;
    if (!scale_ok(scale)) return KDA_ERR_BAD_SHAPE;
    const int64_t es = elem_size(in_dtype), HD = (int64_t)H * D, GD = (int64_t)G * D;
    if (n_seqs > 0 && (rc = check_cache(k_pages, v_pages, page_stride, n_pages, page_size, table, max_pages, lengths,
                                        cu_seqlens, GD, es)))
        return rc;
    if (rows == 0) return KDA_OK;
    if (!q || !o) return KDA_ERR_NULL_POINTER;
    if ((rc = check_stride(q_stride, HD, es))) return rc;
    if (!aligned(q, 16) || !aligned(o, 16) || !aligned(lse, 4) || !aligned(workspace, 16)) return KDA_ERR_MISALIGNED;
    const PagedPlan plan = paged_plan(in_dtype == KDA_BF16, n_seqs, T, rows, H, G, D, (int64_t)max_pages * page_size, varlen);
    if (plan.step ? (int64_t)n_seqs * G > kMaxWorkgroups / plan.max_rows
                  : plan.slots > kMaxWideGroups / G / plan.splits / 32)
        return KDA_ERR_TOO_LARGE;
    if (plan.bytes > 0 && (!workspace || workspace_bytes < (size_t)plan.bytes)) return KDA_ERR_WORKSPACE;
    const Span outs[] = {span(o, rows * HD * es), span(lse, rows * H * 4), span(workspace, plan.bytes)};
    const Span ins[] = {rows_span(q, rows, q_stride, HD, es), rows_span(k_pages, n_pages, page_stride, GD * page_size, es),
                        rows_span(v_pages, n_pages, page_stride, GD * page_size, es),
                        span(table, (int64_t)n_seqs * max_pages * 4), span(lengths, (int64_t)n_seqs * 4),
                        span(cu_seqlens, ((int64_t)n_seqs + 1) * 4)};
    for (const Span& a : outs)
        for (const Span& b : ins)
            if (overlaps(a, b)) return KDA_ERR_ALIASING;
    for (int i = 0; i < 3; ++i)
        for (int j = 0; j < i; ++j)
            if (overlaps(outs[i], outs[j])) return KDA_ERR_ALIASING;
    kda::AttnParams p = attn_params(q, q_stride, k_pages, 0, v_pages, 0, cu_seqlens, n_seqs, T, rows, H, G, D, scale,
                                    1, o, lse);
    p.table = table;
    p.lengths = lengths;
    p.page_stride = page_stride;
    p.n_pages = n_pages;
    p.max_pages = max_pages;
    p.page_shift = page_shift(page_size);
    p.slots = plan.slots;
    p.splits = (int32_t)plan.splits;
    p.workgroups = (int32_t)plan.workgroups;
    p.part = (float*)workspace;
    if (plan.step) return status(kda::launch_attn_step(p, in_dtype == KDA_BF16, (int32_t)plan.max_rows, stream));
    return status(in_dtype == KDA_BF16 ? kda::launch_attn_fwd_bf16(p, stream) : kda::launch_attn_fwd_f32(p, stream));
}

// ------------------------------------------------------------------ pages

static int check_pages(const void* table, const void* lengths, const void* refs, int32_t n_slots, int32_t max_pages,
                       int32_t n_pages, int32_t page_size) {
    if (n_slots < 0 || max_pages < 0 || n_pages < 0 || page_shift(page_size) < 0) return KDA_ERR_BAD_SHAPE;
    if (n_slots > KDA_PAGES_MAX_SLOTS || max_pages > INT32_MAX / page_size / 2 ||
        (int64_t)n_slots * max_pages > INT32_MAX / 2 || n_pages > INT32_MAX / 4)
        return KDA_ERR_TOO_LARGE;
    if ((n_slots > 0 && (!lengths || (max_pages > 0 && !table))) || (n_pages > 0 && !refs)) return KDA_ERR_NULL_POINTER;
    return aligned(table, 4) && aligned(lengths, 4) && aligned(refs, 4) ? KDA_OK : KDA_ERR_MISALIGNED;
}
static int check_data(void* const* pages, const int64_t* bytes, const int64_t* stride, int32_t n_tensors,
                      int32_t n_pages, kda::PageData* d, Span* spans) {
    if (n_tensors < 0) return KDA_ERR_BAD_SHAPE;
    if (n_tensors > KDA_PAGES_MAX_TENSORS) return KDA_ERR_TOO_LARGE;
    if (n_tensors > 0 && (!pages || !bytes || !stride)) return KDA_ERR_NULL_POINTER;
    d->n = n_pages > 0 ? n_tensors : 0;
    for (int t = 0; t < d->n; ++t) {
        if (!pages[t]) return KDA_ERR_NULL_POINTER;
        if (bytes[t] <= 0 || (n_pages > 1 && stride[t] < bytes[t])) return KDA_ERR_BAD_SHAPE;
        if (bytes[t] > ((int64_t)1 << 36) || stride[t] > ((int64_t)1 << 41)) return KDA_ERR_TOO_LARGE;
        if (!aligned(pages[t], 16) || bytes[t] % 16 != 0 || (n_pages > 1 && stride[t] % 16 != 0)) return KDA_ERR_MISALIGNED;
        d->base[t] = (char*)pages[t];
        d->bytes[t] = bytes[t];
        d->stride[t] = n_pages > 1 ? stride[t] : bytes[t];
        spans[t] = rows_span(pages[t], n_pages, d->stride[t], bytes[t], 1);
        for (int u = 0; u < t; ++u)
            if (overlaps_rows(spans[t], spans[u])) return KDA_ERR_ALIASING;
    }
    return KDA_OK;
}
static bool apart(const Span* a, int n, const Span* b, int m) {   // nothing of a in b, nor in another of a
    for (int i = 0; i < n; ++i) {
        for (int j = 0; j < m; ++j)
            if (overlaps(a[i], b[j])) return false;
        for (int j = 0; j < i; ++j)
            if (overlaps(a[i], a[j])) return false;
    }
    return true;
}
static kda::PagesParams pages_params(const int32_t* table, const int32_t* lengths, const int32_t* refs,
                                     int32_t n_slots, int32_t max_pages, int32_t n_pages, int32_t page_size) {
    kda::PagesParams p{};
    p.table = table;
    p.lengths = lengths;
    p.refs = refs;
    p.table_out = const_cast<int32_t*>(table);
    p.lengths_out = const_cast<int32_t*>(lengths);
    p.refs_out = const_cast<int32_t*>(refs);
    p.n_slots = n_slots;
    p.max_pages = max_pages;
    p.n_pages = n_pages;
    p.page_shift = page_shift(page_size);
    return p;
}

int kda_kv_resize(int32_t* table, int32_t* lengths, int32_t* refs, const int32_t* want, int32_t* ok, int32_t n_slots,
                  int32_t max_pages, int32_t n_pages, int32_t page_size, hipStream_t stream) {
    int rc = check_pages(table, lengths, refs, n_slots, max_pages, n_pages, page_size);
    if (rc) return rc;
    if (n_slots == 0) return KDA_OK;
    if (!want) return KDA_ERR_NULL_POINTER;
    if (!aligned(want, 4) || !aligned(ok, 4)) return KDA_ERR_MISALIGNED;
    const Span outs[] = {span(table, (int64_t)n_slots * max_pages * 4), span(lengths, (int64_t)n_slots * 4),
                         span(refs, (int64_t)n_pages * 4), span(ok, (int64_t)n_slots * 4)};
    const Span ins[] = {span(want, (int64_t)n_slots * 4)};
    if (!apart(outs, 4, ins, 1)) return KDA_ERR_ALIASING;
    kda::PagesParams p = pages_params(table, lengths, refs, n_slots, max_pages, n_pages, page_size);
    p.want = want;
    p.ok = ok;
    return status(kda::launch_kv_resize(p, stream));
}

size_t kda_kv_fork_workspace_bytes(int32_t n, int32_t n_slots, int32_t max_pages) {
    if (n < 0 || n > KDA_PAGES_MAX_SLOTS || n_slots < 0 || n_slots > KDA_PAGES_MAX_SLOTS || max_pages < 0) return 0;
    return (((size_t)n_slots + 3) / 4 * 4 + (size_t)n * (5 + (size_t)max_pages)) * 4 + 16;
}

int kda_kv_fork(int32_t* table, int32_t* lengths, int32_t* refs, const int32_t* src, const int32_t* dst, int32_t* ok,
                int32_t n, int32_t n_slots, int32_t max_pages, int32_t n_pages, int32_t page_size, void* const* pages,
                const int64_t* page_bytes, const int64_t* page_stride_bytes, int32_t n_tensors, void* workspace,
                size_t workspace_bytes, hipStream_t stream) {
    int rc = check_pages(table, lengths, refs, n_slots, max_pages, n_pages, page_size);
    if (rc) return rc;
    if (n < 0) return KDA_ERR_BAD_SHAPE;
    if (n > KDA_PAGES_MAX_SLOTS || n * (ceil_div(max_pages, 256) + 64) > kMaxWorkgroups) return KDA_ERR_TOO_LARGE;
    kda::PagesParams p = pages_params(table, lengths, refs, n_slots, max_pages, n_pages, page_size);
    Span data[KDA_PAGES_MAX_TENSORS];
    if ((rc = check_data(pages, page_bytes, page_stride_bytes, n_tensors, n_pages, &p.data, data))) return rc;
    if (n == 0) return KDA_OK;
    if (!src || !dst) return KDA_ERR_NULL_POINTER;
    if (!aligned(src, 4) || !aligned(dst, 4) || !aligned(ok, 4) || !aligned(workspace, 16)) return KDA_ERR_MISALIGNED;
    const size_t need = kda_kv_fork_workspace_bytes(n, n_slots, max_pages);
    if (!workspace || workspace_bytes < need) return KDA_ERR_WORKSPACE;
    const Span outs[] = {span(table, (int64_t)n_slots * max_pages * 4), span(lengths, (int64_t)n_slots * 4),
                         span(refs, (int64_t)n_pages * 4), span(ok, (int64_t)n * 4), span(workspace, (int64_t)need)};
    const Span ins[] = {span(src, (int64_t)n * 4), span(dst, (int64_t)n * 4)};
    if (!apart(outs, 5, ins, 2) || !apart(outs, 5, data, p.data.n)) return KDA_ERR_ALIASING;
    for (int t = 0; t < p.data.n; ++t)
        if (overlaps(data[t], ins[0]) || overlaps(data[t], ins[1])) return KDA_ERR_ALIASING;
    p.src = src;
    p.dst = dst;
    p.ok = ok;
    p.n = n;
    p.ws = (int32_t*)workspace;
    return status(kda::launch_kv_fork(p, stream));
}

size_t kda_kv_compact_workspace_bytes(int32_t n_pages) {
    return n_pages < 0 ? 0 : 16 + 12 * (size_t)n_pages;
}

int kda_kv_compact(const int32_t* table, const int32_t* lengths, const int32_t* refs, int32_t* table_out,
                   int32_t* refs_out, int32_t* n_live, int32_t n_slots, int32_t max_pages, int32_t n_pages,
                   int32_t page_size, void* const* pages, const int64_t* page_bytes, const int64_t* page_stride_bytes,
                   int32_t n_tensors, void* workspace, size_t workspace_bytes, hipStream_t stream) {
    int rc = check_pages(table, lengths, refs, n_slots, max_pages, n_pages, page_size);
    if (rc) return rc;
    if (!n_live || (n_slots > 0 && max_pages > 0 && !table_out) || (n_pages > 0 && !refs_out)) return KDA_ERR_NULL_POINTER;
    kda::PagesParams p = pages_params(table, lengths, refs, n_slots, max_pages, n_pages, page_size);
    Span data[KDA_PAGES_MAX_TENSORS];
    if ((rc = check_data(pages, page_bytes, page_stride_bytes, n_tensors, n_pages, &p.data, data))) return rc;
    if (!aligned(table_out, 4) || !aligned(refs_out, 4) || !aligned(n_live, 4) || !aligned(workspace, 16))
        return KDA_ERR_MISALIGNED;
    const size_t need = kda_kv_compact_workspace_bytes(n_pages);
    if (!workspace || workspace_bytes < need) return KDA_ERR_WORKSPACE;
    const int64_t tb = (int64_t)n_slots * max_pages * 4, rb = (int64_t)n_pages * 4;
    const Span outs[] = {span(table_out, tb), span(refs_out, rb), span(n_live, 4), span(workspace, (int64_t)need)};
    const Span ins[] = {span(lengths, (int64_t)n_slots * 4)};
    if (!apart(outs, 4, ins, 1) || !apart(outs, 4, data, p.data.n)) return KDA_ERR_ALIASING;
    for (int i = 0; i < 4; ++i) {
        if (!(i == 0 && table_out == table) && overlaps(outs[i], span(table, tb))) return KDA_ERR_ALIASING;
        if (!(i == 1 && refs_out == refs) && overlaps(outs[i], span(refs, rb))) return KDA_ERR_ALIASING;
    }
    for (int t = 0; t < p.data.n; ++t)
        if (overlaps(data[t], span(table, tb)) || overlaps(data[t], span(refs, rb)) || overlaps(data[t], ins[0]))
            return KDA_ERR_ALIASING;
    p.table_out = table_out;
    p.refs_out = refs_out;
    p.n_live = n_live;
    p.ws = (int32_t*)workspace;
    return status(kda::launch_kv_compact(p, stream));
}

}  // extern "C"
