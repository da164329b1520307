// Host-side launch interface between the C ABI (kda_attn_abi.hip) and the
// kernels of softmax attention, its paged cache and the pages' upkeep.
#pragma once

#include <hip/hip_runtime_api.h>
#include <stddef.h>
#include <stdint.h>

namespace kda {

// Rows of one (sequence, group): token t and head hh of the group's hpg heads
// are row t * hpg + hh, so that a block of rows shares its keys and values.
// Block j of sequence n, of `block` rows, has slot
//   equal lengths:  n * ceil(T * hpg / block) + j,
//   packed:         cu[n] * hpg / block + n + j   (slots = rows * hpg / block + n_seqs).
struct AttnParams {
    const void* q;           // rows of q_stride elements, [H, D] each
    const void* k;           // rows of k_stride elements, [G, D] each; paged: pages [G, page, D]
    const void* v;
    const int32_t* cu;       // packed: device [n_seqs + 1]; equal lengths: nullptr
    const int32_t* table;    // paged: [n_seqs, max_pages]
    const int32_t* lengths;  // paged: [n_seqs]; nullptr: k and v are token rows
    void* o;                 // [rows, H, D]
    float* lse;              // [rows, H] or nullptr
    float* part;             // split: results of the parts, see below
    int64_t q_stride, k_stride, v_stride;
    int64_t page_stride;     // elements
    int64_t rows, T;         // token rows; tokens per sequence (packed: rows)
    int64_t slots;           // blocks of rows per group
    int32_t n_seqs, H, G, D, hpg;
    int32_t n_pages, max_pages, page_shift;
    int32_t causal;
    int32_t splits;          // parts of a block's keys, each its own workgroup (float32 block kernel)
    int32_t workgroups;      // see the kernels below
    float scale;
};

// Block kernels.  float32: with splits > 1, part s of block (slot, g) leaves
// for each of its rows D sums of e^{s - m} v, then the sum of e^{s - m}, then m
// (base 2), at part + (((slot * G + g) * splits + s) * block + row) * (D + 2).
// bf16: with workgroups > 0, that many take equal pieces of all blocks' keys; at
// `part`: two numbers for each (group, slot), then (from the next 16 bytes on)
// two parts for each workgroup, of D sums, the sum of weights, m and two
// unused floats for each row of a block.
constexpr int kAttnBlockF32 = 64;    // rows of a block
constexpr int kAttnBlockBf16 = 128;
constexpr int kAttnBwdBlockF32 = 16;
hipError_t launch_attn_fwd_f32(const AttnParams& p, hipStream_t stream);
hipError_t launch_attn_fwd_bf16(const AttnParams& p, hipStream_t stream);

// Step kernel, for (request, group) pairs of at most kAttnStepRows rows, with
// step_row_tiles tiles of 16 rows.  At `part`: two numbers for each pair u = b *
// G + g, then (from the next 16 bytes on) the parts; workgroup w's part of pair
// u has slot w + u, with D sums, the sum of weights, m and two unused floats
// for each row of the tiles.
constexpr int kAttnStepRows = 64;
constexpr int step_row_tiles(int64_t rows) { return (int)((rows + 15) / 16); }
hipError_t launch_attn_step(const AttnParams& p, bool bf16_in, int32_t max_rows, hipStream_t stream);

struct AttnBwdParams {
    AttnParams f;            // inputs; o and lse as the forward call gave them
    const void* go;          // [rows, H, D]
    void* gq;                // rows of gq_stride elements
    void* gk;
    void* gv;
    float* delta;            // [rows, H]: grad_o . o
    float* part;             // parts > 1: [parts, rows, G, 2, D] sums of grad_k and grad_v
    int32_t parts;           // of a block of keys' rows, each its own workgroup
    int64_t gq_stride, gk_stride, gv_stride;
    int64_t key_slots;       // blocks of keys per group
    int32_t zero_rest;       // KDA_FRESH_*: these outputs' rows of no sequence become zero
};
constexpr int kAttnRest = 256;   // workgroups that see to the rows of no sequence
hipError_t launch_attn_bwd_rest(const AttnBwdParams& p, bool bf16_in, hipStream_t stream);
hipError_t launch_attn_bwd_f32(const AttnBwdParams& p, hipStream_t stream);
hipError_t launch_attn_bwd_bf16(const AttnBwdParams& p, hipStream_t stream);

struct AppendParams {
    const void* k;
    const void* v;
    void* k_pages;
    void* v_pages;
    const int32_t* table;
    const int32_t* lengths;
    const int32_t* cu;
    int64_t k_stride, v_stride, page_stride;
    int64_t rows, T;
    int32_t n_seqs, G, D, n_pages, max_pages, page_shift;
};
hipError_t launch_kv_append(const AppendParams& p, bool bf16_in, hipStream_t stream);

constexpr int kPagesTensors = 16;
struct PageData {
    char* base[kPagesTensors];
    int64_t bytes[kPagesTensors];
    int64_t stride[kPagesTensors];
    int32_t n;
};
struct PagesParams {
    const int32_t* table;
    const int32_t* lengths;
    const int32_t* refs;
    int32_t* table_out;      // resize, fork: table itself
    int32_t* lengths_out;
    int32_t* refs_out;
    const int32_t* want;     // resize: [n_slots]
    const int32_t* src;      // fork: [n]
    const int32_t* dst;
    int32_t* ok;             // or nullptr
    int32_t* n_live;         // compact
    int32_t* ws;
    PageData data;
    int32_t n, n_slots, max_pages, n_pages, page_shift;
};
hipError_t launch_kv_resize(const PagesParams& p, hipStream_t stream);
hipError_t launch_kv_fork(const PagesParams& p, hipStream_t stream);
hipError_t launch_kv_compact(const PagesParams& p, hipStream_t stream);

}  // namespace kda

// The backward pass for outputs of the binding's own making: rows of no
// sequence become zero in the outputs that `fresh` names.
#define KDA_FRESH_Q 1
#define KDA_FRESH_K 2
#define KDA_FRESH_V 4
extern "C" int kda_attn_bwd_fresh(const void* q, int64_t q_stride, const void* k, int64_t k_stride,
                                  const void* v, int64_t v_stride, int in_dtype,
                                  const int32_t* cu_seqlens, int32_t n_seqs, int64_t T, int32_t H,
                                  int32_t G, int32_t D, float scale, int causal, const void* o,
                                  const float* lse, const void* grad_o, void* grad_q,
                                  int64_t grad_q_stride, void* grad_k, int64_t grad_k_stride,
                                  void* grad_v, int64_t grad_v_stride, void* workspace,
                                  size_t workspace_bytes, hipStream_t stream, int fresh);
