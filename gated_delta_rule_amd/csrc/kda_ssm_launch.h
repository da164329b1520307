// Host-side launch interface between the C ABI (kda_ssm_abi.hip) and the
// kernels of the state space scan, its convolution and the draft verification.
#pragma once

#include <hip/hip_runtime_api.h>
#include <stddef.h>
#include <stdint.h>

namespace kda {

struct ConvParams {
    const void* x;           // rows of x_stride elements
    const void* rx;          // replay rows (step form) or nullptr
    const float* w;          // [channels, width]
    const float* bias;       // [channels] or nullptr
    float* cache;            // [n_seqs, width - 1, channels] or nullptr
    const int32_t* cu;       // packed: device [n_seqs + 1]; equal lengths: nullptr
    const int32_t* n_replay; // [n_seqs] or nullptr (step form)
    void* y;                 // [rows, channels]
    int64_t x_stride, rx_stride;
    int64_t rows, T;         // token rows; tokens per sequence (equal lengths)
    int32_t n_seqs, channels, width, activation;
    int32_t Tr, commit;      // step form
};
hipError_t launch_conv_fwd(const ConvParams& p, bool bf16_in, hipStream_t stream);
hipError_t launch_conv_step(const ConvParams& p, bool bf16_in, hipStream_t stream);

// Token rows per wave (a wave takes 256 channels of them): whole rounds of
// the 4096 waves that run at once (16 per compute unit), with 32 to 64 rows
// per wave where there are that many, at least 8.  A workgroup's waves share
// a partial sum of the weight gradient: the backward workspace holds
// [conv_bwd_parts, width + 1, channels] floats.
constexpr int64_t kConvWaves = 4;
constexpr int64_t conv_rows_per_wave(int64_t rows, int64_t channels) {
    const int64_t units = rows * ((channels + 255) / 256);
    const int64_t rounds = units / (4096 * 32) > 0 ? units / (4096 * 32) : 1;
    const int64_t r = (units + 4096 * rounds - 1) / (4096 * rounds);
    return r < 8 ? 8 : (r + 3) / 4 * 4;
}
constexpr int64_t conv_bwd_parts(int64_t rows, int64_t channels) {
    const int64_t per = kConvWaves * conv_rows_per_wave(rows, channels);
    return (rows + per - 1) / per;
}
struct ConvBwdParams {
    ConvParams f;            // x, w, bias, cache (before the forward call), cu, sizes
    const void* gy;          // rows of gy_stride elements
    void* gx;                // [rows, channels]
    float* gw;               // [channels, width]
    float* gbias;            // [channels] or nullptr
    float* gcache;           // [n_seqs, width - 1, channels] or nullptr
    float* partial;
    int64_t gy_stride;
    int32_t rows_per_wave;
    int32_t zero_rest;       // rows of gx that belong to no sequence become zero
};
hipError_t launch_conv_bwd(const ConvBwdParams& p, bool bf16_in, hipStream_t stream);

// One stream of tokens of the recurrent form.
struct SsmTokens {
    const void* x;           // [B, T] rows of x_stride elements, [H, P] each
    const void* Bm;          // rows of B_stride elements, [G, N] each
    const void* C;           // rows of C_stride elements (nullptr for replay)
    const float* dt;         // [B, T, H]
    int64_t x_stride, B_stride, C_stride;
    int32_t T;
};
struct SsmRecParams {
    SsmTokens rep, out;
    const int32_t* n_replay; // [B] or nullptr
    const float* dt_bias;    // [H] or nullptr
    const float* A;          // [H]
    const float* D;          // [H] or nullptr
    float* S;                // [B, H, N, P]
    void* y;                 // [B, T, H, P]
    int32_t B, H, G, N, P, softplus, commit;
};
hipError_t launch_ssm_recurrent(const SsmRecParams& p, bool bf16_in, hipStream_t stream);

struct VerifyParams {
    const void* p;           // [B, K + 1, V]
    const void* q;           // [B, K, V] or nullptr
    const int32_t* drafts;   // [B, K]
    const int32_t* n_draft;  // [B] or nullptr
    const float* u;          // [B, K]
    const float* u_next;     // [B]
    int32_t* n_accepted;     // [B]
    int32_t* tokens;         // [B, K + 1]
    double* partial;         // [B, n_parts, 2]
    int64_t V;
    int32_t B, K, n_parts, run;   // run: parts per workgroup of the first launch
};
// Vocabulary entries per partial sum of a row, threads that read them.
constexpr int64_t kVerifyPart = 4096;
constexpr int kVerifyThreads = 256;
hipError_t launch_verify(const VerifyParams& p, bool bf16_in, hipStream_t stream);

// Scan over whole sequences.  Every sequence is cut into segments of seg_len
// tokens (a multiple of 64; at least the longest sequence: no cut), each one
// chain of chunks; segment j of sequence n has slot
//   equal lengths:  n * ceil(T / seg_len) + j,
//   packed:         cu[n] / seg_len + n + j   (slots = T / seg_len + n_seqs),
//   no cut:         n.
struct SsmScanParams {
    const void* x;           // rows of x_stride elements, [H, P] each
    const void* B;           // rows of B_stride elements, [G, N] each
    const void* C;           // rows of C_stride elements
    const float* dt;         // [rows, H]
    const float* dt_bias;    // [H] or nullptr
    const float* A;          // [H]
    const float* D;          // [H] or nullptr
    const float* S0;         // [n_seqs, H, N, P] or nullptr
    const int32_t* cu;       // packed: device [n_seqs + 1]; equal lengths: nullptr
    void* y;                 // [rows, H, P]
    float* S_T;              // [n_seqs, H, N, P] or nullptr
    float* seg;              // cut: [slots, H, N, P] local final, then incoming states
    float* seg_decay;        // cut: [slots, H] the segments' decay factors
    int64_t x_stride, B_stride, C_stride;
    int64_t rows, T;         // token rows; tokens per sequence (packed: rows)
    int64_t seg_len, slots;
    int32_t cut;             // sequences are cut into segments
    int32_t n_seqs, H, G, N, P, softplus;
    // Groups g0 .. g0 + gn - 1 only (the forward call: all).  The arrays seg,
    // seg_decay and states hold the gn * H / G heads of those groups.
    int32_t g0, gn;
    float* states;           // walks: [chunk slots, heads, N, P], see below
};
hipError_t launch_ssm_chunk_fwd(const SsmScanParams& p, bool bf16_in, hipStream_t stream);

// The backward pass's walks: dir[0], the state at every chunk's start; dir[1],
// from the sequences' ends, the state gradient at every chunk's end, from C as
// B, grad_y as x, grad_S_T as S0, leaving the gradient of the initial states
// in S_T.  Same shapes, segments and slots in both.
// Chunks of ssm_chunk_tokens(bf16) tokens; chunk c of sequence n has slot
//   equal lengths: n * ceil(T / tokens) + c,  packed: cu[n] / tokens + n + c.
struct SsmScanDirs {
    SsmScanParams dir[2];
};
hipError_t launch_ssm_walks(const SsmScanDirs& d, bool bf16_in, hipStream_t stream);
constexpr int64_t ssm_chunk_tokens(bool bf16_in) { return bf16_in ? 64 : 32; }

struct SsmGradParams {
    SsmScanParams f;         // inputs; g0, gn the groups of this launch
    const void* gy;          // [rows, H, P]
    const float* states;     // [chunk slots, heads, N, P]
    const float* dstates;    // [chunk slots, heads, N, P]
    void* gx;                // rows of gx_stride elements
    void* gB;                // rows of gB_stride elements
    void* gC;                // rows of gC_stride elements
    float* gdt;              // [rows, H]
    float* gA;               // [H]
    float* gD;               // [H] or nullptr
    float* gbias;            // [H] or nullptr
    float* part;             // [2, blocks, gn, rows, N] when a group's heads take several blocks
    float* sums;             // [chunk slots, heads, 3]: sums for A, D and dt_bias
    int64_t gx_stride, gB_stride, gC_stride;
    int64_t slots;           // chunk slots
    int32_t heads_per_block, blocks;   // heads of a group per workgroup; workgroups per group
    int32_t zero_rest;       // KDA_FRESH_*: these outputs' rows of no sequence become zero
};
constexpr int64_t kGradRest = 256;   // workgroups that see to them, at most
hipError_t launch_ssm_grad(const SsmGradParams& p, bool bf16_in, hipStream_t stream);

}  // namespace kda

// The backward passes for outputs of the binding's own making: as their
// namesakes in include/kda_ssm.h, but rows of no sequence become zero (the
// gradient of rows that affect nothing) in the outputs that `fresh` names,
// where the others keep what their owner has put there.
#define KDA_FRESH_X 1
#define KDA_FRESH_B 2
#define KDA_FRESH_C 4
#define KDA_FRESH_DT 8
extern "C" {
int kda_ssm_conv_bwd_fresh(const void* x, int64_t x_stride, int in_dtype, const float* w,
                           const float* bias, const float* cache, const int32_t* cu_seqlens,
                           int32_t n_seqs, int64_t T, int32_t channels, int32_t width, int activation,
                           const void* grad_y, int64_t grad_y_stride, void* grad_x, float* grad_w,
                           float* grad_bias, float* grad_cache, void* workspace, size_t workspace_bytes,
                           hipStream_t stream, int fresh);
int kda_ssm_chunk_bwd_fresh(const void* x, int64_t x_stride, const void* B, int64_t B_stride,
                            const void* C, int64_t C_stride, int in_dtype, const float* dt,
                            const float* dt_bias, int softplus, const float* A, const float* D,
                            const float* S0, const int32_t* cu_seqlens, int32_t n_seqs, int64_t T,
                            int32_t H, int32_t G, int32_t N, int32_t P, const void* grad_y,
                            const float* grad_S_T, void* grad_x, int64_t grad_x_stride, void* grad_B,
                            int64_t grad_B_stride, void* grad_C, int64_t grad_C_stride, float* grad_dt,
                            float* grad_A, float* grad_D, float* grad_dt_bias, float* grad_S0,
                            void* workspace, size_t workspace_bytes, hipStream_t stream, int fresh);
}
