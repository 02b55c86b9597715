// qmm_attn.h -- the attention calls' launchers and the views they take.
#pragma once
#include <cuda_runtime.h>
#include <stdint.h>

#include "qmm.h"

namespace qmm {

// Largest head size of the attention calls (a multiple of 8).
constexpr int kMaxHeadDim = 128;

// Query heads, key/value heads and the size of one head.
struct HeadShape {
    int hq, hk, d;
};

// Strides of a [tokens][heads][d] view in elements (d contiguous).
struct HeadStrides {
    int64_t t, h;
};

struct RopeArgs {
    const void *q, *k, *v;  // v == nullptr: no values
    void *qo, *ko, *vo;
    HeadStrides sq, sk, sv, sqo, sko, svo;
    HeadShape shape;
    const float *wq, *wk;  // nullptr: no norm for that side
    const int32_t *positions;
    const float *inv_freq;
    int rotary;  // even number of leading elements that are rotated; 0: none
    int interleaved;
    float eps;
    int64_t m;
};
cudaError_t launch_qk_norm_rope(const RopeArgs &a, qmm_float in_type, qmm_float out_type, cudaStream_t st);

struct PromptArgs {
    const void *q, *k, *v;
    void *out;
    float *lse;  // [tokens_q][hq] or nullptr
    HeadStrides sq, sk, sv, so;
    HeadShape shape;
    const int32_t *cu_q, *cu_k;  // [n_seqs + 1]
    int64_t n_seqs, tokens_q, tokens_k;
    int causal;
    float scale;
};
size_t attn_prompt_workspace_bytes(const PromptArgs &a);
cudaError_t launch_attn_prompt(const PromptArgs &a, qmm_float t, void *ws, cudaStream_t st);

struct DecodeArgs {
    const void *q, *k, *v, *pk, *pv;  // pk, pv: the shared prefix (prefix == 0: unused)
    void *out;
    float *lse;  // [batch][hq] or nullptr
    HeadStrides sq, sk, sv, spk, spv, so;
    int64_t k_batch, v_batch;  // elements from one request's cache to the next
    HeadShape shape;
    const int32_t *lens;  // [batch]
    int64_t batch, room, prefix;
    float scale;
};
// Largest number of key splits of the tensor-core kernel.
constexpr int kMaxSplits = 64;

// The prefix phase of a decode call on the tensor cores: normalised fp32 partial rows
// [splits][batch * hq][d] and their log2 denominators [splits][batch * hq].
int attn_prefix_splits(const DecodeArgs &a);
cudaError_t launch_attn_prefix(const DecodeArgs &a, qmm_float t, int splits, float *part, float *part_lse, void *ws,
                               cudaStream_t st);
// Whether a kernel of the two files has given up a wait on the current device since the last call.
cudaError_t attn_tc_take_gave_up(bool *yes, cudaStream_t st);
cudaError_t attn_decode_take_gave_up(bool *yes, cudaStream_t st);
size_t attn_decode_workspace_bytes(const DecodeArgs &a);
cudaError_t launch_attn_decode(const DecodeArgs &a, qmm_float t, void *ws, cudaStream_t st);

}  // namespace qmm
