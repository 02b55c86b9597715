// qmm_kv.h -- the paged key/value cache in 4 or 8 bits: its layout and the launchers of its calls.
//
// A page holds page_size tokens of heads_kv heads as [head][group of 16 tokens][record].  A record is
// one bulk copy: the 16 tokens' key codes, key scales, value codes and value scales.  Codes lie
// as [16-byte unit of a head][token][16 bytes], so that eight tokens of a unit are the 128
// consecutive bytes that one ldmatrix phase reads without bank conflicts, and no byte holds two
// tokens, so that tokens are written without reading.  Scales lie as [block of 32][place of the token], the places of
// tokens 2t, 2t + 1, 2t + 8, 2t + 9 side by side: the four that a lane of the MMA fragments needs are one load.
#pragma once
#include <cuda_runtime.h>
#include <stdint.h>

#include "qmm.h"
#include "qmm_attn.h"

namespace qmm {

constexpr int kKvGroup = 16;  // tokens of a record

// Bytes of one side (keys or values) of a record, and where its scales start.
__host__ __device__ constexpr int kv_unit_elems(bool q8) { return q8 ? 16 : 32; }
__host__ __device__ constexpr int kv_scales_at(bool q8, int d) { return d / kv_unit_elems(q8) * 256; }
__host__ __device__ constexpr int kv_side_bytes(bool q8, int d) { return kv_scales_at(q8, d) + d / 32 * 32; }
__host__ __device__ constexpr int kv_record_bytes(bool q8, int d) { return 2 * kv_side_bytes(q8, d); }
// Place of token 0..15 of a group among the scales of a block.
__host__ __device__ constexpr int kv_scale_place(int token) {
    return (token & 7) / 2 * 4 + (token & 1) + 2 * (token >> 3);
}

struct KvCache {
    uint8_t *pages;
    int64_t page_stride;  // bytes
    int64_t n_pages;
    int page_log2;        // log2 of the tokens of a page
    int q8;               // Q8_0, else Q4_0
};

struct KvAppendArgs {
    RopeArgs rope;        // q may be null; ko, vo: the values the cache stands for, or null
    KvCache cache;
    const int32_t *slots; // [m]
};
cudaError_t launch_kv_append(const KvAppendArgs &a, qmm_float in_type, qmm_float out_type, cudaStream_t st);

struct KvReadArgs {
    KvCache cache;
    const int32_t *table;  // [n_seqs][table_stride]
    int64_t table_stride, table_width;
    const int32_t *cu;     // [n_seqs + 1]
    int64_t n_seqs, tokens;
    int hk, d;
    void *ko, *vo;
    HeadStrides sko, svo;
};
cudaError_t launch_kv_read(const KvReadArgs &a, qmm_float out_type, cudaStream_t st);

struct KvDecodeArgs {
    const void *q;
    void *out;
    float *lse;  // [batch][hq] or nullptr
    HeadStrides sq, so;
    HeadShape shape;
    KvCache cache;
    const int32_t *table;  // [batch][table_stride]
    int64_t table_stride;
    const int32_t *lens;   // [batch]
    int64_t batch, max_len;
    float scale;
};
size_t kv_decode_workspace_bytes(const KvDecodeArgs &a);
cudaError_t launch_kv_decode(const KvDecodeArgs &a, qmm_float t, void *ws, cudaStream_t st);

// QMM_OK, or what a kernel of the file has reported on the current device since the last call.
cudaError_t kv_take_error(int *code, cudaStream_t st);         // pages outside the cache
cudaError_t kv_decode_take_error(int *code, cudaStream_t st);  // the same, or a wait that gave up

}  // namespace qmm
