// qmm_attn_api.cu -- the attention calls of the C ABI (include/qmm.h): argument checks and
// the launchers' argument blocks.
#include <cuda_runtime.h>

#include <algorithm>
#include <cmath>

#include "qmm.h"
#include "qmm_attn.h"
#include "qmm_internal.h"
#include "qmm_kv.h"

using namespace qmm;

namespace {

constexpr int64_t kMaxTokens = (int64_t(1) << 31) - 1024;  // a tile past the last token still counts in 32 bits
constexpr int64_t kMaxHeads = 4096;
constexpr int64_t kMaxSeqs = int64_t(1) << 20;
constexpr int64_t kMaxGroup = 128;  // query heads of one key/value head
constexpr int64_t kMaxStride = (int64_t(1) << 38) - 1;  // below the 2^40 bytes of a tensor map

bool aligned_to(const void *p, uintptr_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }
bool is_16bit(qmm_float t) { return t == QMM_F16 || t == QMM_BF16; }

qmm_status check_heads(int64_t hq, int64_t hk, int64_t d) {
    if (hq <= 0 || hk <= 0 || d <= 0) return QMM_ERR_ARG;
    if (hq % hk || d % 8 || d > kMaxHeadDim || hq > kMaxHeads || hq / hk > kMaxGroup) return QMM_ERR_SHAPE;
    return QMM_OK;
}

// A view of `tokens` tokens of `heads` heads of d `size`-byte elements.
qmm_status check_view(const qmm_heads *x, int64_t tokens, int64_t heads, int64_t d, int size) {
    if (!x || !x->data) return QMM_ERR_ARG;
    if (!aligned_to(x->data, 16)) return QMM_ERR_ALIGN;
    const int64_t unit = 16 / size;
    if ((tokens > 1 && x->token_stride % unit) || (heads > 1 && x->head_stride % unit)) return QMM_ERR_ALIGN;
    if ((tokens > 1 && (x->token_stride < d || x->token_stride > kMaxStride)) ||
        (heads > 1 && (x->head_stride < d || x->head_stride > kMaxStride)))
        return QMM_ERR_SHAPE;
    return QMM_OK;
}

// The strides that a view's tokens and heads take; 0 for one that is never taken.
HeadStrides strides(const qmm_heads *x, int64_t tokens, int64_t heads) {
    return {tokens > 1 ? x->token_stride : 0, heads > 1 ? x->head_stride : 0};
}

qmm_status check_workspace(const void *ws, size_t bytes, size_t need) {
    if (!ws || bytes < need) return QMM_ERR_WORKSPACE;
    return aligned_to(ws, 256) ? QMM_OK : QMM_ERR_ALIGN;
}

qmm_status cuda_status(cudaError_t e) { return e == cudaSuccess ? QMM_OK : QMM_ERR_CUDA; }

qmm_status prompt_sizes(PromptArgs &a, int64_t tokens_q, int64_t tokens_k, int64_t n_seqs, int64_t hq, int64_t hk,
                        int64_t d) {
    if (tokens_q < 0 || tokens_k < 0 || n_seqs < 0) return QMM_ERR_ARG;
    const qmm_status s = check_heads(hq, hk, d);
    if (s != QMM_OK) return s;
    if (tokens_q > kMaxTokens || tokens_k > kMaxTokens || n_seqs > kMaxSeqs) return QMM_ERR_SHAPE;
    a.shape = {(int)hq, (int)hk, (int)d};
    a.n_seqs = n_seqs;
    a.tokens_q = tokens_q;
    a.tokens_k = tokens_k;
    return QMM_OK;
}

qmm_status decode_sizes(DecodeArgs &a, int64_t batch, int64_t room, int64_t prefix, int64_t hq, int64_t hk,
                        int64_t d) {
    if (batch < 0 || room < 0 || prefix < 0) return QMM_ERR_ARG;
    const qmm_status s = check_heads(hq, hk, d);
    if (s != QMM_OK) return s;
    if (batch > kMaxTokens || room > kMaxTokens || prefix > kMaxTokens) return QMM_ERR_SHAPE;
    a.shape = {(int)hq, (int)hk, (int)d};
    a.batch = batch;
    a.room = room;
    a.prefix = prefix;
    return QMM_OK;
}

// A cache of heads_kv heads of d elements; fills c.
qmm_status check_cache(const qmm_kv_cache *x, int64_t hk, int64_t d, KvCache &c) {
    if (!x) return QMM_ERR_ARG;
    if (x->type != QMM_Q4_0 && x->type != QMM_Q8_0) return QMM_ERR_TYPE;
    if (x->n_pages < 0) return QMM_ERR_ARG;
    const size_t bytes = qmm_kv_page_bytes((qmm_type)x->type, x->page_size, hk, d);
    if (bytes == 0 || x->n_pages > 0x7fffffff / x->page_size) return QMM_ERR_SHAPE;
    if (x->n_pages > 0) {
        if (!x->pages) return QMM_ERR_ARG;
        if (!aligned_to(x->pages, 16) || (x->n_pages > 1 && x->page_stride % 16)) return QMM_ERR_ALIGN;
        if (x->n_pages > 1 && (x->page_stride < (int64_t)bytes || x->page_stride > kMaxStride)) return QMM_ERR_SHAPE;
    }
    c.pages = static_cast<uint8_t *>(x->pages);
    c.page_stride = x->page_stride;
    c.n_pages = x->n_pages;
    c.q8 = x->type == QMM_Q8_0;
    c.page_log2 = 4;
    while ((1 << c.page_log2) < x->page_size) ++c.page_log2;
    return QMM_OK;
}

// A table of pages, [rows][width] int32 with `stride` entries from row to row.
qmm_status check_table(const int32_t *table, int64_t rows, int64_t width, int64_t stride) {
    if (width < 0) return QMM_ERR_ARG;
    if (width > kMaxTokens || (rows > 1 && (stride < width || stride > kMaxStride))) return QMM_ERR_SHAPE;
    if (rows > 0 && width > 0 && !table) return QMM_ERR_ARG;
    return aligned_to(table, 4) ? QMM_OK : QMM_ERR_ALIGN;
}

qmm_status kv_decode_sizes(KvDecodeArgs &a, int64_t batch, int64_t max_len, int64_t hq, int64_t hk, int64_t d) {
    if (batch < 0 || max_len < 0) return QMM_ERR_ARG;
    const qmm_status s = check_heads(hq, hk, d);
    if (s != QMM_OK) return s;
    if (d % 32 || batch > kMaxTokens || max_len > kMaxTokens) return QMM_ERR_SHAPE;
    a.shape = {(int)hq, (int)hk, (int)d};
    a.batch = batch;
    a.max_len = max_len;
    return QMM_OK;
}

}  // namespace

extern "C" {

qmm_status qmm_qk_norm_rope(const qmm_heads *q, const qmm_heads *k, const qmm_heads *v, qmm_float in_type, int64_t m,
                            int64_t heads_q, int64_t heads_kv, int64_t head_dim, const float *w_q, const float *w_k,
                            float eps, const int32_t *positions, const float *inv_freq, int64_t rotary_dim,
                            int interleaved, const qmm_heads *q_out, const qmm_heads *k_out, const qmm_heads *v_out,
                            qmm_float out_type, void *stream) {
    if (in_type != QMM_F32 && !is_16bit(in_type)) return QMM_ERR_TYPE;
    if (!is_16bit(out_type)) return QMM_ERR_TYPE;
    if (m < 0 || rotary_dim < 0 || heads_q <= 0 || heads_kv <= 0 || head_dim <= 0 || !(eps >= 0.f)) return QMM_ERR_ARG;
    if (m > kMaxTokens || heads_q > kMaxHeads || heads_kv > kMaxHeads || head_dim % 8 || head_dim > kMaxHeadDim ||
        rotary_dim % 8 || rotary_dim > head_dim)
        return QMM_ERR_SHAPE;
    if (!v != !v_out) return QMM_ERR_ARG;
    if (m == 0) return QMM_OK;
    const int in_size = in_type == QMM_F32 ? 4 : 2;
    qmm_status s;
    if ((s = check_view(q, m, heads_q, head_dim, in_size)) != QMM_OK || (s = check_view(k, m, heads_kv, head_dim, in_size)) != QMM_OK ||
        (s = check_view(q_out, m, heads_q, head_dim, 2)) != QMM_OK || (s = check_view(k_out, m, heads_kv, head_dim, 2)) != QMM_OK)
        return s;
    if (v && ((s = check_view(v, m, heads_kv, head_dim, in_size)) != QMM_OK || (s = check_view(v_out, m, heads_kv, head_dim, 2)) != QMM_OK))
        return s;
    if (rotary_dim > 0 && (!positions || !inv_freq)) return QMM_ERR_ARG;
    if (!aligned_to(positions, 4) || !aligned_to(inv_freq, 4) || !aligned_to(w_q, 4) || !aligned_to(w_k, 4))
        return QMM_ERR_ALIGN;
    RopeArgs a{};
    a.q = q->data;
    a.k = k->data;
    a.qo = q_out->data;
    a.ko = k_out->data;
    a.sq = strides(q, m, heads_q);
    a.sk = strides(k, m, heads_kv);
    a.sqo = strides(q_out, m, heads_q);
    a.sko = strides(k_out, m, heads_kv);
    if (v) {
        a.v = v->data;
        a.vo = v_out->data;
        a.sv = strides(v, m, heads_kv);
        a.svo = strides(v_out, m, heads_kv);
    }
    a.shape = {(int)heads_q, (int)heads_kv, (int)head_dim};
    a.wq = w_q;
    a.wk = w_k;
    a.positions = positions;
    a.inv_freq = inv_freq;
    a.rotary = (int)rotary_dim;
    a.interleaved = interleaved != 0;
    a.eps = eps;
    a.m = m;
    return cuda_status(launch_qk_norm_rope(a, in_type, out_type, static_cast<cudaStream_t>(stream)));
}

size_t qmm_workspace_bytes_attn_prompt(int64_t tokens_q, int64_t tokens_k, int64_t n_seqs, int64_t heads_q,
                                       int64_t heads_kv, int64_t head_dim) {
    PromptArgs a{};
    if (prompt_sizes(a, tokens_q, tokens_k, n_seqs, heads_q, heads_kv, head_dim) != QMM_OK) return 0;
    return attn_prompt_workspace_bytes(a);
}

qmm_status qmm_attn_prompt(const qmm_heads *q, const qmm_heads *k, const qmm_heads *v, qmm_float t, int64_t tokens_q,
                           int64_t tokens_k, int64_t heads_q, int64_t heads_kv, int64_t head_dim, const int32_t *cu_q,
                           const int32_t *cu_k, int64_t n_seqs, int causal, float scale, const qmm_heads *out,
                           float *lse, void *workspace, size_t ws_bytes, void *stream) {
    if (!is_16bit(t)) return QMM_ERR_TYPE;
    PromptArgs a{};
    qmm_status s = prompt_sizes(a, tokens_q, tokens_k, n_seqs, heads_q, heads_kv, head_dim);
    if (s != QMM_OK) return s;
    if (!std::isfinite(scale)) return QMM_ERR_ARG;
    if ((s = check_workspace(workspace, ws_bytes, attn_prompt_workspace_bytes(a))) != QMM_OK) return s;
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    if (tokens_q == 0 || n_seqs == 0) return cuda_status(cudaMemsetAsync(workspace, 0, 16, st));
    if ((s = check_view(q, tokens_q, heads_q, head_dim, 2)) != QMM_OK || (s = check_view(out, tokens_q, heads_q, head_dim, 2)) != QMM_OK)
        return s;
    if (tokens_k > 0 &&
        ((s = check_view(k, tokens_k, heads_kv, head_dim, 2)) != QMM_OK || (s = check_view(v, tokens_k, heads_kv, head_dim, 2)) != QMM_OK))
        return s;
    if (!cu_q || !cu_k) return QMM_ERR_ARG;
    if (!aligned_to(cu_q, 4) || !aligned_to(cu_k, 4) || !aligned_to(lse, 4)) return QMM_ERR_ALIGN;
    a.q = q->data;
    a.out = out->data;
    a.sq = strides(q, tokens_q, heads_q);
    a.so = strides(out, tokens_q, heads_q);
    if (tokens_k > 0) {
        a.k = k->data;
        a.v = v->data;
        a.sk = strides(k, tokens_k, heads_kv);
        a.sv = strides(v, tokens_k, heads_kv);
    }
    a.lse = lse;
    a.cu_q = cu_q;
    a.cu_k = cu_k;
    a.causal = causal != 0;
    a.scale = scale;
    return cuda_status(launch_attn_prompt(a, t, workspace, st));
}

size_t qmm_workspace_bytes_attn_decode(int64_t batch, int64_t room, int64_t prefix_len, int64_t heads_q,
                                       int64_t heads_kv, int64_t head_dim) {
    DecodeArgs a{};
    if (decode_sizes(a, batch, room, prefix_len, heads_q, heads_kv, head_dim) != QMM_OK) return 0;
    return attn_decode_workspace_bytes(a);
}

qmm_status qmm_attn_decode(const qmm_heads *q, const qmm_heads *k, const qmm_heads *v, int64_t k_batch_stride,
                           int64_t v_batch_stride, const int32_t *lens, int64_t batch, int64_t room,
                           const qmm_heads *prefix_k, const qmm_heads *prefix_v, int64_t prefix_len, qmm_float t,
                           int64_t heads_q, int64_t heads_kv, int64_t head_dim, float scale, const qmm_heads *out,
                           float *lse, void *workspace, size_t ws_bytes, void *stream) {
    if (!is_16bit(t)) return QMM_ERR_TYPE;
    DecodeArgs a{};
    qmm_status s = decode_sizes(a, batch, room, prefix_len, heads_q, heads_kv, head_dim);
    if (s != QMM_OK) return s;
    if (!std::isfinite(scale)) return QMM_ERR_ARG;
    if ((s = check_workspace(workspace, ws_bytes, attn_decode_workspace_bytes(a))) != QMM_OK) return s;
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    if (batch == 0) return cuda_status(cudaMemsetAsync(workspace, 0, 16, st));
    if ((s = check_view(q, batch, heads_q, head_dim, 2)) != QMM_OK || (s = check_view(out, batch, heads_q, head_dim, 2)) != QMM_OK) return s;
    if (room > 0) {
        if ((s = check_view(k, room, heads_kv, head_dim, 2)) != QMM_OK || (s = check_view(v, room, heads_kv, head_dim, 2)) != QMM_OK)
            return s;
        if (!lens) return QMM_ERR_ARG;
        if (!aligned_to(lens, 4)) return QMM_ERR_ALIGN;
        if (batch > 1 && (k_batch_stride % 8 || v_batch_stride % 8)) return QMM_ERR_ALIGN;
        if (batch > 1 && (k_batch_stride < head_dim || v_batch_stride < head_dim || k_batch_stride > kMaxStride ||
                          v_batch_stride > kMaxStride))
            return QMM_ERR_SHAPE;
    }
    if (prefix_len > 0 && ((s = check_view(prefix_k, prefix_len, heads_kv, head_dim, 2)) != QMM_OK ||
                           (s = check_view(prefix_v, prefix_len, heads_kv, head_dim, 2)) != QMM_OK))
        return s;
    if (!aligned_to(lse, 4)) return QMM_ERR_ALIGN;
    a.q = q->data;
    a.out = out->data;
    a.sq = strides(q, batch, heads_q);
    a.so = strides(out, batch, heads_q);
    if (room > 0) {
        a.k = k->data;
        a.v = v->data;
        a.sk = strides(k, room, heads_kv);
        a.sv = strides(v, room, heads_kv);
        a.k_batch = batch > 1 ? k_batch_stride : 0;
        a.v_batch = batch > 1 ? v_batch_stride : 0;
        a.lens = lens;
    }
    if (prefix_len > 0) {
        a.pk = prefix_k->data;
        a.pv = prefix_v->data;
        a.spk = strides(prefix_k, prefix_len, heads_kv);
        a.spv = strides(prefix_v, prefix_len, heads_kv);
    }
    a.lse = lse;
    a.scale = scale;
    return cuda_status(launch_attn_decode(a, t, workspace, st));
}

size_t qmm_kv_page_bytes(qmm_type t, int64_t page_size, int64_t heads_kv, int64_t head_dim) {
    if (t != QMM_Q4_0 && t != QMM_Q8_0) return 0;
    if (page_size < kKvGroup || page_size > 256 || (page_size & (page_size - 1))) return 0;
    if (heads_kv <= 0 || heads_kv > kMaxHeads || head_dim <= 0 || head_dim % 32 || head_dim > kMaxHeadDim) return 0;
    return size_t(heads_kv) * (page_size / kKvGroup) * kv_record_bytes(t == QMM_Q8_0, (int)head_dim);
}

qmm_status qmm_kv_append(const qmm_heads *q, const qmm_heads *k, const qmm_heads *v, qmm_float in_type, int64_t m,
                         int64_t heads_q, int64_t heads_kv, int64_t head_dim, const float *w_q, const float *w_k,
                         float eps, const int32_t *positions, const float *inv_freq, int64_t rotary_dim,
                         int interleaved, const qmm_kv_cache *cache, const int32_t *slots, const qmm_heads *q_out,
                         const qmm_heads *k_out, const qmm_heads *v_out, qmm_float out_type, void *stream) {
    if (in_type != QMM_F32 && !is_16bit(in_type)) return QMM_ERR_TYPE;
    if (!is_16bit(out_type)) return QMM_ERR_TYPE;
    if (!q != !q_out || !k_out != !v_out) return QMM_ERR_ARG;
    if (m < 0 || rotary_dim < 0 || (q && heads_q <= 0) || heads_kv <= 0 || head_dim <= 0 || !(eps >= 0.f)) return QMM_ERR_ARG;
    if (m > kMaxTokens || (q && heads_q > kMaxHeads) || heads_kv > kMaxHeads || head_dim % 32 || head_dim > kMaxHeadDim ||
        rotary_dim % 8 || rotary_dim > head_dim)
        return QMM_ERR_SHAPE;
    KvAppendArgs a{};
    RopeArgs &r = a.rope;
    qmm_status s = check_cache(cache, heads_kv, head_dim, a.cache);
    if (s != QMM_OK) return s;
    if (m == 0) return QMM_OK;
    const int in_size = in_type == QMM_F32 ? 4 : 2;
    if (q && ((s = check_view(q, m, heads_q, head_dim, in_size)) != QMM_OK || (s = check_view(q_out, m, heads_q, head_dim, 2)) != QMM_OK))
        return s;
    if ((s = check_view(k, m, heads_kv, head_dim, in_size)) != QMM_OK || (s = check_view(v, m, heads_kv, head_dim, in_size)) != QMM_OK)
        return s;
    if (k_out && ((s = check_view(k_out, m, heads_kv, head_dim, 2)) != QMM_OK || (s = check_view(v_out, m, heads_kv, head_dim, 2)) != QMM_OK))
        return s;
    if (!slots || (rotary_dim > 0 && (!positions || !inv_freq))) return QMM_ERR_ARG;
    if (!aligned_to(positions, 4) || !aligned_to(inv_freq, 4) || !aligned_to(w_q, 4) || !aligned_to(w_k, 4) || !aligned_to(slots, 4))
        return QMM_ERR_ALIGN;
    if (q) {
        r.q = q->data;
        r.qo = q_out->data;
        r.sq = strides(q, m, heads_q);
        r.sqo = strides(q_out, m, heads_q);
    }
    r.k = k->data;
    r.v = v->data;
    r.sk = strides(k, m, heads_kv);
    r.sv = strides(v, m, heads_kv);
    if (k_out) {
        r.ko = k_out->data;
        r.vo = v_out->data;
        r.sko = strides(k_out, m, heads_kv);
        r.svo = strides(v_out, m, heads_kv);
    }
    r.shape = {q ? (int)heads_q : 0, (int)heads_kv, (int)head_dim};
    r.wq = w_q;
    r.wk = w_k;
    r.positions = positions;
    r.inv_freq = inv_freq;
    r.rotary = (int)rotary_dim;
    r.interleaved = interleaved != 0;
    r.eps = eps;
    r.m = m;
    a.slots = slots;
    return cuda_status(launch_kv_append(a, in_type, out_type, static_cast<cudaStream_t>(stream)));
}

qmm_status qmm_kv_read(const qmm_kv_cache *cache, const int32_t *table, int64_t table_width, int64_t table_stride,
                       const int32_t *cu_k, int64_t n_seqs, int64_t tokens, int64_t heads_kv, int64_t head_dim,
                       const qmm_heads *k_out, const qmm_heads *v_out, qmm_float out_type, void *stream) {
    if (!is_16bit(out_type)) return QMM_ERR_TYPE;
    if (n_seqs < 0 || tokens < 0 || heads_kv <= 0 || head_dim <= 0) return QMM_ERR_ARG;
    if (n_seqs > kMaxSeqs || tokens > kMaxTokens || heads_kv > kMaxHeads || head_dim % 32 || head_dim > kMaxHeadDim)
        return QMM_ERR_SHAPE;
    KvReadArgs a{};
    qmm_status s = check_cache(cache, heads_kv, head_dim, a.cache);
    if (s != QMM_OK || (s = check_table(table, n_seqs, table_width, table_stride)) != QMM_OK) return s;
    if (n_seqs == 0 || tokens == 0) return QMM_OK;
    if ((s = check_view(k_out, tokens, heads_kv, head_dim, 2)) != QMM_OK || (s = check_view(v_out, tokens, heads_kv, head_dim, 2)) != QMM_OK)
        return s;
    if (!cu_k) return QMM_ERR_ARG;
    if (!aligned_to(cu_k, 4)) return QMM_ERR_ALIGN;
    a.table = table;
    a.table_stride = n_seqs > 1 ? table_stride : 0;
    a.table_width = table_width;
    a.cu = cu_k;
    a.n_seqs = n_seqs;
    a.tokens = tokens;
    a.hk = (int)heads_kv;
    a.d = (int)head_dim;
    a.ko = k_out->data;
    a.vo = v_out->data;
    a.sko = strides(k_out, tokens, heads_kv);
    a.svo = strides(v_out, tokens, heads_kv);
    return cuda_status(launch_kv_read(a, out_type, static_cast<cudaStream_t>(stream)));
}

size_t qmm_workspace_bytes_attn_decode_kv(int64_t batch, int64_t max_len, int64_t heads_q, int64_t heads_kv,
                                          int64_t head_dim) {
    KvDecodeArgs a{};
    if (kv_decode_sizes(a, batch, max_len, heads_q, heads_kv, head_dim) != QMM_OK || batch == 0) return 0;
    return kv_decode_workspace_bytes(a);
}

qmm_status qmm_attn_decode_kv(const qmm_heads *q, const qmm_kv_cache *cache, const int32_t *table, int64_t table_width,
                              int64_t table_stride, const int32_t *lens, int64_t batch, int64_t max_len, qmm_float t,
                              int64_t heads_q, int64_t heads_kv, int64_t head_dim, float scale, const qmm_heads *out,
                              float *lse, void *workspace, size_t ws_bytes, void *stream) {
    if (!is_16bit(t)) return QMM_ERR_TYPE;
    KvDecodeArgs a{};
    qmm_status s = kv_decode_sizes(a, batch, max_len, heads_q, heads_kv, head_dim);
    if (s != QMM_OK) return s;
    if (!std::isfinite(scale)) return QMM_ERR_ARG;
    if ((s = check_cache(cache, heads_kv, head_dim, a.cache)) != QMM_OK) return s;
    if ((s = check_table(table, batch, table_width, table_stride)) != QMM_OK) return s;
    if (max_len > table_width << a.cache.page_log2) return QMM_ERR_SHAPE;
    if (batch == 0) return QMM_OK;
    const size_t need = kv_decode_workspace_bytes(a);
    if (need > 0 && (s = check_workspace(workspace, ws_bytes, need)) != QMM_OK) return s;
    if ((s = check_view(q, batch, heads_q, head_dim, 2)) != QMM_OK || (s = check_view(out, batch, heads_q, head_dim, 2)) != QMM_OK)
        return s;
    if (!lens) return QMM_ERR_ARG;
    if (!aligned_to(lens, 4) || !aligned_to(lse, 4)) return QMM_ERR_ALIGN;
    a.q = q->data;
    a.out = out->data;
    a.lse = lse;
    a.sq = strides(q, batch, heads_q);
    a.so = strides(out, batch, heads_q);
    a.table = table;
    a.table_stride = batch > 1 ? table_stride : 0;
    a.lens = lens;
    a.scale = scale;
    return cuda_status(launch_kv_decode(a, t, workspace, static_cast<cudaStream_t>(stream)));
}

qmm_status qmm_take_attn_error(int32_t *status, void *stream) {
    if (!status) return QMM_ERR_ARG;
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    int worst = QMM_OK;  // QMM_ERR_DEVICE over QMM_ERR_IDS
    cudaError_t failed = cudaSuccess;
    for (auto take : {attn_tc_take_error, attn_decode_take_error, kv_take_error, kv_decode_take_error}) {
        int code = QMM_OK;
        const cudaError_t e = take(&code, st);
        if (failed == cudaSuccess) failed = e;
        worst = std::max(worst, code);
    }
    *status = worst;
    return cuda_status(failed);
}

}  // extern "C"
