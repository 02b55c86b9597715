// qmm_attn_api.cu -- the attention calls of the C ABI (include/qmm.h): argument checks and
// the launchers' argument blocks.
#include <cuda_runtime.h>

#include <cmath>

#include "qmm.h"
#include "qmm_attn.h"
#include "qmm_internal.h"

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

qmm_status qmm_take_attn_error(int32_t *status, void *stream) {
    if (!status) return QMM_ERR_ARG;
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    bool prompt = false, decode = false;
    const cudaError_t e = attn_tc_take_gave_up(&prompt, st), f = attn_decode_take_gave_up(&decode, st);
    *status = prompt || decode ? QMM_ERR_DEVICE : QMM_OK;
    return cuda_status(e != cudaSuccess ? e : f);
}

}  // extern "C"
