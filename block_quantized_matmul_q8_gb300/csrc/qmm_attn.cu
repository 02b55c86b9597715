// qmm_attn.cu -- attention of a decoding batch.
//
//   out = sum_j p_j v_j,  p = softmax_j(scale q.k_j) over the keys that the row sees.
//
// One warp takes one (query token, query head) row and streams its keys in one pass with a
// running maximum and sum (fp32): lane l holds the elements 4l..4l+3 of q, of each key and of
// the output.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <algorithm>

#include "qmm_attn.h"
#include "qmm_internal.h"

namespace qmm {

namespace {

constexpr int kRowWarps = 4;
constexpr int kBatch = 4;  // keys of one step

__device__ __forceinline__ float4 load4(const __half *p) {
    const uint2 u = *reinterpret_cast<const uint2 *>(p);
    const float2 a = __half22float2(*reinterpret_cast<const __half2 *>(&u.x));
    const float2 b = __half22float2(*reinterpret_cast<const __half2 *>(&u.y));
    return make_float4(a.x, a.y, b.x, b.y);
}
__device__ __forceinline__ float4 load4(const __nv_bfloat16 *p) {
    const uint2 u = *reinterpret_cast<const uint2 *>(p);
    return make_float4(__uint_as_float(u.x << 16), __uint_as_float(u.x & 0xffff0000u), __uint_as_float(u.y << 16),
                       __uint_as_float(u.y & 0xffff0000u));
}
__device__ __forceinline__ void store4(__half *p, float4 v) {
    p[0] = __float2half_rn(v.x);
    p[1] = __float2half_rn(v.y);
    p[2] = __float2half_rn(v.z);
    p[3] = __float2half_rn(v.w);
}
__device__ __forceinline__ void store4(__nv_bfloat16 *p, float4 v) {
    p[0] = __float2bfloat16_rn(v.x);
    p[1] = __float2bfloat16_rn(v.y);
    p[2] = __float2bfloat16_rn(v.z);
    p[3] = __float2bfloat16_rn(v.w);
}

// The running softmax of one row: maximum of scale*q.k so far, sum of exp(score - top), and
// the weighted sum of the values (this lane's four elements).
struct Row {
    float top = -INFINITY, sum = 0.f;
    float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
};

template <typename T>
__device__ __forceinline__ void take_keys(Row &s, float4 q, const T *k, const T *v, int64_t k_stride,
                                          int64_t v_stride, int64_t n, bool live) {
    const float4 zero = make_float4(0.f, 0.f, 0.f, 0.f);
    for (int64_t j = 0; j < n; j += kBatch) {
        float z[kBatch];
        float4 vv[kBatch];
#pragma unroll
        for (int i = 0; i < kBatch; ++i) {
            const bool on = live && j + i < n;
            const float4 kk = on ? load4(k + (j + i) * k_stride) : zero;
            vv[i] = on ? load4(v + (j + i) * v_stride) : zero;
            z[i] = q.x * kk.x + q.y * kk.y + q.z * kk.z + q.w * kk.w;
        }
#pragma unroll
        for (int i = 0; i < kBatch; ++i) {
            for (int o = 16; o > 0; o >>= 1) z[i] += __shfl_xor_sync(0xffffffffu, z[i], o);
            if (j + i >= n) z[i] = -INFINITY;
        }
        float top = s.top;
#pragma unroll
        for (int i = 0; i < kBatch; ++i) top = fmaxf(top, z[i]);
        const float base = top == -INFINITY ? 0.f : top;
        const float f = expf(s.top - base);
        s.sum *= f;
        s.acc = make_float4(s.acc.x * f, s.acc.y * f, s.acc.z * f, s.acc.w * f);
#pragma unroll
        for (int i = 0; i < kBatch; ++i) {
            if (j + i >= n) continue;
            const float p = expf(z[i] - base);
            s.sum += p;
            s.acc.x += p * vv[i].x;
            s.acc.y += p * vv[i].y;
            s.acc.z += p * vv[i].z;
            s.acc.w += p * vv[i].w;
        }
        s.top = top;
    }
}

template <typename T> __device__ __forceinline__ void finish(const Row &s, T *out, float *lse, int lane, bool live) {
    const float inv = s.sum == 0.f ? 0.f : 1.f / s.sum;
    if (live) store4(out, make_float4(s.acc.x * inv, s.acc.y * inv, s.acc.z * inv, s.acc.w * inv));
    if (lse && lane == 0) *lse = s.sum == 0.f ? -INFINITY : s.top + logf(s.sum);
}

__device__ __forceinline__ float4 scaled(float4 q, float f) { return make_float4(q.x * f, q.y * f, q.z * f, q.w * f); }

template <typename T> __global__ void __launch_bounds__(kRowWarps * 32) decode_rows_kernel(const DecodeArgs a) {
    const int lane = threadIdx.x & 31, h = blockIdx.y;
    const int64_t b = int64_t(blockIdx.x) * kRowWarps + (threadIdx.x >> 5);
    if (b >= a.batch) return;
    const bool live = 4 * lane < a.shape.d;
    const int hk = h / (a.shape.hq / a.shape.hk);
    const float4 q = live ? scaled(load4(static_cast<const T *>(a.q) + b * a.sq.t + h * a.sq.h + 4 * lane), a.scale)
                          : make_float4(0.f, 0.f, 0.f, 0.f);
    Row row;
    if (a.prefix > 0)
        take_keys(row, q, static_cast<const T *>(a.pk) + hk * a.spk.h + 4 * lane,
                  static_cast<const T *>(a.pv) + hk * a.spv.h + 4 * lane, a.spk.t, a.spv.t, a.prefix, live);
    const int64_t n = a.room > 0 ? min(max(int64_t(a.lens[b]), int64_t(0)), a.room) : 0;
    if (n > 0)
        take_keys(row, q, static_cast<const T *>(a.k) + b * a.k_batch + hk * a.sk.h + 4 * lane,
                  static_cast<const T *>(a.v) + b * a.v_batch + hk * a.sv.h + 4 * lane, a.sk.t, a.sv.t, n, live);
    finish(row, static_cast<T *>(a.out) + b * a.so.t + h * a.so.h + 4 * lane,
           a.lse ? a.lse + b * a.shape.hq + h : nullptr, lane, live);
}

}  // namespace

size_t attn_decode_workspace_bytes(const DecodeArgs &) { return 256; }

cudaError_t launch_attn_decode(const DecodeArgs &a, qmm_float t, void *ws, cudaStream_t st) {
    cudaError_t e = cudaMemsetAsync(ws, 0, 16, st);
    if (e != cudaSuccess) return e;
    const dim3 grid((unsigned)((a.batch + kRowWarps - 1) / kRowWarps), (unsigned)a.shape.hq);
    if (t == QMM_F16) decode_rows_kernel<__half><<<grid, kRowWarps * 32, 0, st>>>(a);
    else decode_rows_kernel<__nv_bfloat16><<<grid, kRowWarps * 32, 0, st>>>(a);
    return cudaGetLastError();
}

}  // namespace qmm
