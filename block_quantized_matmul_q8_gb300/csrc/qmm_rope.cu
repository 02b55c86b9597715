// qmm_rope.cu -- RMS norm of query and key heads, rotation by position and rounding to 16
// bits, one pass over the qkv product:
//   n = x * w / sqrt(mean(x^2) + eps),  (a, b) -> (a cos - b sin, b cos + a sin).
//
// Bound by HBM: each element is read once and written once.  One block takes one token (or a
// share of its heads when there are few tokens); its first threads compute the token's
// rotary/2 angles once for all heads while the first heads are being loaded.  Four
// consecutive elements sit in one lane, so that a head's sum of squares is a shuffle
// reduction over at most 32 lanes and the partner half of a rotated pair is one shuffle away.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <algorithm>

#include "qmm_attn.h"
#include "qmm_internal.h"

namespace qmm {

namespace {

constexpr int kRopeThreads = 256;
constexpr int kRopeWarps = kRopeThreads / 32;
constexpr int kRopeBatch = 4;  // heads whose loads a warp has in flight

__device__ __forceinline__ float4 load4(const float *p) { return *reinterpret_cast<const float4 *>(p); }
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
    const __half2 a = __floats2half2_rn(v.x, v.y), b = __floats2half2_rn(v.z, v.w);
    *reinterpret_cast<uint2 *>(p) =
        make_uint2(*reinterpret_cast<const uint32_t *>(&a), *reinterpret_cast<const uint32_t *>(&b));
}
__device__ __forceinline__ void store4(__nv_bfloat16 *p, float4 v) {
    const __nv_bfloat162 a = __floats2bfloat162_rn(v.x, v.y), b = __floats2bfloat162_rn(v.z, v.w);
    *reinterpret_cast<uint2 *>(p) =
        make_uint2(*reinterpret_cast<const uint32_t *>(&a), *reinterpret_cast<const uint32_t *>(&b));
}

template <typename In, typename Out>
__global__ void __launch_bounds__(kRopeThreads) qk_norm_rope_kernel(const RopeArgs a, int lanes_log2, int share) {
    __shared__ float2 cs[kMaxHeadDim / 2];
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int64_t t = blockIdx.x;
    const int d = a.shape.d, hq = a.shape.hq, hk = a.shape.hk, r = a.rotary;
    const int lanes = 1 << lanes_log2;                // lanes of one head
    const int sub = lane >> lanes_log2, c = lane & (lanes - 1), e0 = 4 * c;
    const int per_warp = 32 >> lanes_log2;            // heads of one warp at a time
    const int total = hq + (a.v ? 2 : 1) * hk;
    const int h_begin = blockIdx.y * share, h_end = min(total, h_begin + share);
    const bool live = e0 < d;

    auto load = [&](int h) -> float4 {
        if (!live || h >= h_end) return make_float4(0.f, 0.f, 0.f, 0.f);
        const In *p;
        if (h < hq) p = static_cast<const In *>(a.q) + t * a.sq.t + h * a.sq.h;
        else if (h < hq + hk) p = static_cast<const In *>(a.k) + t * a.sk.t + (h - hq) * a.sk.h;
        else p = static_cast<const In *>(a.v) + t * a.sv.t + (h - hq - hk) * a.sv.h;
        return load4(p + e0);
    };
    float4 x[kRopeBatch];
    int h0 = h_begin + warp * per_warp + sub;
    const int step = kRopeWarps * per_warp;
#pragma unroll
    for (int i = 0; i < kRopeBatch; ++i) x[i] = load(h0 + i * step);

    if (tid < r / 2) {
        // the angle in turns, reduced in fp64: exact to about 1e-7 rad at every int32 position
        const double turns = double(a.positions[t]) * double(a.inv_freq[tid]) * 0.15915494309189533577;
        float s, co;
        sincospif(2.0f * float(turns - rint(turns)), &s, &co);
        cs[tid] = make_float2(co, s);
    }
    float4 wq = make_float4(1.f, 1.f, 1.f, 1.f), wk = wq;
    if (live && a.wq) wq = make_float4(a.wq[e0], a.wq[e0 + 1], a.wq[e0 + 2], a.wq[e0 + 3]);
    if (live && a.wk) wk = make_float4(a.wk[e0], a.wk[e0 + 1], a.wk[e0 + 2], a.wk[e0 + 3]);
    __syncthreads();

    // this lane's cosines and sines: out = n * co + partner * si, element by element
    float co[4] = {1.f, 1.f, 1.f, 1.f}, si[4] = {0.f, 0.f, 0.f, 0.f};
    int partner = lane;
    if (e0 < r) {
        if (a.interleaved) {
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                const float2 v = cs[2 * c + j];
                co[2 * j] = co[2 * j + 1] = v.x;
                si[2 * j] = -v.y;
                si[2 * j + 1] = v.y;
            }
        } else {
            const int half = r / 8;  // lanes of the first half (r is a multiple of 8)
            const bool first = c < half;
            partner = first ? lane + half : lane - half;
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const float2 v = cs[e0 + j - (first ? 0 : r / 2)];
                co[j] = v.x;
                si[j] = first ? -v.y : v.y;
            }
        }
    }
    const float inv_d = 1.0f / float(d);

    for (; h0 - sub < h_end; h0 += kRopeBatch * step) {
#pragma unroll
        for (int i = 0; i < kRopeBatch; ++i) {
            const int h = h0 + i * step;
            float4 n = x[i];
            const bool is_q = h < hq, is_k = !is_q && h < hq + hk;
            float ss = n.x * n.x + n.y * n.y + n.z * n.z + n.w * n.w;
            for (int o = lanes >> 1; o > 0; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
            if ((is_q && a.wq) || (is_k && a.wk)) {
                const float inv = rsqrtf(ss * inv_d + a.eps);
                const float4 w = is_q ? wq : wk;
                n.x = n.x * inv * w.x;
                n.y = n.y * inv * w.y;
                n.z = n.z * inv * w.z;
                n.w = n.w * inv * w.w;
            }
            float4 p;
            if (a.interleaved) {
                p = make_float4(n.y, n.x, n.w, n.z);
            } else {
                p.x = __shfl_sync(0xffffffffu, n.x, partner);
                p.y = __shfl_sync(0xffffffffu, n.y, partner);
                p.z = __shfl_sync(0xffffffffu, n.z, partner);
                p.w = __shfl_sync(0xffffffffu, n.w, partner);
            }
            if (live && h < h_end) {
                Out *out;
                if (is_q) out = static_cast<Out *>(a.qo) + t * a.sqo.t + h * a.sqo.h;
                else if (is_k) out = static_cast<Out *>(a.ko) + t * a.sko.t + (h - hq) * a.sko.h;
                else out = static_cast<Out *>(a.vo) + t * a.svo.t + (h - hq - hk) * a.svo.h;
                if ((is_q || is_k) && e0 < r) {
                    n.x = n.x * co[0] + p.x * si[0];
                    n.y = n.y * co[1] + p.y * si[1];
                    n.z = n.z * co[2] + p.z * si[2];
                    n.w = n.w * co[3] + p.w * si[3];
                }
                store4(out + e0, n);
            }
            x[i] = load(h + kRopeBatch * step);
        }
    }
}

template <typename In, typename Out> cudaError_t launch_typed(const RopeArgs &a, cudaStream_t st) {
    const int lanes_log2 = a.shape.d > 64 ? 5 : a.shape.d > 32 ? 4 : 3;
    const int total = a.shape.hq + (a.v ? 2 : 1) * a.shape.hk;
    // few tokens: the heads of a token are shared among blocks, one round of a block's warps each
    const int round = kRopeWarps * (32 >> lanes_log2);
    const int share = a.m < 2 * device_sm_count() ? round : total;
    const dim3 grid((unsigned)a.m, (unsigned)((total + share - 1) / share));
    qk_norm_rope_kernel<In, Out><<<grid, kRopeThreads, 0, st>>>(a, lanes_log2, share);
    return cudaGetLastError();
}

template <typename In> cudaError_t launch_in(const RopeArgs &a, qmm_float out_type, cudaStream_t st) {
    return out_type == QMM_F16 ? launch_typed<In, __half>(a, st) : launch_typed<In, __nv_bfloat16>(a, st);
}

}  // namespace

cudaError_t launch_qk_norm_rope(const RopeArgs &a, qmm_float in_type, qmm_float out_type, cudaStream_t st) {
    if (in_type == QMM_F32) return launch_in<float>(a, out_type, st);
    return in_type == QMM_F16 ? launch_in<__half>(a, out_type, st) : launch_in<__nv_bfloat16>(a, out_type, st);
}

}  // namespace qmm
