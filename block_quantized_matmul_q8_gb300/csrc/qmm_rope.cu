// qmm_rope.cu -- RMS norm of query and key heads, rotation by position and rounding to 16
// bits, one pass over the qkv product:
//   n = x * w / sqrt(mean(x^2) + eps),  (a, b) -> (a cos - b sin, b cos + a sin).
//
// Bound by HBM: each element is read once and written once.  One block takes one token (or a
// share of its heads when there are few tokens); its first threads compute the token's
// rotary/2 angles once for all heads while the first heads are being loaded.  A lane holds eight
// elements of a head, four of them the partners of the other four, so that a pair turns inside a
// lane and a head's sum of squares is a reduction over at most 16 lanes (with four elements a lane
// and the partner a shuffle away the arithmetic took longer than the traffic: 90 against 62 us for
// 8192 tokens of 40 + 8 + 8 fp32 heads of 128, 5.6 TB/s).  16-bit heads of 64 stay below that, 4.1 TB/s
// (4100 tokens of 96 heads, 24.8 us in a graph and 27.3 in a row of calls): half the bytes for the same
// instructions, and at 20 warps an SM the loads' latency shows.
#include <cuda_runtime.h>

#include <algorithm>

#include "qmm_attn.h"
#include "qmm_internal.h"
#include "qmm_rope.cuh"

namespace qmm {

namespace {

constexpr int kRopeThreads = 128;
constexpr int kRopeWarps = kRopeThreads / 32;

template <typename In, typename Out, bool kInterleaved>
__global__ void __launch_bounds__(kRopeThreads) qk_norm_rope_kernel(const RopeArgs a, int lanes_log2, int share) {
    __shared__ float2 cs[kMaxHeadDim / 2];
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int64_t t = blockIdx.x;
    const int d = a.shape.d, hq = a.shape.hq, hk = a.shape.hk, r = a.rotary;
    const int lanes = 1 << lanes_log2;                // lanes of one head
    const int sub = lane >> lanes_log2, c = lane & (lanes - 1);
    const int per_warp = 32 >> lanes_log2;            // heads of one warp at a time
    const int total = hq + (a.v ? 2 : 1) * hk;
    const int h_begin = blockIdx.y * share, h_end = min(total, h_begin + share);
    const bool live = 8 * c < d, turned = 8 * c < r;
    // this lane's elements e0..e0+3 and e1..e1+3: pairs across them, or within each when interleaved
    const int e0 = turned && !kInterleaved ? 4 * c : 8 * c, e1 = turned && !kInterleaved ? r / 2 + 4 * c : 8 * c + 4;

    auto load = [&](int h, float4 &x, float4 &y) {
        x = y = make_float4(0.f, 0.f, 0.f, 0.f);
        if (!live || h >= h_end) return;
        const In *p = h < hq        ? static_cast<const In *>(a.q) + t * a.sq.t + h * a.sq.h
                      : h < hq + hk ? static_cast<const In *>(a.k) + t * a.sk.t + (h - hq) * a.sk.h
                                    : static_cast<const In *>(a.v) + t * a.sv.t + (h - hq - hk) * a.sv.h;
        load8<kInterleaved>(p, e0, e1, x, y);
    };
    int h = h_begin + warp * per_warp + sub;
    const int step = kRopeWarps * per_warp;
    float4 x, y;
    load(h, x, y);
    if (tid < r / 2) cs[tid] = cos_sin(a.positions[t], a.inv_freq[tid]);
    __syncthreads();
    float2 turn[4];  // of the lane's four pairs
#pragma unroll
    for (int j = 0; j < 4; ++j) turn[j] = turned ? cs[4 * c + j] : make_float2(1.f, 0.f);
    const float inv_d = 1.0f / float(d);

    for (; h - sub < h_end; h += step) {
        float4 A = x, B = y;
        load(h + step, x, y);
        const bool is_q = h < hq, is_v = h >= hq + hk;
        const float *w = is_v ? nullptr : is_q ? a.wq : a.wk;
        float ss = A.x * A.x + A.y * A.y + A.z * A.z + A.w * A.w + B.x * B.x + B.y * B.y + B.z * B.z + B.w * B.w;
        for (int o = lanes >> 1; o > 0; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
        if (!live || h >= h_end) continue;
        if (w) {  // read again for every head: from the L1 cache, where registers would cost occupancy
            const float inv = rsqrtf(ss * inv_d + a.eps);
            A = make_float4(A.x * inv * w[e0], A.y * inv * w[e0 + 1], A.z * inv * w[e0 + 2], A.w * inv * w[e0 + 3]);
            B = make_float4(B.x * inv * w[e1], B.y * inv * w[e1 + 1], B.z * inv * w[e1 + 2], B.w * inv * w[e1 + 3]);
        }
        if (!is_v && turned) {
            auto rotate = [](float &p, float &q, float2 cs) {
                const float n = p * cs.x - q * cs.y;
                q = q * cs.x + p * cs.y;
                p = n;
            };
            if (kInterleaved) {
                rotate(A.x, A.y, turn[0]);
                rotate(A.z, A.w, turn[1]);
                rotate(B.x, B.y, turn[2]);
                rotate(B.z, B.w, turn[3]);
            } else {
                rotate(A.x, B.x, turn[0]);
                rotate(A.y, B.y, turn[1]);
                rotate(A.z, B.z, turn[2]);
                rotate(A.w, B.w, turn[3]);
            }
        }
        Out *out = is_q    ? static_cast<Out *>(a.qo) + t * a.sqo.t + h * a.sqo.h
                   : !is_v ? static_cast<Out *>(a.ko) + t * a.sko.t + (h - hq) * a.sko.h
                           : static_cast<Out *>(a.vo) + t * a.svo.t + (h - hq - hk) * a.svo.h;
        store8<kInterleaved>(out, e0, e1, A, B);
    }
}

template <typename In, typename Out> cudaError_t launch_typed(const RopeArgs &a, cudaStream_t st) {
    int lanes_log2 = 0;
    while ((8 << lanes_log2) < a.shape.d) ++lanes_log2;
    const int total = a.shape.hq + (a.v ? 2 : 1) * a.shape.hk;
    // few tokens: the heads of a token are shared among blocks, one round of a block's warps each
    // (48 fp32 heads of 128, shared and whole: 1 token 2.3 and 5.0 us, 152 tokens 3.2 and 5.6, 300 5.0 and
    // 6.0, 600 6.5 and 6.4, 1200 12.0 and 9.4, where each block turns its token's angles again)
    const int round = kRopeWarps * (32 >> lanes_log2);
    const int share = a.m < 4 * device_sm_count() ? round : (total + round - 1) / round * round;
    const dim3 grid((unsigned)a.m, (unsigned)((total + share - 1) / share));
    auto kern = a.interleaved ? qk_norm_rope_kernel<In, Out, true> : qk_norm_rope_kernel<In, Out, false>;
    kern<<<grid, kRopeThreads, 0, st>>>(a, lanes_log2, share);
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
