// qmm_attn.cuh -- pieces shared by the attention kernels.
#pragma once
#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <type_traits>

#include "qmm_attn.h"
#include "qmm_tc_common.cuh"
#include "qmm_tc_ptx.cuh"

namespace qmm {

constexpr float kLog2e = 1.4426950408889634f, kLn2 = 0.6931471805599453f;

__device__ __forceinline__ float ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
// Two values rounded to T, lo in the low half.
template <typename T> __device__ __forceinline__ uint32_t pack2(float lo, float hi) {
    uint32_t r;
    if (std::is_same<T, __half>::value) asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    else asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
}
// Set by a kernel of this file that gave up a wait, and only taken back by take_gave_up.
static __device__ int gave_up;

// Whether the flag was set on the current device; clears it.  Synchronises the stream.
static inline cudaError_t take_gave_up(bool *yes, cudaStream_t st) {
    int v = 0;
    cudaError_t e = cudaMemcpyFromSymbolAsync(&v, gave_up, sizeof(v), 0, cudaMemcpyDeviceToHost, st);
    if (e == cudaSuccess) e = cudaStreamSynchronize(st);
    *yes = v != 0;
    if (e != cudaSuccess || !v) return e;
    v = 0;
    e = cudaMemcpyToSymbolAsync(gave_up, &v, sizeof(v), 0, cudaMemcpyHostToDevice, st);
    return e == cudaSuccess ? cudaStreamSynchronize(st) : e;
}

// mbar_wait by a whole warp: all lanes go on, or all give up.
__device__ __forceinline__ bool warp_wait(uint32_t bar, uint32_t parity, volatile int *abort,
                                          long long limit = ptx::kWaitCycles) {
    return __all_sync(0xffffffffu, ptx::mbar_wait(bar, parity, abort, limit));
}

// A [tokens][heads][d] view (batch of them: batch_stride elements apart) as a tensor map with
// boxes of 64 elements x box_heads x box_tokens, 128-byte swizzled.  A stride that is never
// taken is given as one that the encoder accepts.
inline bool attn_make_map(CUtensorMap *map, qmm_float t, const void *data, int d, int64_t heads, int64_t tokens,
                          HeadStrides s, int box_heads, int box_tokens, int64_t batch = 0, int64_t batch_stride = 0) {
    const uint64_t dims[4] = {uint64_t(d), uint64_t(heads), uint64_t(tokens), uint64_t(batch)};
    const uint64_t strides[3] = {uint64_t(heads > 1 ? s.h : d) * 2, uint64_t(tokens > 1 ? s.t : d) * 2,
                                 uint64_t(batch > 1 ? batch_stride : d) * 2};
    const uint32_t box[4] = {64, uint32_t(box_heads), uint32_t(box_tokens), 1};
    return tc_make_map(map, t == QMM_F16 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT16 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16,
                       batch > 0 ? 4 : 3, data, dims, strides, box, CU_TENSOR_MAP_SWIZZLE_128B);
}

}  // namespace qmm
