// qmm_rope.cuh -- pieces shared by the kernels that norm and turn heads: loads and stores of four
// and eight elements, and the sine and cosine of a position's angle.
#pragma once
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <stdint.h>

namespace qmm {

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

// Eight elements: x at p + e0 and y at p + e1, one access when they are neighbours and 16 bits wide.
template <bool kNext, typename In> __device__ __forceinline__ void load8(const In *p, int e0, int e1, float4 &x, float4 &y) {
    if constexpr (kNext && sizeof(In) == 2) {
        const uint4 u = *reinterpret_cast<const uint4 *>(p + e0);
        const uint2 h[2] = {make_uint2(u.x, u.y), make_uint2(u.z, u.w)};
        x = load4(reinterpret_cast<const In *>(&h[0]));
        y = load4(reinterpret_cast<const In *>(&h[1]));
    } else {
        x = load4(p + e0);
        y = load4(p + e1);
    }
}
template <bool kNext, typename Out> __device__ __forceinline__ void store8(Out *p, int e0, int e1, float4 x, float4 y) {
    if constexpr (kNext) {
        uint2 h[2];
        store4(reinterpret_cast<Out *>(&h[0]), x);
        store4(reinterpret_cast<Out *>(&h[1]), y);
        *reinterpret_cast<uint4 *>(p + e0) = make_uint4(h[0].x, h[0].y, h[1].x, h[1].y);
    } else {
        store4(p + e0, x);
        store4(p + e1, y);
    }
}

// Sine and cosine of pos * freq.  The angle is taken in turns as a 64-bit fraction, whose whole
// turns fall off by themselves: freq / (2 pi) = m 2^q / (2 pi) for freq's mantissa m, with 1 / (2 pi)
// as a 64-bit integer over 2^66, times pos modulo 2^64.  Exact to 2^-32 of a turn at every int32 position.
__device__ __forceinline__ float2 cos_sin(int pos, float freq) {
    const uint32_t bits = __float_as_uint(freq), expo = (bits >> 23) & 255u;
    const uint64_t m = (bits & 0x7fffffu) | (expo ? 0x800000u : 0u);
    const int q = int(expo ? expo : 1u) - 150;
    constexpr uint64_t kInv2Pi = 0xA2F9836E4E44152Aull;  // round(2^66 / (2 pi))
    const uint64_t lo = m * kInv2Pi, hi = __umul64hi(m, kInv2Pi);
    const int right = 2 - q;  // turns per position in units of 2^-64: (hi:lo) 2^-right
    uint64_t f;
    if (right <= 0) f = right > -64 ? lo << -right : 0;
    else if (right < 64) f = (hi << (64 - right)) | (lo >> right);
    else f = right < 128 ? hi >> (right - 64) : 0;
    uint64_t turns = f * uint64_t(int64_t(pos));
    if (bits >> 31) turns = 0 - turns;
    float s, c;
    sincospif(float(int32_t(turns >> 32)) * 4.6566128730773926e-10f, &s, &c);  // 2^-31: half turns
    if (expo == 255u) s = c = __int_as_float(0x7fffffff);
    return make_float2(c, s);
}

}  // namespace qmm
