// qmm_kv.cu -- writing and reading the paged key/value cache in 4 or 8 bits.
//
// Appending: what qmm_qk_norm_rope computes (n = x w / sqrt(mean(x^2) + eps), (a, b) -> (a cos - b sin,
// b cos + a sin)), with keys and values quantized on the way, in blocks of 32 of a head:
//   Q4_0: d = fp16(e / -8), e the element of largest magnitude (the positive one of two), code = rint(x / d) in -8..7
//   Q8_0: d = fp16(max |x| / 127), code = rint(x / d) in -127..127
// Codes are the nearest ones for the scale as it is stored (an IEEE division, so that a value half way
// between two codes is seen as such), and a scale that rounds to zero gives zeros.
//
// Reading: value = d * code, exact in fp32, rounded once to 16 bits.
//
// Both move each byte once.  8192 tokens of 32 + 8 + 8 fp32 heads of 128, with the values: 62.3 us, 5.0 TB/s (74% of the
// measured copy rate; issue slots 70% busy: a third of the heads are quantized); 2048 tokens 19.7 us, 6 of them start
// and end; one token 4.3.  131072 tokens of 8 heads of 128 read back: 110.8 us, 6.2 TB/s (92%); 32768 31.9 us.
#include <cuda_runtime.h>

#include <algorithm>
#include <atomic>

#include "qmm_attn.cuh"
#include "qmm_internal.h"
#include "qmm_kv.h"
#include "qmm_rope.cuh"

namespace qmm {

namespace {

constexpr int kThreads = 128;
constexpr int kWarps = kThreads / 32;

template <typename T> __device__ __forceinline__ uint4 round8(const float (&v)[8]) {
    return make_uint4(pack2<T>(v[0], v[1]), pack2<T>(v[2], v[3]), pack2<T>(v[4], v[5]), pack2<T>(v[6], v[7]));
}

// One block a token, or a share of its heads where tokens are few (as in qmm_rope.cu, whose lanes these
// are: eight elements of a head each, four of them the partners of the other four).  Four lanes with
// eight neighbours each hold a block of 32: value heads are loaded so, key heads whose partners are half a rotation apart
// go through shared memory after the turn.
template <typename In, typename Out, bool kInterleaved, bool kQ8>
__global__ void __launch_bounds__(kThreads) kv_append_kernel(const KvAppendArgs a, int lanes_log2, int share) {
    __shared__ float2 cs[kMaxHeadDim / 2];
    __shared__ __align__(16) float rows[kWarps][256];
    ptx::grid_dependency_wait();
    ptx::grid_launch_dependents();  // the attention that reads these pages may start, and waits
    const RopeArgs &p = a.rope;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int64_t t = blockIdx.x;
    const int d = p.shape.d, hq = p.shape.hq, hk = p.shape.hk, r = p.rotary;
    const int lanes = 1 << lanes_log2;                // lanes of one head
    const int sub = lane >> lanes_log2, c = lane & (lanes - 1);
    const int per_warp = 32 >> lanes_log2;            // heads of one warp at a time
    const int total = hq + 2 * hk;
    const int h_begin = blockIdx.y * share, h_end = min(total, h_begin + share);
    const bool live = 8 * c < d, turned = 8 * c < r;
    const int e0 = turned && !kInterleaved ? 4 * c : 8 * c, e1 = turned && !kInterleaved ? r / 2 + 4 * c : 8 * c + 4;

    auto load = [&](int h, float4 &x, float4 &y) {
        x = y = make_float4(0.f, 0.f, 0.f, 0.f);
        if (!live || h >= h_end) return;
        if (h >= hq + hk) {
            load8<true>(static_cast<const In *>(p.v) + t * p.sv.t + (h - hq - hk) * p.sv.h, 8 * c, 8 * c + 4, x, y);
            return;
        }
        const In *s = h < hq ? static_cast<const In *>(p.q) + t * p.sq.t + h * p.sq.h
                             : static_cast<const In *>(p.k) + t * p.sk.t + (h - hq) * p.sk.h;
        load8<kInterleaved>(s, e0, e1, x, y);
    };
    int h = h_begin + warp * per_warp + sub;
    const int step = kWarps * per_warp;
    float4 x, y;
    load(h, x, y);
    const int slot = a.slots[t];
    if (tid < r / 2) cs[tid] = cos_sin(p.positions[t], p.inv_freq[tid]);
    __syncthreads();
    float2 turn[4];  // of the lane's four pairs
#pragma unroll
    for (int j = 0; j < 4; ++j) turn[j] = turned ? cs[4 * c + j] : make_float2(1.f, 0.f);
    const float inv_d = 1.0f / float(d);
    const int page = slot >> a.cache.page_log2, in_page = slot & ((1 << a.cache.page_log2) - 1);
    const bool held = slot >= 0 && page < a.cache.n_pages;  // else the token goes into no page
    const int groups_log2 = a.cache.page_log2 - 4, token = in_page & 15;
    uint8_t *const group = a.cache.pages + (held ? page * a.cache.page_stride : 0) + (in_page >> 4) * kv_record_bytes(kQ8, d);

    for (; h - sub < h_end; h += step) {
        float4 A = x, B = y;
        load(h + step, x, y);
        const bool is_q = h < hq, is_v = h >= hq + hk;
        const float *w = is_v ? nullptr : is_q ? p.wq : p.wk;
        float ss = A.x * A.x + A.y * A.y + A.z * A.z + A.w * A.w + B.x * B.x + B.y * B.y + B.z * B.z + B.w * B.w;
        for (int o = lanes >> 1; o > 0; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
        const bool mine = live && h < h_end;
        if (w && mine) {
            const float inv = rsqrtf(ss * inv_d + p.eps);
            A = make_float4(A.x * inv * w[e0], A.y * inv * w[e0 + 1], A.z * inv * w[e0 + 2], A.w * inv * w[e0 + 3]);
            B = make_float4(B.x * inv * w[e1], B.y * inv * w[e1 + 1], B.z * inv * w[e1 + 2], B.w * inv * w[e1 + 3]);
        }
        if (!is_v && turned) {
            auto rotate = [](float &u, float &v, float2 cs) {
                const float n = u * cs.x - v * cs.y;
                v = v * cs.x + u * cs.y;
                u = n;
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
        if (is_q && mine) store8<kInterleaved>(static_cast<Out *>(p.qo) + t * p.sqo.t + h * p.sqo.h, e0, e1, A, B);
        if (__all_sync(0xffffffffu, is_q)) continue;

        // ---- keys and values: eight neighbours a lane
        if (!kInterleaved && __any_sync(0xffffffffu, !is_q && !is_v)) {
            float *row = &rows[warp][sub * 8 * lanes];
            __syncwarp();
            if (live && !is_v) {
                *reinterpret_cast<float4 *>(row + e0) = A;
                *reinterpret_cast<float4 *>(row + e1) = B;
            }
            __syncwarp();
            if (live && !is_v) {
                A = *reinterpret_cast<const float4 *>(row + 8 * c);
                B = *reinterpret_cast<const float4 *>(row + 8 * c + 4);
            }
        }
        float v[8] = {A.x, A.y, A.z, A.w, B.x, B.y, B.z, B.w}, top = -INFINITY, low = INFINITY;
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            v[j] = live && v[j] == v[j] ? v[j] : 0.f;  // NaN is held as zero, an infinity as the largest value
            top = fmaxf(top, v[j]);
            low = fminf(low, v[j]);
        }
#pragma unroll
        for (int o = 1; o < 4; o <<= 1) {
            top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
            low = fminf(low, __shfl_xor_sync(0xffffffffu, low, o));
        }
        if (!mine || is_q) continue;
        float scale = kQ8 ? fmaxf(top, -low) / 127.f : (top >= -low ? top : low) * -0.125f;
        const __half hs = __float2half_rn(fminf(fmaxf(scale, -65504.f), 65504.f));
        scale = __half2float(hs);
        // codes as floats, and side by side as words: adding 1.5 2^23 leaves an integer in the low bits
        uint32_t word[2] = {0, 0};
        constexpr int kShift = kQ8 ? 8 : 4, kPer = 32 / kShift;
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const float q = scale == 0.f ? 0.f : rintf(__fdiv_rn(v[j], scale));
            v[j] = kQ8 ? fminf(fmaxf(q, -127.f), 127.f) : fminf(fmaxf(q, -8.f), 7.f);
            const uint32_t bits = __float_as_uint(v[j] + (12582912.f + (kQ8 ? 128.f : 8.f))) - 0x4B400000u;
            word[j / kPer] += bits << (kShift * (j % kPer));
        }
        const int kv = h - hq - (is_v ? hk : 0);
        if (held) {
            uint8_t *side = group + (int64_t(kv) << groups_log2) * kv_record_bytes(kQ8, d) + (is_v ? kv_side_bytes(kQ8, d) : 0);
            if (kQ8) *reinterpret_cast<uint2 *>(side + (c >> 1) * 256 + token * 16 + (c & 1) * 8) = make_uint2(word[0], word[1]);
            else *reinterpret_cast<uint32_t *>(side + (c >> 2) * 256 + token * 16 + (c & 3) * 4) = word[0];
            if ((c & 3) == 0)
                reinterpret_cast<__half *>(side + kv_scales_at(kQ8, d) + (c >> 2) * 32)[kv_scale_place(token)] = hs;
        }
        Out *out = is_v ? static_cast<Out *>(p.vo) : static_cast<Out *>(p.ko);
        if (out) {
            out += is_v ? t * p.svo.t + kv * p.svo.h : t * p.sko.t + kv * p.sko.h;
            float f[8];
#pragma unroll
            for (int j = 0; j < 8; ++j) f[j] = scale * v[j];
            *reinterpret_cast<uint4 *>(out + 8 * c) = round8<Out>(f);
        }
    }
}

template <typename In, typename Out> cudaError_t launch_append(const KvAppendArgs &a, cudaStream_t st) {
    int lanes_log2 = 0;
    while ((8 << lanes_log2) < a.rope.shape.d) ++lanes_log2;
    const int total = a.rope.shape.hq + 2 * a.rope.shape.hk;
    // few tokens: the heads of a token are shared among blocks, one round of a block's warps each
    const int round = kWarps * (32 >> lanes_log2);
    const int share = a.rope.m < 4 * device_sm_count() ? round : (total + round - 1) / round * round;
    const dim3 grid((unsigned)a.rope.m, (unsigned)((total + share - 1) / share));
    auto kern = a.cache.q8 ? (a.rope.interleaved ? kv_append_kernel<In, Out, true, true> : kv_append_kernel<In, Out, false, true>)
                           : (a.rope.interleaved ? kv_append_kernel<In, Out, true, false> : kv_append_kernel<In, Out, false, false>);
    return launch_pdl(kern, grid, dim3(kThreads), 0, st, a, lanes_log2, share);
}
template <typename In> cudaError_t launch_append_in(const KvAppendArgs &a, qmm_float out_type, cudaStream_t st) {
    return out_type == QMM_F16 ? launch_append<In, __half>(a, st) : launch_append<In, __nv_bfloat16>(a, st);
}

// Eight values in 16 bits, scale (fp16 bits) times code, from codes that become fp16 integers two at a time: 1024 + n
// less 1032, (1024 + 16 n) / 16 less 72, 1024 + u less 1152, all exact.  The product is exact in fp32, and fp16's own
// multiplication rounds it once.
__device__ __forceinline__ __half2 as_h2(uint32_t x) { return *reinterpret_cast<const __half2 *>(&x); }
template <typename Out> __device__ __forceinline__ uint32_t times(float scale, float x, float y) { return pack2<Out>(scale * x, scale * y); }
template <typename Out> __device__ __forceinline__ uint4 values_q4(uint32_t x, uint16_t scale) {
    const uint32_t y = x >> 8;
    const __half2 less = __half2half2(__ushort_as_half(0xE408)), part = __half2half2(__ushort_as_half(0x2C00)),
                  rest = __half2half2(__ushort_as_half(0xD480));
    const __half2 n04 = __hadd2(as_h2((x & 0x000f000fu) | 0x64006400u), less), n15 = __hfma2(as_h2((x & 0x00f000f0u) | 0x64006400u), part, rest);
    const __half2 n26 = __hadd2(as_h2((y & 0x000f000fu) | 0x64006400u), less), n37 = __hfma2(as_h2((y & 0x00f000f0u) | 0x64006400u), part, rest);
    if constexpr (std::is_same<Out, __half>::value) {
        const __half2 d = __half2half2(__ushort_as_half(scale));
        const uint32_t a = h2bits(__hmul2(n04, d)), b = h2bits(__hmul2(n15, d)), e = h2bits(__hmul2(n26, d)), f = h2bits(__hmul2(n37, d));
        return make_uint4(__byte_perm(a, b, 0x5410), __byte_perm(e, f, 0x5410), __byte_perm(a, b, 0x7632), __byte_perm(e, f, 0x7632));
    } else {
        const float d = __half2float(__ushort_as_half(scale));
        const float2 a = __half22float2(n04), b = __half22float2(n15), e = __half22float2(n26), f = __half22float2(n37);
        return make_uint4(times<Out>(d, a.x, b.x), times<Out>(d, e.x, f.x), times<Out>(d, a.y, b.y), times<Out>(d, e.y, f.y));
    }
}
template <typename Out> __device__ __forceinline__ uint4 values_q8(uint32_t x, uint32_t y, uint16_t scale) {
    const __half2 less = __half2half2(__ushort_as_half(0xE480));
    const uint32_t w[2] = {x, y};
    uint32_t out[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const __half2 n = __hadd2(as_h2(__byte_perm(w[i >> 1], 0x64646464u, i & 1 ? 0x4342 : 0x4140)), less);
        if constexpr (std::is_same<Out, __half>::value) {
            out[i] = h2bits(__hmul2(n, __half2half2(__ushort_as_half(scale))));
        } else {
            const float2 v = __half22float2(n);
            out[i] = times<Out>(__half2float(__ushort_as_half(scale)), v.x, v.y);
        }
    }
    return make_uint4(out[0], out[1], out[2], out[3]);
}

// Reading: a block takes kReadTokens rows of the packed output and a share of the heads.  Its first threads find
// each row's sequence, page and record once for all heads; a lane then writes eight elements (16 bytes),
// neighbouring lanes a whole row, and two neighbouring tokens fill the 32-byte sectors of the codes.
constexpr int kReadTokens = 32;

template <typename Out, bool kQ8, int D> __global__ void __launch_bounds__(kThreads) kv_read_kernel(const KvReadArgs a, int share) {
    constexpr int kRec = kv_record_bytes(kQ8, D), kSide = kv_side_bytes(kQ8, D), kLanes = D / 8;
    constexpr int kItems = kReadTokens * kLanes / kThreads;  // of a thread, a head and a side
    __shared__ const uint8_t *record_s[kReadTokens];         // of the first head
    __shared__ int token_s[kReadTokens];                     // 0..15; -1: the page does not exist, the row is zero; -2: it is not written
    ptx::grid_dependency_wait();
    ptx::grid_launch_dependents();
    const int tid = threadIdx.x, log2p = a.cache.page_log2;
    const int64_t t0 = int64_t(blockIdx.x) * kReadTokens;
    if (tid < kReadTokens) {
        const int64_t t = t0 + tid;
        const uint8_t *record = nullptr;
        int token = -2;
        if (t < a.tokens) {
            int64_t lo = 0, hi = a.n_seqs;  // the last sequence that starts at or before t
            while (hi - lo > 1) {
                const int64_t mid = (lo + hi) / 2;
                if (a.cu[mid] <= t) lo = mid;
                else hi = mid;
            }
            const int64_t pos = t - a.cu[lo];
            if (pos >= 0 && t < a.cu[lo + 1]) {
                const int64_t idx = pos >> log2p;
                const int page = idx < a.table_width ? a.table[lo * a.table_stride + idx] : -1;
                const int in_page = int(pos & ((1 << log2p) - 1));
                const bool there = page >= 0 && page < a.cache.n_pages;
                record = a.cache.pages + (there ? page * a.cache.page_stride : 0) + (in_page >> 4) * kRec;
                token = there ? in_page & 15 : -1;
                if (!there) reported = QMM_ERR_IDS;
            }
        }
        record_s[tid] = record;
        token_s[tid] = token;
    }
    __syncthreads();
    const int64_t head_step = int64_t(1 << (log2p - 4)) * kRec;
    const int h0 = blockIdx.y * share, h1 = min(h0 + share, a.hk);
    // each item's codes and scale, and its places in the output
    const uint8_t *codes[kItems], *scales[kItems];
    Out *ko[kItems], *vo[kItems];
    bool there[kItems];
#pragma unroll
    for (int i = 0; i < kItems; ++i) {
        const int row = (tid + i * kThreads) / kLanes, c = (tid + i * kThreads) % kLanes, token = max(token_s[row], 0);
        const uint8_t *p = record_s[row];
        there[i] = token_s[row] >= 0;
        codes[i] = p + h0 * head_step + (kQ8 ? (c >> 1) * 256 + (c & 1) * 8 : (c >> 2) * 256 + (c & 3) * 4) + token * 16;
        scales[i] = p + h0 * head_step + kv_scales_at(kQ8, D) + (c >> 2) * 32 + 2 * kv_scale_place(token);
        ko[i] = token_s[row] > -2 ? static_cast<Out *>(a.ko) + (t0 + row) * a.sko.t + h0 * a.sko.h + 8 * c : nullptr;
        vo[i] = static_cast<Out *>(a.vo) + (t0 + row) * a.svo.t + h0 * a.svo.h + 8 * c;
    }
    for (int h = h0; h < h1; ++h) {
        uint32_t u[2][kItems][kQ8 ? 2 : 1];
        uint16_t s[2][kItems];
#pragma unroll
        for (int is_v = 0; is_v < 2; ++is_v)
#pragma unroll
            for (int i = 0; i < kItems; ++i) {
                u[is_v][i][0] = u[is_v][i][kQ8 ? 1 : 0] = kQ8 ? 0x80808080u : 0x88888888u;  // code 0: a row of no page is +0
                s[is_v][i] = 0;
                if (!there[i]) continue;
                if constexpr (kQ8) {
                    const uint2 w = *reinterpret_cast<const uint2 *>(codes[i] + is_v * kSide);
                    u[is_v][i][0] = w.x;
                    u[is_v][i][1] = w.y;
                } else {
                    u[is_v][i][0] = *reinterpret_cast<const uint32_t *>(codes[i] + is_v * kSide);
                }
                s[is_v][i] = *reinterpret_cast<const uint16_t *>(scales[i] + is_v * kSide);
            }
#pragma unroll
        for (int is_v = 0; is_v < 2; ++is_v)
#pragma unroll
            for (int i = 0; i < kItems; ++i) {
                if (!ko[i]) continue;
                const uint4 out = kQ8 ? values_q8<Out>(u[is_v][i][0], u[is_v][i][kQ8 ? 1 : 0], s[is_v][i])
                                      : values_q4<Out>(u[is_v][i][0], s[is_v][i]);
                *reinterpret_cast<uint4 *>(is_v ? vo[i] : ko[i]) = out;
            }
#pragma unroll
        for (int i = 0; i < kItems; ++i) {
            codes[i] += head_step;
            scales[i] += head_step;
            if (ko[i]) ko[i] += a.sko.h;
            vo[i] += a.svo.h;
        }
    }
}

template <typename Out, bool kQ8> cudaError_t launch_read(const KvReadArgs &a, cudaStream_t st) {
    const int64_t blocks = (a.tokens + kReadTokens - 1) / kReadTokens;
    // few rows: the heads are shared among blocks
    int share = a.hk;
    while (share > 1 && blocks * ((a.hk + share - 1) / share) < 8 * device_sm_count()) share = (share + 1) / 2;
    const dim3 grid((unsigned)blocks, (unsigned)((a.hk + share - 1) / share));
    switch (a.d) {
        case 32: return launch_pdl(kv_read_kernel<Out, kQ8, 32>, grid, dim3(kThreads), 0, st, a, share);
        case 64: return launch_pdl(kv_read_kernel<Out, kQ8, 64>, grid, dim3(kThreads), 0, st, a, share);
        case 96: return launch_pdl(kv_read_kernel<Out, kQ8, 96>, grid, dim3(kThreads), 0, st, a, share);
        default: return launch_pdl(kv_read_kernel<Out, kQ8, 128>, grid, dim3(kThreads), 0, st, a, share);
    }
}

}  // namespace

cudaError_t launch_kv_append(const KvAppendArgs &a, qmm_float in_type, qmm_float out_type, cudaStream_t st) {
    if (in_type == QMM_F32) return launch_append_in<float>(a, out_type, st);
    return in_type == QMM_F16 ? launch_append_in<__half>(a, out_type, st) : launch_append_in<__nv_bfloat16>(a, out_type, st);
}

namespace {
std::atomic<bool> launched{false};  // a kernel that may report has been launched (or captured) by this process
}

cudaError_t launch_kv_read(const KvReadArgs &a, qmm_float out_type, cudaStream_t st) {
    launched = true;
    if (a.cache.q8) return out_type == QMM_F16 ? launch_read<__half, true>(a, st) : launch_read<__nv_bfloat16, true>(a, st);
    return out_type == QMM_F16 ? launch_read<__half, false>(a, st) : launch_read<__nv_bfloat16, false>(a, st);
}

cudaError_t kv_take_error(int *code, cudaStream_t st) {
    *code = QMM_OK;
    return launched ? take_error(code, st) : cudaSuccess;
}

}  // namespace qmm
