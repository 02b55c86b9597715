// qmm_kv_attn.cu -- attention of a decoding batch over a paged cache in 4 or 8 bits.
//
//   out = sum_j p_j v_j,  p = softmax_j(scale q.k_j),  k_j = d_jb (code - bias) in block b of 32 elements
//
// Bound by reading the codes and scales once: 0.5625 bytes an element in 4 bits, so that at the copy rate
// an SM gets 42 elements a cycle and has about 3 lane operations for each.  What the kernel does for that:
//   - scores: the codes enter the MMA as fp16 subnormals (a nibble masked in place is code 2^-24, or 16 code
//     2^-24 with the query's elements divided by 16): one operation for two codes.  The bias is the accumulator's first
//     value, -bias sum q of the block, and the block's scale multiplies the fp32 accumulator.  Queries
//     are scaled by a power of two to fp16's upper range, where 16-bit inputs are exact down to 2^-14 of a head's largest.
//   - values: the block's scale multiplies the weights, p d_jb rounded to fp16 (fp16's 11 bits; below
//     2^-14 an absolute 2^-25), codes become exact fp16 integers, and the sums are fp32.
//   - the fragments come from shared memory by ldmatrix with neighbouring codes in one 16-bit unit, transposed for V,
//     so that a nibble's mask gives the pairs of keys or elements that the MMA wants.
// A warp takes tiles of 32 keys on its own: a private ring of bulk copies (a record of 16 tokens is
// contiguous), its running softmax, no barrier with other warps until the join.  A cluster of up to 16 CTAs
// takes one request and kv head and joins through distributed shared memory; where that leaves SMs idle, several
// clusters do, joined by a second launch.  mma.sync: 8 query heads would leave tcgen05's 128 rows empty.
#include <cuda.h>
#include <cuda_runtime.h>

#include <algorithm>

#include "qmm_attn.cuh"
#include "qmm_internal.h"
#include "qmm_kv.h"
#include "qmm_mma.cuh"
#include "qmm_tc_ptx.cuh"

namespace qmm {

namespace {

using namespace ptx;

constexpr int kTileKeys = 32;
constexpr int kWarps = 4;
constexpr int kThreads = kWarps * 32;
constexpr int kRows = 8;         // query heads of one CTA: the MMA's N side
constexpr int kMaxCluster = 16;
constexpr int kMaxParts = 64;    // clusters of one request and kv head

template <bool kQ8, int D> struct Tile {
    static constexpr int kSide = kv_side_bytes(kQ8, D), kScales = kv_scales_at(kQ8, D);
    static constexpr int kRec = kv_record_bytes(kQ8, D), kBytes = 2 * kRec;
    static constexpr int kStages = std::max(2, std::min(6, 56 * 1024 / (kWarps * kBytes)));
    static constexpr int kStride = D + 4;  // floats between partial rows
    static constexpr int kRing = kWarps * kStages * kBytes;
    static constexpr int kParts = kWarps * kRows * kStride * 4;  // partial rows, in place of the ring
    static constexpr int kSmem = (std::max(kRing, kParts) + 127) / 128 * 128;
};

struct Args {
    KvDecodeArgs d;
    int group, row_blocks;  // query heads of a kv head, blocks of 8 of them
    int splits;             // clusters of a request and kv head
    float scale_log2;
    float *part, *part_lse; // [splits][batch * hq][d] normalised, their log2 denominators
    int fault;              // as in qmm_attn.cu
};

__device__ __forceinline__ void ldsm2(uint32_t (&r)[4], uint32_t addr) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x2.shared.b16 {%0,%1}, [%2];" : "=r"(r[0]), "=r"(r[1]) : "r"(addr) : "memory");
}
__device__ __forceinline__ void ldsm2_t(uint32_t (&r)[4], uint32_t addr) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x2.trans.shared.b16 {%0,%1}, [%2];" : "=r"(r[0]), "=r"(r[1]) : "r"(addr) : "memory");
}
__device__ __forceinline__ uint2 lds64(uint32_t addr) {
    uint2 v;
    asm volatile("ld.shared.v2.u32 {%0,%1}, [%2];" : "=r"(v.x), "=r"(v.y) : "r"(addr) : "memory");
    return v;
}
__device__ __forceinline__ float2 halves(uint32_t x) { return __half22float2(*reinterpret_cast<const __half2 *>(&x)); }
__device__ __forceinline__ uint32_t mul2(uint32_t x, uint32_t y) {
    return h2bits(__hmul2(*reinterpret_cast<const __half2 *>(&x), *reinterpret_cast<const __half2 *>(&y)));
}
// fp16 (1024 + n) -> n - 8, (1024 + 16 n) -> n - 8, (1024 + u) -> u - 128, each exact
__device__ __forceinline__ uint32_t low_codes(uint32_t x) {
    x = (x & 0x000f000fu) | 0x64006400u;
    return h2bits(__hadd2(*reinterpret_cast<const __half2 *>(&x), __half2half2(__ushort_as_half(0xE408))));
}
__device__ __forceinline__ uint32_t high_codes(uint32_t x) {
    x = (x & 0x00f000f0u) | 0x64006400u;
    return h2bits(__hfma2(*reinterpret_cast<const __half2 *>(&x), __half2half2(__ushort_as_half(0x2C00)), __half2half2(__ushort_as_half(0xD480))));
}
__device__ __forceinline__ uint32_t byte_codes(uint32_t x, uint32_t select) {
    x = __byte_perm(x, 0x64646464u, select);
    return h2bits(__hadd2(*reinterpret_cast<const __half2 *>(&x), __half2half2(__ushort_as_half(0xE480))));
}

template <typename T> __device__ __forceinline__ float value(T x);
template <> __device__ __forceinline__ float value<__half>(__half x) { return __half2float(x); }
template <> __device__ __forceinline__ float value<__nv_bfloat16>(__nv_bfloat16 x) { return __bfloat162float(x); }

template <typename T, bool kQ8, int D> __global__ void __launch_bounds__(kThreads, 4) kv_decode_kernel(const __grid_constant__ Args a) {
    using L = Tile<kQ8, D>;
    constexpr int ST = L::kStages, NB = D / 32;
    extern __shared__ __align__(128) uint8_t ring[];
    __shared__ uint64_t full[kWarps * ST];
    __shared__ int abort_s;
    __shared__ float ml_s[kWarps][kRows][2];         // each warp's maximum and sum (log2 domain)
    __shared__ float joined_s[kRows][2];             // the CTA's
    __shared__ float weight_s[kRows][kMaxCluster];
    const KvDecodeArgs &d = a.d;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, g = lane >> 2, t = lane & 3;
    const int rank = (int)cluster_rank(), ranks = (int)cluster_size();
    int64_t rest = blockIdx.x / ranks;
    const int split = int(rest % a.splits);
    rest /= a.splits;
    const int block = int(rest % a.row_blocks);
    rest /= a.row_blocks;
    const int hk = int(rest % d.shape.hk);
    const int64_t b = rest / d.shape.hk;
    const int head0 = hk * a.group + block * kRows, rows = min(a.group - block * kRows, kRows);

    const int len = (int)min(max(int64_t(d.lens[b]), int64_t(0)), d.max_len);
    const int tiles = (len + kTileKeys - 1) / kTileKeys;
    const int workers = a.splits * ranks * kWarps, me = (split * ranks + rank) * kWarps + warp;
    const int j0 = int(int64_t(tiles) * me / workers), n = int(int64_t(tiles) * (me + 1) / workers) - j0;

    const uint32_t my_ring = smem_u32(ring) + warp * ST * L::kBytes, my_full = smem_u32(full) + warp * ST * 8;
    if (tid == 0) abort_s = 0;
    if (lane == 0) {
        for (int i = 0; i < ST; ++i) mbar_init(my_full + 8 * i, 1);
        fence_mbar_init();
    }
    __syncthreads();
    volatile int *abort = &abort_s;

    // pages of the records 2 (j0 + i).. of 16 tiles, one a lane, and of the 16 after them: -1 for one that
    // does not exist, -2 past the last
    const int log2p = d.cache.page_log2, records = min((len + 15) / 16, 2 * (j0 + n));
    const int32_t *table = d.table + b * d.table_stride;
    auto pages_of = [&](int record) {
        if (record >= records) return -2;
        const int p = table[record >> (log2p - 4)];
        return p >= 0 && p < d.cache.n_pages ? p : -1;
    };
    int held = pages_of(2 * j0 + lane), next = pages_of(2 * j0 + 32 + lane);
    uint32_t missing = 0;  // two bits a stage: its records that were not copied
    const uint8_t *const head_base = d.cache.pages + (int64_t(hk) << (log2p - 4)) * L::kRec;
    const int in_page = (1 << (log2p - 4)) - 1;
    auto issue = [&](int i, int stg) {
        if ((i & 15) == 0 && i > 0) {
            held = next;
            next = pages_of(2 * (j0 + i) + 32 + lane);
        }
        const int p0 = __shfl_sync(0xffffffffu, held, 2 * (i & 15)), p1 = __shfl_sync(0xffffffffu, held, 2 * (i & 15) + 1);
        missing = (missing & ~(3u << (2 * stg))) | (uint32_t((p0 < 0) | (p1 < 0) << 1) << (2 * stg));
        if (lane == 0) {
            const uint32_t bar = my_full + 8 * stg, dst = my_ring + stg * L::kBytes;
            const int record = 2 * (j0 + i);
            const uint8_t *src = head_base + (record & in_page) * L::kRec;
            mbar_arrive_expect_tx(bar, ((p0 >= 0) + (p1 >= 0)) * L::kRec);
            if (p0 >= 0 && p1 >= 0 && in_page > 0) {
                bulk_g2s(dst, src + p0 * d.cache.page_stride, 2 * L::kRec, bar);
            } else {
                if (p0 >= 0) bulk_g2s(dst, src + p0 * d.cache.page_stride, L::kRec, bar);
                if (p1 >= 0)
                    bulk_g2s(dst + L::kRec, head_base + ((record + 1) & in_page) * L::kRec + p1 * d.cache.page_stride, L::kRec, bar);
            }
            if (p0 == -1 || p1 == -1) atomicMax(&reported, int(QMM_ERR_IDS));
        }
    };
    int issued = 0;
    if (a.fault != 1)
        for (; issued < ST && issued < n; ++issued) issue(issued, issued);

    // the warp's running softmax: head g (its lane's), and output elements of heads 2 t, 2 t + 1
    float top = -INFINITY, sum = 0.f, o[D / 16][4];
#pragma unroll
    for (int i = 0; i < D / 16; ++i) o[i][0] = o[i][1] = o[i][2] = o[i][3] = 0.f;
    if (n > 0) {
        uint32_t qa[NB][2][2];  // A fragments of two MMAs a block: k 2t, 2t + 1 and 2t + 8, 2t + 9 of row g
        float qc[NB], factor;
        {
            float v[NB][8], most = 0.f;
            const T *src = static_cast<const T *>(d.q) + b * d.sq.t + (head0 + g) * d.sq.h;
#pragma unroll
            for (int i = 0; i < NB; ++i)
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    v[i][j] = g < rows ? value<T>(src[32 * i + (kQ8 ? 4 * t + (j & 3) + (j >> 2) * 16 : 8 * t + j)]) : 0.f;
                    most = fmaxf(most, fabsf(v[i][j]));
                }
            most = fmaxf(most, __shfl_xor_sync(0xffffffffu, most, 1));
            most = fmaxf(most, __shfl_xor_sync(0xffffffffu, most, 2));
            // times 2^up: the largest element into [2^13, 2^14)
            const int up = most > 0.f ? max(-100, min(100, 140 - int(__float_as_uint(most) >> 23))) : 0;
            const float times = __int_as_float((127 + up) << 23);
            factor = a.scale_log2 * __int_as_float((127 + 12 - up / 2) << 23) * __int_as_float((127 + 12 - (up - up / 2)) << 23);
#pragma unroll
            for (int i = 0; i < NB; ++i) {
                float total = 0.f;
#pragma unroll
                for (int m = 0; m < 2; ++m) {
                    // nibbles 0, 4 (and 2, 6) as they are, 1, 5 (and 3, 7) 16 times as large; bytes in order
                    const float e[4] = {v[i][kQ8 ? 4 * m : 2 * m] * times, v[i][kQ8 ? 4 * m + 1 : 2 * m + 4] * times,
                                        v[i][kQ8 ? 4 * m + 2 : 2 * m + 1] * (kQ8 ? times : times * 0.0625f),
                                        v[i][kQ8 ? 4 * m + 3 : 2 * m + 5] * (kQ8 ? times : times * 0.0625f)};
                    qa[i][m][0] = pack2<__half>(e[0], e[1]);
                    qa[i][m][1] = pack2<__half>(e[2], e[3]);
                    const float2 x = halves(qa[i][m][0]), y = halves(qa[i][m][1]);
                    total += x.x + x.y + (kQ8 ? 1.f : 16.f) * (y.x + y.y);
                }
                total += __shfl_xor_sync(0xffffffffu, total, 1);
                total += __shfl_xor_sync(0xffffffffu, total, 2);
                qc[i] = total * (kQ8 ? -128.f : -8.f) * 0x1p-24f;
            }
        }
        int stg = 0, phase = 0;
        bool ok = a.fault != 2;
        int i = 0;
        for (; i < n && ok; ++i) {
            ok = warp_wait(my_full + 8 * stg, phase, abort, a.fault ? 100000 : kWaitCycles);
            if (!ok) break;
            const uint32_t tile = my_ring + stg * L::kBytes;
            const int valid = len - (j0 + i) * kTileKeys;
            const uint32_t lost = (missing >> (2 * stg)) & 3u;
            uint32_t seen = 0xffffffffu;
            if (valid < kTileKeys || lost) {
                // keys that nobody sees may hold anything: their value scales become zero, their scores minus infinity
                if (valid < kTileKeys) seen = (1u << valid) - 1;
                if (lost & 1) seen &= 0xffff0000u;
                if (lost & 2) seen &= 0x0000ffffu;
                for (int e = lane; e < 2 * NB * 16; e += 32) {
                    const int rec = e / (NB * 16), at = e % (NB * 16), place = at & 15;
                    const int token = 2 * (place >> 2) + (place & 1) + 8 * ((place >> 1) & 1);
                    if (!(seen >> (16 * rec + token) & 1u))
                        *reinterpret_cast<uint16_t *>(ring + (tile - smem_u32(ring)) + rec * L::kRec + L::kSide + L::kScales + at * 2) = 0;
                }
                fence_proxy_async_smem();
                __syncwarp();
            }
            float s[2][4];
#pragma unroll
            for (int r = 0; r < 2; ++r) {
                const uint32_t codes = tile + r * L::kRec;
                s[r][0] = s[r][1] = s[r][2] = s[r][3] = 0.f;
                uint32_t f[4];  // words of keys 0-7 and 8-15, of two units
#pragma unroll
                for (int blk = 0; blk < NB; ++blk) {
                    float acc[2][4];
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        acc[h][0] = acc[h][1] = qc[blk];
                        acc[h][2] = acc[h][3] = 0.f;
                    }
                    const uint32_t a0[4] = {qa[blk][0][0], 0, qa[blk][0][1], 0}, a1[4] = {qa[blk][1][0], 0, qa[blk][1][1], 0};
                    if constexpr (kQ8) {
                        ldsm4(f, codes + blk * 512 + lane * 16);
#pragma unroll
                        for (int h = 0; h < 2; ++h) {
                            mma16816<__half>(acc[h], a0, __byte_perm(f[h], 0, 0x4140), __byte_perm(f[h], 0, 0x4342));
                            mma16816<__half>(acc[h], a1, __byte_perm(f[2 + h], 0, 0x4140), __byte_perm(f[2 + h], 0, 0x4342));
                        }
                    } else {
                        if ((blk & 1) == 0) {
                            if (blk + 1 < NB) ldsm4(f, codes + blk * 256 + lane * 16);
                            else ldsm2(f, codes + blk * 256 + (lane & 15) * 16);
                        }
#pragma unroll
                        for (int h = 0; h < 2; ++h) {
                            const uint32_t x = f[(blk & 1) * 2 + h], y = x >> 8;
                            mma16816<__half>(acc[h], a0, x & 0x000f000fu, x & 0x00f000f0u);
                            mma16816<__half>(acc[h], a1, y & 0x000f000fu, y & 0x00f000f0u);
                        }
                    }
                    const uint2 sc = lds64(codes + L::kScales + blk * 32 + t * 8);
                    const float2 lo = halves(sc.x), hi = halves(sc.y);
                    s[r][0] += lo.x * acc[0][0];
                    s[r][1] += lo.y * acc[0][1];
                    s[r][2] += hi.x * acc[1][0];
                    s[r][3] += hi.y * acc[1][1];
                }
            }
            float m = -INFINITY;
#pragma unroll
            for (int r = 0; r < 2; ++r)
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    s[r][e] *= factor;
                    if (seen != 0xffffffffu && !(seen >> (16 * r + 2 * t + (e & 1) + 8 * (e >> 1)) & 1u)) s[r][e] = -INFINITY;
                    m = fmaxf(m, s[r][e]);
                }
            m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, 1));
            m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, 2));
            if (__any_sync(0xffffffffu, m > top)) {
                const float now = fmaxf(top, m);
                const float f = top == -INFINITY ? 1.f : ex2(top - now);
                top = now;
                sum *= f;
                const float f0 = __shfl_sync(0xffffffffu, f, t * 8), f1 = __shfl_sync(0xffffffffu, f, t * 8 + 4);
#pragma unroll
                for (int c = 0; c < D / 16; ++c) {
                    o[c][0] *= f0;
                    o[c][1] *= f1;
                    o[c][2] *= f0;
                    o[c][3] *= f1;
                }
            }
            const float base = top == -INFINITY ? 0.f : top;
#pragma unroll
            for (int r = 0; r < 2; ++r)
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    s[r][e] = ex2(s[r][e] - base);
                    sum += s[r][e];
                }
#pragma unroll
            for (int r = 0; r < 2; ++r) {
                const uint32_t codes = tile + r * L::kRec + L::kSide;
                const uint32_t p0 = pack2<__half>(s[r][0], s[r][1]), p1 = pack2<__half>(s[r][2], s[r][3]);
                uint32_t f[4];
#pragma unroll
                for (int blk = 0; blk < NB; ++blk) {
                    const uint2 sc = lds64(codes + L::kScales + blk * 32 + t * 8);
                    uint32_t w0, w1;  // weights times scales, of keys 2t, 2t + 1 and 2t + 8, 2t + 9
                    if constexpr (std::is_same<T, __half>::value) {
                        const float2 lo = halves(sc.x), hi = halves(sc.y);  // one rounding: the output's own is as fine
                        w0 = pack2<__half>(s[r][0] * lo.x, s[r][1] * lo.y);
                        w1 = pack2<__half>(s[r][2] * hi.x, s[r][3] * hi.y);
                    } else {
                        w0 = mul2(p0, sc.x);
                        w1 = mul2(p1, sc.y);
                    }
                    if constexpr (kQ8) {
                        ldsm4_t(f, codes + blk * 512 + lane * 16);
#pragma unroll
                        for (int m2 = 0; m2 < 2; ++m2) {
                            const uint32_t av[4] = {byte_codes(f[2 * m2], 0x4240), byte_codes(f[2 * m2], 0x4341),
                                                    byte_codes(f[2 * m2 + 1], 0x4240), byte_codes(f[2 * m2 + 1], 0x4341)};
                            mma16816<__half>(o[2 * blk + m2], av, w0, w1);
                        }
                    } else {
                        if ((blk & 1) == 0) {
                            if (blk + 1 < NB) ldsm4_t(f, codes + blk * 256 + lane * 16);
                            else ldsm2_t(f, codes + blk * 256 + (lane & 15) * 16);
                        }
                        const uint32_t x = f[(blk & 1) * 2], y = f[(blk & 1) * 2 + 1];
                        const uint32_t a0[4] = {low_codes(x), high_codes(x), low_codes(y), high_codes(y)};
                        const uint32_t a1[4] = {low_codes(x >> 8), high_codes(x >> 8), low_codes(y >> 8), high_codes(y >> 8)};
                        mma16816<__half>(o[2 * blk], a0, w0, w1);
                        mma16816<__half>(o[2 * blk + 1], a1, w0, w1);
                    }
                }
            }
            __syncwarp();
            if (issued < n) {
                issue(issued, stg);
                ++issued;
            }
            if (++stg == ST) {
                stg = 0;
                phase ^= 1;
            }
        }
        if (!ok) {  // copies in flight land before the ring is reused or released
            *abort = 1;
            for (int k = i; k < issued; ++k) {
                int never = 0;
                mbar_wait(my_full + 8 * (k % ST), (k / ST) & 1, &never);
            }
        }
        sum += __shfl_xor_sync(0xffffffffu, sum, 1);
        sum += __shfl_xor_sync(0xffffffffu, sum, 2);
    }
    __syncthreads();  // the ring is free
    float *part = reinterpret_cast<float *>(ring);
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        const int row = 2 * t + h;
        float *dst = part + (warp * kRows + row) * L::kStride;
        if (row >= rows) continue;
#pragma unroll
        for (int blk = 0; blk < NB; ++blk) {
            if constexpr (kQ8) {
                *reinterpret_cast<float2 *>(dst + 32 * blk + 2 * g) = make_float2(o[2 * blk][h], o[2 * blk][2 + h]);
                *reinterpret_cast<float2 *>(dst + 32 * blk + 16 + 2 * g) = make_float2(o[2 * blk + 1][h], o[2 * blk + 1][2 + h]);
            } else {
                *reinterpret_cast<float4 *>(dst + 32 * blk + 4 * g) =
                    make_float4(o[2 * blk][h], o[2 * blk][2 + h], o[2 * blk + 1][h], o[2 * blk + 1][2 + h]);
            }
        }
    }
    if (t == 0) {
        ml_s[warp][g][0] = top;
        ml_s[warp][g][1] = sum;
    }
    __syncthreads();
    // the warps' rows joined into the first warp's
    constexpr int kQuads = D / 4;
    for (int e = tid; e < rows * kQuads; e += kThreads) {
        const int row = e / kQuads, col = (e % kQuads) * 4;
        float m[kWarps], most = -INFINITY;
#pragma unroll
        for (int w = 0; w < kWarps; ++w) most = fmaxf(most, m[w] = ml_s[w][row][0]);
        const float base = most == -INFINITY ? 0.f : most;
        float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
        float total = 0.f;
#pragma unroll
        for (int w = 0; w < kWarps; ++w) {
            const float f = ex2(m[w] - base);
            const float4 x = *reinterpret_cast<const float4 *>(part + (w * kRows + row) * L::kStride + col);
            acc.x += f * x.x;
            acc.y += f * x.y;
            acc.z += f * x.z;
            acc.w += f * x.w;
            total += f * ml_s[w][row][1];
        }
        *reinterpret_cast<float4 *>(part + row * L::kStride + col) = acc;
        if (col == 0) {
            joined_s[row][0] = most;
            joined_s[row][1] = total;
        }
    }
    if (*abort && tid == 0) atomicMax(&reported, int(QMM_ERR_DEVICE));
    if (ranks > 1) cluster_sync();
    else __syncthreads();

    // ------------------------------------------------ the cluster's rows
    const int64_t row0 = b * d.shape.hq + head0, all_rows = d.batch * d.shape.hq;
    for (int row = warp; row < rows; row += kWarps) {
        float m = -INFINITY, l = 0.f;
        if (ranks == 1) {
            m = lane == 0 ? joined_s[row][0] : m;
            l = lane == 0 ? joined_s[row][1] : l;
        } else if (lane < ranks) {
            m = peer_f32(smem_u32(&joined_s[row][0]), lane);
            l = peer_f32(smem_u32(&joined_s[row][1]), lane);
        }
        float most = m;
#pragma unroll
        for (int x = 16; x > 0; x >>= 1) most = fmaxf(most, __shfl_xor_sync(0xffffffffu, most, x));
        const float base = most == -INFINITY ? 0.f : most;
        const float w = ex2(m - base);
        float total = w * l;
#pragma unroll
        for (int x = 16; x > 0; x >>= 1) total += __shfl_xor_sync(0xffffffffu, total, x);
        const bool none = !(total != 0.f);
        if (lane < ranks) weight_s[row][lane] = none ? 0.f : w / total;
        if (lane == 0 && rank == 0) {
            const float log2_total = none ? -INFINITY : base + log2f(total);
            if (a.splits > 1) a.part_lse[split * all_rows + row0 + row] = log2_total;
            else if (d.lse) d.lse[row0 + row] = log2_total * kLn2;
        }
    }
    __syncthreads();
    for (int e = rank + tid * ranks; e < rows * kQuads; e += ranks * kThreads) {
        const int row = e / kQuads, col = (e % kQuads) * 4;
        float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
        const uint32_t addr = smem_u32(part + row * L::kStride + col);
#pragma unroll 4
        for (int p = 0; p < ranks; ++p) {
            const float w = weight_s[row][p];
            const float4 x = ranks == 1 ? *reinterpret_cast<const float4 *>(part + row * L::kStride + col) : peer_f32x4(addr, p);
            acc.x += w * x.x;
            acc.y += w * x.y;
            acc.z += w * x.z;
            acc.w += w * x.w;
        }
        if (a.splits > 1) {
            *reinterpret_cast<float4 *>(a.part + (split * all_rows + row0 + row) * D + col) = acc;
        } else {
            T *out = static_cast<T *>(d.out) + b * d.so.t + (head0 + row) * d.so.h + col;
            *reinterpret_cast<uint2 *>(out) = make_uint2(pack2<T>(acc.x, acc.y), pack2<T>(acc.z, acc.w));
        }
    }
    if (ranks > 1) cluster_sync();  // no CTA leaves while its shared memory may be read
}

// Rows of several clusters joined, a warp a row.
template <typename T> __global__ void __launch_bounds__(128) kv_join_kernel(const __grid_constant__ Args a) {
    const KvDecodeArgs &d = a.d;
    const int lane = threadIdx.x & 31;
    const int64_t rows = d.batch * d.shape.hq, row = int64_t(blockIdx.x) * 4 + (threadIdx.x >> 5);
    grid_dependency_wait();
    if (row >= rows) return;
    float l[2], most = -INFINITY;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const int p = lane + 32 * i;
        l[i] = p < a.splits ? __ldcg(a.part_lse + p * rows + row) : -INFINITY;
        most = fmaxf(most, l[i]);
    }
#pragma unroll
    for (int x = 16; x > 0; x >>= 1) most = fmaxf(most, __shfl_xor_sync(0xffffffffu, most, x));
    const float base = most == -INFINITY ? 0.f : most;
    float w[2] = {ex2(l[0] - base), ex2(l[1] - base)}, total = w[0] + w[1];
#pragma unroll
    for (int x = 16; x > 0; x >>= 1) total += __shfl_xor_sync(0xffffffffu, total, x);
    const bool none = !(total != 0.f);
    const float inv = none ? 0.f : 1.f / total;
    if (d.lse && lane == 0) d.lse[row] = none ? -INFINITY : (base + log2f(total)) * kLn2;
    const int D = d.shape.d, col = lane * 4;
    float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
    for (int p = 0; p < a.splits; ++p) {
        const float f = __shfl_sync(0xffffffffu, p < 32 ? w[0] : w[1], p & 31) * inv;
        if (col >= D) continue;
        const float4 x = __ldcg(reinterpret_cast<const float4 *>(a.part + (p * rows + row) * D + col));
        acc.x += f * x.x;
        acc.y += f * x.y;
        acc.z += f * x.z;
        acc.w += f * x.w;
    }
    if (col >= D) return;
    T *out = static_cast<T *>(d.out) + row / d.shape.hq * d.so.t + row % d.shape.hq * d.so.h + col;
    *reinterpret_cast<uint2 *>(out) = make_uint2(pack2<T>(acc.x, acc.y), pack2<T>(acc.z, acc.w));
}

size_t align256(size_t x) { return (x + 255) & ~size_t(255); }

struct Plan {
    int ranks, splits;
};

// CTAs of a cluster (a power of two) and clusters of one request and kv head.
Plan plan(const KvDecodeArgs &d) {
    const int64_t group = d.shape.hq / d.shape.hk, pairs = d.batch * d.shape.hk * ((group + kRows - 1) / kRows);
    const int64_t tiles = (d.max_len + kTileKeys - 1) / kTileKeys, room = 3 * device_sm_count();
    Plan p{1, 1};
    while (p.ranks < kMaxCluster && tiles >= 2 * p.ranks * kWarps && (pairs * 2 * p.ranks <= room || tiles >= 128 * kWarps * p.ranks)) p.ranks *= 2;
    while (p.ranks == kMaxCluster && p.splits < kMaxParts && pairs * kMaxCluster * (p.splits + 1) <= room &&
           tiles >= int64_t(8) * kMaxCluster * kWarps * (p.splits + 1))
        ++p.splits;
    return p;
}

template <typename T, bool kQ8, int D> cudaError_t launch(const Args &a, Plan p, int64_t pairs, cudaStream_t st) {
    using L = Tile<kQ8, D>;
    auto kern = kv_decode_kernel<T, kQ8, D>;
    cudaError_t e = ensure_smem(kern, L::kSmem);
    if (e != cudaSuccess) return e;
    if (p.ranks > 8) {
        e = cudaFuncSetAttribute(kern, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
        if (e != cudaSuccess) return e;
    }
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3((unsigned)(pairs * p.ranks * p.splits));
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = L::kSmem;
    cfg.stream = st;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = p.ranks;
    attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    e = cudaLaunchKernelEx(&cfg, kern, a);
    if (e != cudaSuccess || p.splits == 1) return e;
    return launch_pdl(kv_join_kernel<T>, dim3((unsigned)((a.d.batch * a.d.shape.hq + 3) / 4)), dim3(128), 0, st, a);
}

template <typename T, bool kQ8> cudaError_t launch_d(const Args &a, Plan p, int64_t pairs, cudaStream_t st) {
    switch (a.d.shape.d) {
        case 32: return launch<T, kQ8, 32>(a, p, pairs, st);
        case 64: return launch<T, kQ8, 64>(a, p, pairs, st);
        case 96: return launch<T, kQ8, 96>(a, p, pairs, st);
        default: return launch<T, kQ8, 128>(a, p, pairs, st);
    }
}

}  // namespace

cudaError_t kv_decode_take_error(int *code, cudaStream_t st) { return take_error(code, st); }

size_t kv_decode_workspace_bytes(const KvDecodeArgs &d) {
    const Plan p = plan(d);
    if (p.splits == 1) return 0;
    const size_t rows = size_t(p.splits) * d.batch * d.shape.hq;
    return align256(rows * d.shape.d * 4) + align256(rows * 4);
}

cudaError_t launch_kv_decode(const KvDecodeArgs &d, qmm_float t, void *ws, cudaStream_t st) {
    const Plan p = plan(d);
    Args a{};
    a.d = d;
    a.group = d.shape.hq / d.shape.hk;
    a.row_blocks = (a.group + kRows - 1) / kRows;
    a.splits = p.splits;
    a.scale_log2 = d.scale * kLog2e;
    a.fault = test_fault_mode();
    if (p.splits > 1) {
        a.part = static_cast<float *>(ws);
        a.part_lse = reinterpret_cast<float *>(static_cast<uint8_t *>(ws) +
                                               align256(size_t(p.splits) * d.batch * d.shape.hq * d.shape.d * 4));
    }
    const int64_t pairs = d.batch * d.shape.hk * a.row_blocks;
    if (pairs * p.ranks * p.splits > 0x7fffffff) return cudaErrorInvalidConfiguration;
    if (t == QMM_F16) return d.cache.q8 ? launch_d<__half, true>(a, p, pairs, st) : launch_d<__half, false>(a, p, pairs, st);
    return d.cache.q8 ? launch_d<__nv_bfloat16, true>(a, p, pairs, st) : launch_d<__nv_bfloat16, false>(a, p, pairs, st);
}

}  // namespace qmm
