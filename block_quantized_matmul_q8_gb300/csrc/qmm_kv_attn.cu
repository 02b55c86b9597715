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
//   - values: the block's scale multiplies the weights, p d_jb rounded to fp16 (11 bits; below
//     2^-14 an absolute 2^-25); codes enter as subnormals too, and a second MMA adds -bias times the same weights
//     to the same fp32 sums, at once, so that the sums stay as small as the output.
//   - keys are the MMA's 16 rows and query heads its 8 columns, so that no row is empty; the weights reach the
//     second product's layout by movmatrix.  Codes come by ldmatrix with neighbouring codes in one 16-bit unit,
//     transposed for V, so that a nibble's mask gives the pairs of keys or elements that the MMA wants.
// A warp takes tiles of 32 keys on its own: a private ring of bulk copies (a record of 16 tokens is
// contiguous), its running softmax, no barrier with other warps until the join.
//
// Two ways to share the work out.  Calls that fit the SMs at once: a cluster of up to 16 CTAs takes one request
// and kv head and joins through distributed shared memory, one launch.  Larger ones: the tiles of all
// requests lie in one row that resident CTAs cut into equal parts (each scans the lengths on the device), and a second
// launch joins the requests that were cut.  mma.sync: 8 query heads would leave tcgen05's 128 rows empty.
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
constexpr int kMaxFlatBatch = 1024;
constexpr int kCtas = 4;         // of one SM
constexpr int kPieceUnits = 4;   // what a piece costs beside its tiles, in tiles

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
    float scale_log2;
    int ctas;               // of the flat form
    float *part, *part_lse; // [ctas][first or last piece][8][d] normalised, their log2 denominators
    int4 *cuts;             // [ctas]: request, pair, piece and number of parts that begin in the CTA's last piece
    int fault;              // as in qmm_attn.cu
};

__device__ __forceinline__ int request_tiles(const KvDecodeArgs &d, int64_t b) {
    return (int)((min(max(int64_t(d.lens[b]), int64_t(0)), d.max_len) + kTileKeys - 1) / kTileKeys);
}
// The flat form's row has kPieceUnits units and one for each tile for every request and kv head, so that
// a CTA of many short pieces gets fewer tiles.  CTA c takes the units [total c / ctas, total (c + 1) / ctas) of it.
__device__ __forceinline__ int64_t cut(int64_t total, int c, int ctas) { return total * c / ctas; }
__device__ __forceinline__ int cta_of(int64_t total, int64_t unit, int ctas) { return int(((unit + 1) * ctas - 1) / total); }
__device__ __forceinline__ int units_of(int tiles) { return tiles > 0 ? tiles + kPieceUnits : 0; }

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
template <typename T> __device__ __forceinline__ float value(T x);
template <> __device__ __forceinline__ float value<__half>(__half x) { return __half2float(x); }
template <> __device__ __forceinline__ float value<__nv_bfloat16>(__nv_bfloat16 x) { return __bfloat162float(x); }

__device__ __forceinline__ uint32_t transpose8x8(uint32_t x) {
    uint32_t y;
    asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
    return y;
}
// c = a b + first
__device__ __forceinline__ void mma_first(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                          uint32_t b1, const float (&first)[4]) {
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%10,%11,%12,%13};"
        : "=f"(c[0]), "=f"(c[1]), "=f"(c[2]), "=f"(c[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(first[0]), "f"(first[1]), "f"(first[2]), "f"(first[3]));
}
__device__ __forceinline__ void mma_more(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0, uint32_t b1) {
    const uint32_t a[4] = {a0, a1, a2, a3};
    mma16816<__half>(c, a, b0, b1);
}

template <typename T, bool kQ8, int D, bool kFlat> __global__ void __launch_bounds__(kThreads, kCtas) kv_decode_kernel(const __grid_constant__ Args a) {
    using L = Tile<kQ8, D>;
    constexpr int ST = L::kStages, NB = D / 32, kQuads = D / 4;
    extern __shared__ __align__(128) uint8_t ring[];
    __shared__ uint64_t full[kWarps * ST];
    __shared__ int abort_s;
    __shared__ float ml_s[kWarps][kRows][2];         // each warp's maximum and sum (log2 domain)
    __shared__ float joined_s[kRows][2];             // the CTA's
    __shared__ float weight_s[kRows][kMaxCluster];
    __shared__ int warp_sum_s[kWarps];
    const KvDecodeArgs &d = a.d;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, g = lane >> 2, t = lane & 3;
    const int rank = kFlat ? 0 : (int)cluster_rank(), ranks = kFlat ? 1 : (int)cluster_size();
    const int pairs = d.shape.hk * a.row_blocks;     // of a request

    const uint32_t my_ring = smem_u32(ring) + warp * ST * L::kBytes, my_full = smem_u32(full) + warp * ST * 8;
    if (tid == 0) abort_s = 0;
    if (lane == 0) {
        for (int i = 0; i < ST; ++i) mbar_init(my_full + 8 * i, 2);
        fence_mbar_init();
    }
    // the pieces: some tiles each of one request and kv head
    int64_t b, begin = 0, end = 0, total = 1;  // the piece's request, its first unit, the CTA's last, all units
    int pair, tiles, first = 0;                // its heads, all its tiles, the first of this CTA
    if (kFlat) {
        int *const before = reinterpret_cast<int *>(ring);  // units of one head of the requests up to this one
        int sum = 0;
        for (int base = 0; base < d.batch; base += kThreads) {
            int v = base + tid < d.batch ? units_of(request_tiles(d, base + tid)) : 0;
#pragma unroll
            for (int s = 1; s < 32; s <<= 1) {
                const int u = __shfl_up_sync(0xffffffffu, v, s);
                if (lane >= s) v += u;
            }
            if (lane == 31) warp_sum_s[warp] = v;
            __syncthreads();
            int here = 0;
#pragma unroll
            for (int w = 0; w < kWarps; ++w) {
                if (w == warp) v += sum + here;
                here += warp_sum_s[w];
            }
            if (base + tid < d.batch) before[base + tid] = v;
            sum += here;
            __syncthreads();
        }
        total = int64_t(sum) * pairs;
        const int64_t x = cut(total, blockIdx.x, a.ctas);
        end = cut(total, blockIdx.x + 1, a.ctas);
        int lo = 0, hi = (int)d.batch - 1;  // the first request that ends after x
        while (lo < hi) {
            const int mid = (lo + hi) / 2;
            if (int64_t(before[mid]) * pairs > x) hi = mid;
            else lo = mid + 1;
        }
        b = lo;
        const int start = lo > 0 ? before[lo - 1] : 0, units = max(before[lo] - start, kPieceUnits);
        tiles = units - kPieceUnits;
        begin = int64_t(start) * pairs;
        pair = int((x - begin) / units);
        begin += int64_t(pair) * units;
        first = max(int(x - begin) - kPieceUnits, 0);
        fence_proxy_async_smem();  // the sums' place is the ring from here on
    } else {
        const int64_t at = blockIdx.x / ranks;
        b = at / pairs;
        pair = int(at - b * pairs);
        tiles = request_tiles(d, b);
    }
    int4 cut_here = make_int4(0, 0, 0, 0);
    __syncthreads();
    volatile int *abort = &abort_s;
    int stg = 0, phase = 0;  // the warp's next stage

    for (int slot = 0;; slot = 1) {
        bool whole = true;
        int j0, n;  // tiles of the warp
        if (kFlat) {
            const int count = int(min(end - begin - kPieceUnits, int64_t(tiles))) - first;
            if (count <= 0) break;
            whole = count == tiles;
            if (!whole && first == 0)
                cut_here = make_int4(int(b), pair, slot, cta_of(total, begin + units_of(tiles) - 1, a.ctas) - int(blockIdx.x) + 1);
            j0 = first + int(int64_t(count) * warp / kWarps);
            n = first + int(int64_t(count) * (warp + 1) / kWarps) - j0;
        } else {
            const int64_t workers = ranks * kWarps, me = rank * kWarps + warp;
            j0 = int(tiles * me / workers);
            n = int(tiles * (me + 1) / workers) - j0;
        }
        const int hk = pair / a.row_blocks, block = pair - hk * a.row_blocks;
        const int head0 = hk * a.group + block * kRows, rows = min(a.group - block * kRows, kRows);
        const int len = (int)min(max(int64_t(d.lens[b]), int64_t(0)), d.max_len);

        // where the records 2 (j0 + i).. of 16 tiles lie, one a lane, and the pages of the 16 tiles after them: -1 for
        // a page that does not exist, -2 past the last
        const int log2g = d.cache.page_log2 - 4, records = min((len + 15) / 16, 2 * (j0 + n));
        const int32_t *const table = d.table + b * d.table_stride;
        auto page_of = [&](int record) {
            if (record >= records) return -2;
            const int p = table[record >> log2g];
            return p >= 0 && p < d.cache.n_pages ? p : -1;
        };
        auto source = [&](int record, int page) {
            if (page == -1) atomicMax(&reported, int(QMM_ERR_IDS));
            const int64_t at = (int64_t(hk) << log2g) + (record & ((1 << log2g) - 1));
            return page >= 0 ? d.cache.pages + page * d.cache.page_stride + at * L::kRec : nullptr;
        };
        const uint8_t *src = source(2 * j0 + lane, page_of(2 * j0 + lane));
        int next = page_of(2 * j0 + 32 + lane);
        uint32_t missing_ahead = __ballot_sync(0xffffffffu, !src), missing = missing_ahead;  // records that are not copied
        auto issue = [&](int i, int to) {  // the lanes of its two records copy a tile
            if ((i & 15) == 0 && i > 0) {
                const int record = 2 * (j0 + i) + lane;
                src = source(record, next);
                next = page_of(record + 32);
                missing_ahead = __ballot_sync(0xffffffffu, !src);
            }
            if ((lane >> 1) == (i & 15)) {
                const uint32_t bar = my_full + 8 * to;
                if (src) {
                    mbar_arrive_expect_tx(bar, L::kRec);
                    bulk_g2s(my_ring + to * L::kBytes + (lane & 1) * L::kRec, src, L::kRec, bar);
                } else {
                    mbar_arrive(bar);
                }
            }
        };
        int issued = 0;
        if (a.fault != 1)
            for (; issued < ST && issued < n; ++issued) issue(issued, stg + issued < ST ? stg + issued : stg + issued - ST);

        // the warp's running softmax of heads 2 t, 2 t + 1: its keys are those of lanes with the same t
        float top[2] = {-INFINITY, -INFINITY}, sum[2] = {0.f, 0.f}, o[D / 16][4];
#pragma unroll
        for (int i = 0; i < D / 16; ++i) o[i][0] = o[i][1] = o[i][2] = o[i][3] = 0.f;
        if (n > 0) {
            uint32_t qb[NB][2][2];  // B fragments of two MMAs a block: k 2t, 2t + 1 and 2t + 8, 2t + 9 of head g
            float qc[NB][4], factor[2];  // the accumulators' first values
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
                // times 2^up: the largest element into [2^13, 2^14); a negative scale turns the queries
                const int up = most > 0.f ? max(-100, min(100, 140 - int(__float_as_uint(most) >> 23))) : 0;
                const float times = copysignf(__int_as_float((127 + up) << 23), a.scale_log2);
                const float f = fabsf(a.scale_log2) * __int_as_float((127 + 12 - up / 2) << 23) * __int_as_float((127 + 12 - (up - up / 2)) << 23);
                factor[0] = __shfl_sync(0xffffffffu, f, 8 * t);
                factor[1] = __shfl_sync(0xffffffffu, f, 8 * t + 4);
#pragma unroll
                for (int i = 0; i < NB; ++i) {
                    float total = 0.f;
#pragma unroll
                    for (int m = 0; m < 2; ++m) {
                        // nibbles 0, 4 (and 2, 6) as they are, 1, 5 (and 3, 7) 16 times as large; bytes in order
                        const float e[4] = {v[i][kQ8 ? 4 * m : 2 * m] * times, v[i][kQ8 ? 4 * m + 1 : 2 * m + 4] * times,
                                            v[i][kQ8 ? 4 * m + 2 : 2 * m + 1] * (kQ8 ? times : times * 0.0625f),
                                            v[i][kQ8 ? 4 * m + 3 : 2 * m + 5] * (kQ8 ? times : times * 0.0625f)};
                        qb[i][m][0] = pack2<__half>(e[0], e[1]);
                        qb[i][m][1] = pack2<__half>(e[2], e[3]);
                        const float2 y = halves(qb[i][m][0]), z = halves(qb[i][m][1]);
                        total += y.x + y.y + (kQ8 ? 1.f : 16.f) * (z.x + z.y);
                    }
                    total += __shfl_xor_sync(0xffffffffu, total, 1);
                    total += __shfl_xor_sync(0xffffffffu, total, 2);
                    total *= (kQ8 ? -128.f : -8.f) * 0x1p-24f;
#pragma unroll
                    for (int e = 0; e < 4; ++e) qc[i][e] = __shfl_sync(0xffffffffu, total, 8 * t + 4 * (e & 1));
                }
            }
            const uint32_t odd = (g & 1) ? 0x7632u : 0x5410u;  // halves of keys g and g + 8 out of four scales
            bool ok = a.fault != 2;
            int i = 0;
            for (; i < n && ok; ++i) {
                ok = warp_wait(my_full + 8 * stg, phase, abort, a.fault ? 100000 : kWaitCycles);
                if (!ok) break;
                const uint32_t tile = my_ring + stg * L::kBytes;
                const int valid = len - (j0 + i) * kTileKeys;
                if ((i & 15) == 0 && i > 0) missing = missing_ahead;
                const uint32_t lost = (missing >> (2 * (i & 15))) & 3u;
                uint32_t seen = 0xffffffffu;
                if (valid < kTileKeys || lost) {
                    // keys that nobody sees may hold anything: their value scales become zero, their weights too
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
                // scores of keys g (first two) and g + 8 of both records, heads 2 t and 2 t + 1
                float s[2][4];
#pragma unroll
                for (int r = 0; r < 2; ++r) {
                    const uint32_t codes = tile + r * L::kRec;
                    uint32_t f[4];  // words of keys 0-7 and 8-15, of two units
#pragma unroll
                    for (int blk = 0; blk < NB; ++blk) {
                        float acc[4];
                        const uint32_t(&q0)[2] = qb[blk][0], (&q1)[2] = qb[blk][1];
                        if constexpr (kQ8) {
                            ldsm4(f, codes + blk * 512 + lane * 16);
                            mma_first(acc, __byte_perm(f[0], 0, 0x4140), __byte_perm(f[1], 0, 0x4140), __byte_perm(f[0], 0, 0x4342),
                                      __byte_perm(f[1], 0, 0x4342), q0[0], q0[1], qc[blk]);
                            mma_more(acc, __byte_perm(f[2], 0, 0x4140), __byte_perm(f[3], 0, 0x4140), __byte_perm(f[2], 0, 0x4342),
                                     __byte_perm(f[3], 0, 0x4342), q1[0], q1[1]);
                        } else {
                            if ((blk & 1) == 0) {
                                if (blk + 1 < NB) ldsm4(f, codes + blk * 256 + lane * 16);
                                else ldsm2(f, codes + blk * 256 + (lane & 15) * 16);
                            }
                            constexpr uint32_t lo = 0x000f000fu, hi = 0x00f000f0u;
                            const uint32_t y = f[(blk & 1) * 2], z = f[(blk & 1) * 2 + 1];
                            mma_first(acc, y & lo, z & lo, y & hi, z & hi, q0[0], q0[1], qc[blk]);
                            mma_more(acc, y >> 8 & lo, z >> 8 & lo, y >> 8 & hi, z >> 8 & hi, q1[0], q1[1]);
                        }
                        const uint2 sc = lds64(codes + L::kScales + blk * 32 + (g >> 1) * 8);
                        const float2 ks = halves(__byte_perm(sc.x, sc.y, odd));
                        if (blk == 0) {
                            s[r][0] = ks.x * acc[0];
                            s[r][1] = ks.x * acc[1];
                            s[r][2] = ks.y * acc[2];
                            s[r][3] = ks.y * acc[3];
                        } else {
                            s[r][0] += ks.x * acc[0];
                            s[r][1] += ks.x * acc[1];
                            s[r][2] += ks.y * acc[2];
                            s[r][3] += ks.y * acc[3];
                        }
                    }
                }
                if (seen != 0xffffffffu) {
#pragma unroll
                    for (int r = 0; r < 2; ++r)
#pragma unroll
                        for (int e = 0; e < 4; ++e)
                            if (!(seen >> (16 * r + g + 8 * (e >> 1)) & 1u)) s[r][e] = -INFINITY;
                }
                float m[2];
#pragma unroll
                for (int h = 0; h < 2; ++h) m[h] = fmaxf(fmaxf(s[0][h], s[0][2 + h]), fmaxf(s[1][h], s[1][2 + h]));
                if (__any_sync(0xffffffffu, m[0] > top[0] || m[1] > top[1])) {
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
#pragma unroll
                        for (int y = 4; y < 32; y <<= 1) m[h] = fmaxf(m[h], __shfl_xor_sync(0xffffffffu, m[h], y));
                        const float now = fmaxf(top[h], m[h]);
                        const float f = top[h] == -INFINITY ? 1.f : ex2((top[h] - now) * factor[h]);
                        top[h] = now;
                        sum[h] *= f;
#pragma unroll
                        for (int c = 0; c < D / 16; ++c) {
                            o[c][h] *= f;
                            o[c][2 + h] *= f;
                        }
                    }
                }
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    const float base = top[h] == -INFINITY ? 0.f : top[h] * factor[h];
#pragma unroll
                    for (int r = 0; r < 2; ++r)
#pragma unroll
                        for (int e = h; e < 4; e += 2) s[r][e] = ex2(fmaf(s[r][e], factor[h], -base));
                }
                if (seen != 0xffffffffu) {  // again, for a factor of zero
#pragma unroll
                    for (int r = 0; r < 2; ++r)
#pragma unroll
                        for (int e = 0; e < 4; ++e)
                            if (!(seen >> (16 * r + g + 8 * (e >> 1)) & 1u)) s[r][e] = 0.f;
                }
#pragma unroll
                for (int h = 0; h < 2; ++h) sum[h] += (s[0][h] + s[0][2 + h]) + (s[1][h] + s[1][2 + h]);
#pragma unroll
                for (int r = 0; r < 2; ++r) {
                    const uint32_t codes = tile + r * L::kRec + L::kSide;
                    constexpr bool kExact = std::is_same<T, __half>::value;  // one rounding, the output's own is as fine
                    uint32_t p0 = 0, p1 = 0;
                    if (!kExact) {
                        p0 = transpose8x8(pack2<__half>(s[r][0], s[r][1]));
                        p1 = transpose8x8(pack2<__half>(s[r][2], s[r][3]));
                    }
                    uint32_t f[4];
#pragma unroll
                    for (int blk = 0; blk < NB; ++blk) {
                        uint32_t w0, w1;  // weights times scales of head g, keys 2t, 2t + 1 and 2t + 8, 2t + 9
                        if (kExact) {
                            const uint2 sc = lds64(codes + L::kScales + blk * 32 + (g >> 1) * 8);
                            const float2 vs = halves(__byte_perm(sc.x, sc.y, odd));
                            w0 = transpose8x8(pack2<__half>(s[r][0] * vs.x, s[r][1] * vs.x));
                            w1 = transpose8x8(pack2<__half>(s[r][2] * vs.y, s[r][3] * vs.y));
                        } else {
                            const uint2 sc = lds64(codes + L::kScales + blk * 32 + t * 8);
                            w0 = mul2(p0, sc.x);
                            w1 = mul2(p1, sc.y);
                        }
                        // codes as they are, and then the bias times the same weights
                        if constexpr (kQ8) {
                            ldsm4_t(f, codes + blk * 512 + lane * 16);
#pragma unroll
                            for (int u = 0; u < 2; ++u) {
                                const uint32_t y = f[2 * u], z = f[2 * u + 1];
                                mma_more(o[2 * blk + u], __byte_perm(y, 0, 0x4240), __byte_perm(y, 0, 0x4341), __byte_perm(z, 0, 0x4240),
                                         __byte_perm(z, 0, 0x4341), w0, w1);
                                mma_more(o[2 * blk + u], 0x80808080u, 0x80808080u, 0x80808080u, 0x80808080u, w0, w1);
                            }
                        } else {
                            if ((blk & 1) == 0) {
                                if (blk + 1 < NB) ldsm4_t(f, codes + blk * 256 + lane * 16);
                                else ldsm2_t(f, codes + blk * 256 + (lane & 15) * 16);
                            }
                            constexpr uint32_t lo = 0x000f000fu, hi = 0x00f000f0u;
                            const uint32_t y = f[(blk & 1) * 2], z = f[(blk & 1) * 2 + 1];
                            mma_more(o[2 * blk], y & lo, y & hi, z & lo, z & hi, w0, w1);
                            mma_more(o[2 * blk + 1], y >> 8 & lo, y >> 8 & hi, z >> 8 & lo, z >> 8 & hi, w0, w1);
                            mma_more(o[2 * blk], 0x80088008u, 0x80808080u, 0x80088008u, 0x80808080u, w0, w1);
                            mma_more(o[2 * blk + 1], 0x80088008u, 0x80808080u, 0x80088008u, 0x80808080u, w0, w1);
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
                for (; i < issued; ++i) {
                    int never = 0;
                    mbar_wait(my_full + 8 * stg, phase, &never);
                    if (++stg == ST) {
                        stg = 0;
                        phase ^= 1;
                    }
                }
            }
#pragma unroll
            for (int h = 0; h < 2; ++h)
#pragma unroll
                for (int y = 4; y < 32; y <<= 1) sum[h] += __shfl_xor_sync(0xffffffffu, sum[h], y);
            top[0] *= factor[0];
            top[1] *= factor[1];
        }
        __syncthreads();  // the ring is free
        const bool gave_up = *abort;
        float *part = reinterpret_cast<float *>(ring);
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const int row = 2 * t + h;
            float *dst = part + (warp * kRows + row) * L::kStride;
            if (row >= rows) continue;
#pragma unroll
            for (int blk = 0; blk < NB; ++blk) {
                constexpr float lo = 0x1p24f, hi = kQ8 ? 0x1p24f : 0x1p20f;  // of rows g, of rows g + 8
                const float e[4] = {o[2 * blk][h] * lo, o[2 * blk][2 + h] * hi, o[2 * blk + 1][h] * lo, o[2 * blk + 1][2 + h] * hi};
                if constexpr (kQ8) {
                    *reinterpret_cast<float2 *>(dst + 32 * blk + 2 * g) = make_float2(e[0], e[1]);
                    *reinterpret_cast<float2 *>(dst + 32 * blk + 16 + 2 * g) = make_float2(e[2], e[3]);
                } else {
                    *reinterpret_cast<float4 *>(dst + 32 * blk + 4 * g) = make_float4(e[0], e[1], e[2], e[3]);
                }
            }
            if (g == 0) {
                ml_s[warp][row][0] = top[h];
                ml_s[warp][row][1] = sum[h];
            }
        }
        if (gave_up && tid == 0) atomicMax(&reported, int(QMM_ERR_DEVICE));
        __syncthreads();
        // the warps' rows joined: the flat form's are done, a cluster's go into the first warp's place
        const int64_t row0 = b * d.shape.hq + head0;
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
                const float4 y = *reinterpret_cast<const float4 *>(part + (w * kRows + row) * L::kStride + col);
                acc.x += f * y.x;
                acc.y += f * y.y;
                acc.z += f * y.z;
                acc.w += f * y.w;
                total += f * ml_s[w][row][1];
            }
            if (kFlat) {
                const bool none = !(total != 0.f);
                const float inv = none ? 0.f : 1.f / total;
                acc = make_float4(acc.x * inv, acc.y * inv, acc.z * inv, acc.w * inv);
                const float log2_total = none ? -INFINITY : base + log2f(total);
                const int64_t at = (int64_t(blockIdx.x) * 2 + slot) * kRows + row;
                if (whole) {
                    T *out = static_cast<T *>(d.out) + b * d.so.t + (head0 + row) * d.so.h + col;
                    *reinterpret_cast<uint2 *>(out) = make_uint2(pack2<T>(acc.x, acc.y), pack2<T>(acc.z, acc.w));
                } else {
                    *reinterpret_cast<float4 *>(a.part + at * D + col) = acc;
                }
                if (col == 0) {
                    if (!whole) a.part_lse[at] = log2_total;
                    else if (d.lse) d.lse[row0 + row] = log2_total * kLn2;
                }
            } else {
                *reinterpret_cast<float4 *>(part + row * L::kStride + col) = acc;
                if (col == 0) {
                    joined_s[row][0] = most;
                    joined_s[row][1] = total;
                }
            }
        }
        if (kFlat) {
            fence_proxy_async_smem();  // the partial rows' place is the ring again
            __syncthreads();
            if (gave_up) break;
            begin += units_of(tiles);
            if (begin >= end) break;
            first = 0;
            if (++pair == pairs) {
                pair = 0;
                do tiles = request_tiles(d, ++b);
                while (tiles == 0 && b + 1 < d.batch);
            }
            continue;
        }
        if (ranks > 1) cluster_sync();
        else __syncthreads();

        // ------------------------------------------------ the cluster's rows
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
            for (int y = 16; y > 0; y >>= 1) most = fmaxf(most, __shfl_xor_sync(0xffffffffu, most, y));
            const float base = most == -INFINITY ? 0.f : most;
            const float w = ex2(m - base);
            float total = w * l;
#pragma unroll
            for (int y = 16; y > 0; y >>= 1) total += __shfl_xor_sync(0xffffffffu, total, y);
            const bool none = !(total != 0.f);
            if (lane < ranks) weight_s[row][lane] = none ? 0.f : w / total;
            if (lane == 0 && rank == 0 && d.lse) d.lse[row0 + row] = none ? -INFINITY : (base + log2f(total)) * kLn2;
        }
        __syncthreads();
        for (int e = rank + tid * ranks; e < rows * kQuads; e += ranks * kThreads) {
            const int row = e / kQuads, col = (e % kQuads) * 4;
            float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
            const uint32_t addr = smem_u32(part + row * L::kStride + col);
#pragma unroll 4
            for (int p = 0; p < ranks; ++p) {
                const float w = weight_s[row][p];
                const float4 y = ranks == 1 ? *reinterpret_cast<const float4 *>(part + row * L::kStride + col) : peer_f32x4(addr, p);
                acc.x += w * y.x;
                acc.y += w * y.y;
                acc.z += w * y.z;
                acc.w += w * y.w;
            }
            T *out = static_cast<T *>(d.out) + b * d.so.t + (head0 + row) * d.so.h + col;
            *reinterpret_cast<uint2 *>(out) = make_uint2(pack2<T>(acc.x, acc.y), pack2<T>(acc.z, acc.w));
        }
        if (ranks > 1) cluster_sync();  // no CTA leaves while its shared memory may be read
        break;
    }
    if (kFlat && tid == 0) a.cuts[blockIdx.x] = cut_here;
}

// The flat form's requests that were cut, joined: a block for each CTA, which has left word whether such a one
// begins with it, and a warp a row.  Requests without tiles, which no CTA has seen, give zeros.
constexpr int kJoinThreads = kRows * 32;
template <typename T> __global__ void __launch_bounds__(kJoinThreads) kv_join_kernel(const __grid_constant__ Args a) {
    const KvDecodeArgs &d = a.d;
    const int tid = threadIdx.x, row = tid >> 5, lane = tid & 31, D = d.shape.d, col = lane * 4;
    for (int64_t b = blockIdx.x; b < d.batch; b += gridDim.x) {
        if (request_tiles(d, b) > 0) continue;
        for (int e = tid; e < d.shape.hq * (D / 4); e += kJoinThreads) {
            T *out = static_cast<T *>(d.out) + b * d.so.t + e / (D / 4) * d.so.h + e % (D / 4) * 4;
            *reinterpret_cast<uint2 *>(out) = make_uint2(0, 0);
        }
        if (d.lse)
            for (int h = tid; h < d.shape.hq; h += kJoinThreads) d.lse[b * d.shape.hq + h] = -INFINITY;
    }
    grid_dependency_wait();
    const int4 info = __ldcg(a.cuts + blockIdx.x);
    const int b = info.x, pair = info.y, parts = info.w;
    const int hk = pair / a.row_blocks, block = pair - hk * a.row_blocks;
    const int head = hk * a.group + block * kRows + row;
    if (parts == 0 || row >= a.group - block * kRows) return;
    // the first part is the CTA's last piece, the others are the first ones of the CTAs after it
    auto at = [&](int p) { return (int64_t(blockIdx.x + p) * 2 + (p == 0 ? info.z : 0)) * kRows + row; };
    float most = -INFINITY, sum = 0.f;
    for (int p = lane; p < parts; p += 32) most = fmaxf(most, __ldcg(a.part_lse + at(p)));
#pragma unroll
    for (int s = 16; s > 0; s >>= 1) most = fmaxf(most, __shfl_xor_sync(0xffffffffu, most, s));
    const float base = most == -INFINITY ? 0.f : most;
    for (int p = lane; p < parts; p += 32) sum += ex2(__ldcg(a.part_lse + at(p)) - base);
#pragma unroll
    for (int s = 16; s > 0; s >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, s);
    const float inv = sum != 0.f ? 1.f / sum : 0.f;
    float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
    for (int p0 = 0; p0 < parts; p0 += 16) {  // sixteen loads in flight
        float4 y[16];
        float w = p0 + lane < parts && lane < 16 ? ex2(__ldcg(a.part_lse + at(p0 + lane)) - base) * inv : 0.f;
#pragma unroll
        for (int i = 0; i < 16; ++i)
            y[i] = col < D && p0 + i < parts ? __ldcg(reinterpret_cast<const float4 *>(a.part + at(p0 + i) * D + col))
                                             : make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
        for (int i = 0; i < 16; ++i) {
            const float f = __shfl_sync(0xffffffffu, w, i);
            acc.x += f * y[i].x;
            acc.y += f * y[i].y;
            acc.z += f * y[i].z;
            acc.w += f * y[i].w;
        }
    }
    T *out = static_cast<T *>(d.out) + int64_t(b) * d.so.t + head * d.so.h + col;
    if (col < D) *reinterpret_cast<uint2 *>(out) = make_uint2(pack2<T>(acc.x, acc.y), pack2<T>(acc.z, acc.w));
    if (d.lse && lane == 0) d.lse[int64_t(b) * d.shape.hq + head] = sum != 0.f ? (base + log2f(sum)) * kLn2 : -INFINITY;
}

size_t align256(size_t x) { return (x + 255) & ~size_t(255); }

// How a call is shared out: clusters of `ranks` CTAs, or the flat form's CTAs (ranks == 0).
struct Plan {
    int ranks, ctas;
};
Plan plan(const KvDecodeArgs &d) {
    const int64_t group = d.shape.hq / d.shape.hk, pairs = d.batch * d.shape.hk * ((group + kRows - 1) / kRows);
    const int64_t tiles = (d.max_len + kTileKeys - 1) / kTileKeys, resident = kCtas * device_sm_count();
    if (d.batch <= kMaxFlatBatch && d.batch * (tiles + kPieceUnits) < (int64_t(1) << 30) && pairs * tiles >= resident * kWarps * 4)
        return {0, (int)resident};
    // a power of two, at most a CTA for every four tiles, with room to spare
    int ranks = 1;
    while (ranks < kMaxCluster && tiles >= 2 * ranks * kWarps && pairs * 2 * ranks <= resident - device_sm_count()) ranks *= 2;
    return {ranks, 0};
}

template <typename T, bool kQ8, int D> cudaError_t launch(const Args &a, Plan p, int64_t pairs, cudaStream_t st) {
    using L = Tile<kQ8, D>;
    auto kern = p.ranks ? kv_decode_kernel<T, kQ8, D, false> : kv_decode_kernel<T, kQ8, D, true>;
    cudaError_t e = ensure_smem(kern, L::kSmem);
    if (e != cudaSuccess) return e;
    if (!p.ranks) {
        kern<<<p.ctas, kThreads, L::kSmem, st>>>(a);
        e = cudaGetLastError();
        if (e != cudaSuccess) return e;
        return launch_pdl(kv_join_kernel<T>, dim3((unsigned)p.ctas), dim3(kJoinThreads), 0, st, a);
    }
    if (p.ranks > 8) {
        e = cudaFuncSetAttribute(kern, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
        if (e != cudaSuccess) return e;
    }
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3((unsigned)(pairs * p.ranks));
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = L::kSmem;
    cfg.stream = st;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = p.ranks;
    attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kern, a);
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
    const size_t ctas = plan(d).ctas, rows = ctas * 2 * kRows;
    return align256(rows * d.shape.d * 4) + align256(rows * 4) + align256(ctas * sizeof(int4));
}

cudaError_t launch_kv_decode(const KvDecodeArgs &d, qmm_float t, void *ws, cudaStream_t st) {
    const Plan p = plan(d);
    Args a{};
    a.d = d;
    a.group = d.shape.hq / d.shape.hk;
    a.row_blocks = (a.group + kRows - 1) / kRows;
    a.ctas = p.ctas;
    a.scale_log2 = d.scale * kLog2e;
    a.fault = test_fault_mode();
    if (p.ctas) {
        a.part = static_cast<float *>(ws);
        const size_t rows = size_t(p.ctas) * 2 * kRows;
        uint8_t *lse = static_cast<uint8_t *>(ws) + align256(rows * d.shape.d * 4);
        a.part_lse = reinterpret_cast<float *>(lse);
        a.cuts = reinterpret_cast<int4 *>(lse + align256(rows * 4));
    }
    const int64_t pairs = d.batch * d.shape.hk * a.row_blocks;
    if (pairs * std::max(p.ranks, 1) > 0x7fffffff) return cudaErrorInvalidConfiguration;
    if (t == QMM_F16) return d.cache.q8 ? launch_d<__half, true>(a, p, pairs, st) : launch_d<__half, false>(a, p, pairs, st);
    return d.cache.q8 ? launch_d<__nv_bfloat16, true>(a, p, pairs, st) : launch_d<__nv_bfloat16, false>(a, p, pairs, st);
}

}  // namespace qmm
