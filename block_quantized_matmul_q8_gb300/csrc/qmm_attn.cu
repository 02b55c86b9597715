// qmm_attn.cu -- attention of a decoding batch: one query token a request, over its own cache
// and, in the same pass or joined from the tensor-core phase, the prefix that all requests share.
//
//   out = sum_j p_j v_j,  p = softmax_j(scale q.k_j) over the prefix rows and the cache rows.
//
// Bound by reading the keys and values once.  A cluster of up to 16 CTAs takes one request and
// kv head (up to 16 query heads of it, the rows of one warp-level MMA): its key tiles of 64 are
// shared out among the CTAs, each streams them through a ring of TMA copies, and each of its 4
// warps keeps the running softmax of its own 16 keys of every tile, so no warp waits for another.
// The partial rows stay in shared memory and are joined through the cluster: no second launch
// and no workspace.  The weights are rounded to the inputs' type for the product with V (its operands
// have one type; the sum of the weights stays fp32): an error of the size of the output's own
// rounding.  The products run on mma.sync: with 16 rows the copies take an order of
// magnitude longer than the tensor work, and tcgen05's 128 rows would stay empty.
//
// 48 caches of up to 8192 rows, 32/8 heads of 128: 129 us, 6.35 TB/s (95% of the measured copy
// rate).  One request of 640 rows: 6.2 us, of which a tile's copy, products and join take 4 and the
// launch 2.  64 requests of up to 512 rows after a prefix of 8192: 36 us, the tensor-core phase and
// the caches after one another on most SMs, 4 to 5 us of it starts and joins.
#include <cuda.h>
#include <cuda_runtime.h>

#include <algorithm>

#include "qmm_attn.cuh"
#include "qmm_internal.h"
#include "qmm_mma.cuh"
#include "qmm_tc_ptx.cuh"

namespace qmm {

namespace {

using namespace ptx;

constexpr int kTileKeys = 64;
constexpr int kWarps = 4;              // each takes 16 keys of a tile
constexpr int kThreads = (kWarps + 1) * 32;
constexpr int kMaxRows = 16;           // query heads of one CTA
constexpr int kMaxCluster = 16;

template <int DP> struct Ring {
    // Stages hold a K tile or a V tile by turns: DP/64 blocks of 64 x 128 bytes.  64 KB of them and
    // 128 registers a thread let three CTAs share an SM, so that one's start and join overlap the
    // others' copies; heads up to 64 take 48 KB and 96 registers, and four (35 requests of 16 heads
    // on a prefix of 297: 13.5 -> 9.1 us; with 128-element heads four take 133 us where three take 129).
    static constexpr int kTile = kTileKeys * DP * 2;
    static constexpr int kStages = DP == 128 ? 4 : 6;
    static constexpr int kCtas = DP == 128 ? 3 : 4;   // of one SM
    static constexpr int kPartStride = DP + 4;        // floats between a warp's partial rows
    static constexpr size_t kBytes = size_t(kStages) * kTile + 1024;
    static constexpr int kParts = kWarps * kMaxRows * kPartStride;  // floats of the CTA's partial rows
    static_assert((kParts + kMaxRows * (kMaxCluster + kMaxSplits + 2)) * 4 <= kStages * kTile,
                  "partial rows and weights reuse the ring");
};

struct DecArgs {
    CUtensorMap k, v, pk, pv;
    DecodeArgs d;
    int group, row_blocks;   // query heads of a kv head, blocks of 16 of them
    int64_t inline_prefix;   // prefix rows that this launch reads itself
    int parts;               // partial rows of the tensor-core phase to join
    const float *part, *part_lse;
    float scale_log2;
    int fault;               // qmm_set_test_fault: 1 no copy is issued, and the waits for them are short;
                             // 2 the copies are issued, and the first wait for one gives up at once
    int *status;
};

__device__ __forceinline__ void tma_load_3d(uint32_t dst, const CUtensorMap *map, int x, int y, int z, uint32_t bar) {
    asm volatile(
        "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4}], "
        "[%5];" ::"r"(dst),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(z), "r"(bar)
        : "memory");
}
__device__ __forceinline__ void tma_load_4d(uint32_t dst, const CUtensorMap *map, int x, int y, int z, int w,
                                            uint32_t bar) {
    asm volatile(
        "cp.async.bulk.tensor.4d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4, "
        "%5}], [%6];" ::"r"(dst),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(z), "r"(w), "r"(bar)
        : "memory");
}
// Byte of 16-byte unit u of a row in a block of rows of 128 bytes, 128-byte swizzled.
__device__ __forceinline__ uint32_t swizzled(int row, int u) { return uint32_t(row * 128 + ((u ^ (row & 7)) << 4)); }

template <typename T, int DP> __global__ void __launch_bounds__(kThreads, Ring<DP>::kCtas) attn_decode_kernel(const __grid_constant__ DecArgs a) {
    using R = Ring<DP>;
    constexpr int ST = R::kStages, KS = DP / 16;
    extern __shared__ uint8_t raw[];
    __shared__ uint64_t full[ST], empty[ST];
    __shared__ int abort_s, issued_s;  // issued: copies so far
    __shared__ float ml_s[kWarps][kMaxRows][2];  // each warp's maximum and sum (log2 domain)
    __shared__ float joined_s[kMaxRows][2];      // the CTA's
    const DecodeArgs &d = a.d;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int rank = (int)cluster_rank(), ranks = (int)cluster_size();
    int64_t rest = blockIdx.x / ranks;
    const int block = int(rest % a.row_blocks);
    rest /= a.row_blocks;
    const int hk = int(rest % d.shape.hk);
    const int64_t b = rest / d.shape.hk;
    const int head0 = hk * a.group + block * kMaxRows, rows = min(a.group - block * kMaxRows, kMaxRows);
    if (blockIdx.x == 0 && tid == 0 && a.parts == 0) *a.status = QMM_OK;

    const int64_t len = d.room > 0 ? min(max(int64_t(d.lens[b]), int64_t(0)), d.room) : 0;
    const int64_t ptiles = (a.inline_prefix + kTileKeys - 1) / kTileKeys;
    const int64_t tiles = ptiles + (len + kTileKeys - 1) / kTileKeys, per = (tiles + ranks - 1) / ranks;
    const int64_t j0 = min(rank * per, tiles), j1 = min(j0 + per, tiles);
    const int n = int(j1 - j0);

    const uint32_t sm = (smem_u32(raw) + 1023u) & ~1023u;
    if (tid == 0) {
        abort_s = issued_s = 0;
        for (int i = 0; i < ST; ++i) {
            mbar_init(smem_u32(&full[i]), 1);
            mbar_init(smem_u32(&empty[i]), kWarps);
        }
        fence_mbar_init();
    }
    if (warp == kWarps && lane == 0) {
        prefetch_tmap(&a.k);
        prefetch_tmap(&a.v);
        if (ptiles > 0) {
            prefetch_tmap(&a.pk);
            prefetch_tmap(&a.pv);
        }
    }
    __syncthreads();
    volatile int *abort = &abort_s;

    if (warp == kWarps) {
        // ------------------------------------------------ copies
        bool ok = true;
        if (lane == 0) {
            for (int i = 0; i < 2 * n && ok && a.fault != 1; ++i) {
                const int stg = i % ST, kv = i & 1;
                if (i >= ST) ok = mbar_wait(smem_u32(&empty[stg]), ((i / ST) - 1) & 1, abort);
                if (!ok) break;
                const uint32_t bar = smem_u32(&full[stg]), dst = sm + stg * R::kTile;
                mbar_arrive_expect_tx(bar, R::kTile);
                const int64_t j = j0 + (i >> 1);
#pragma unroll
                for (int c = 0; c < DP / 64; ++c) {
                    const uint32_t to = dst + c * kTileKeys * 128;
                    if (j < ptiles) tma_load_3d(to, kv ? &a.pv : &a.pk, c * 64, hk, int(j * kTileKeys), bar);
                    else tma_load_4d(to, kv ? &a.v : &a.k, c * 64, hk, int((j - ptiles) * kTileKeys), int(b), bar);
                }
                issued_s = i + 1;
            }
        }
        __syncwarp();
    }

    // this warp's running softmax of rows lane/4 and lane/4 + 8
    float top[2] = {-INFINITY, -INFINITY}, sum[2] = {0.f, 0.f}, o[DP / 8][4];
#pragma unroll
    for (int c = 0; c < DP / 8; ++c) o[c][0] = o[c][1] = o[c][2] = o[c][3] = 0.f;
    if (a.fault == 2) {
        if (n > 0) *abort = 1;
    } else if (warp < kWarps && n > 0) {
        uint32_t q[KS][4];
        {
            const T *src = static_cast<const T *>(d.q) + b * d.sq.t + head0 * d.sq.h;
#pragma unroll
            for (int ks = 0; ks < KS; ++ks)
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const int row = (lane >> 2) + (e & 1) * 8, col = ks * 16 + (lane & 3) * 2 + (e >> 1) * 8;
                    q[ks][e] = row < rows && col < d.shape.d
                                   ? *reinterpret_cast<const uint32_t *>(src + row * d.sq.h + col)
                                   : 0u;
                }
        }
        for (int i = 0; i < n; ++i) {
            const int k_stg = (2 * i) % ST, v_stg = k_stg + 1, phase = ((2 * i) / ST) & 1;  // ST is even
            const uint32_t kt = sm + k_stg * R::kTile, vt = kt + R::kTile;
            if (!warp_wait(smem_u32(&full[k_stg]), phase, abort, a.fault ? 100000 : kWaitCycles)) break;
            const int64_t j = j0 + i;
            const int64_t left = j < ptiles ? a.inline_prefix - j * kTileKeys : len - (j - ptiles) * kTileKeys;
            const int valid = int(min(left, int64_t(kTileKeys))) - warp * 16;  // of this warp's keys
            uint32_t p[4];
            if (valid > 0) {
                float s[2][4] = {};
#pragma unroll
                for (int ks = 0; ks < KS; ++ks) {
                    uint32_t f[4];  // keys 0-7 and 8-15, each k 0-7 and 8-15
                    const int key = warp * 16 + (lane & 7) + ((lane >> 4) << 3), u = (ks & 3) * 2 + ((lane >> 3) & 1);
                    ldsm4(f, kt + (ks >> 2) * kTileKeys * 128 + swizzled(key, u));
                    mma16816<T>(s[0], q[ks], f[0], f[1]);
                    mma16816<T>(s[1], q[ks], f[2], f[3]);
                }
                float m[2] = {-INFINITY, -INFINITY};
#pragma unroll
                for (int t = 0; t < 2; ++t)
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        const int key = t * 8 + (lane & 3) * 2 + (e & 1);
                        s[t][e] = key < valid ? s[t][e] * a.scale_log2 : -INFINITY;
                        m[e >> 1] = fmaxf(m[e >> 1], s[t][e]);
                    }
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    m[h] = fmaxf(m[h], __shfl_xor_sync(0xffffffffu, m[h], 1));
                    m[h] = fmaxf(m[h], __shfl_xor_sync(0xffffffffu, m[h], 2));
                }
                if (__any_sync(0xffffffffu, m[0] > top[0] || m[1] > top[1])) {
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        const float now = fmaxf(top[h], m[h]);
                        const float f = top[h] == -INFINITY ? 1.f : ex2(top[h] - now);
                        top[h] = now;
                        sum[h] *= f;
#pragma unroll
                        for (int c = 0; c < DP / 8; ++c) {
                            o[c][2 * h] *= f;
                            o[c][2 * h + 1] *= f;
                        }
                    }
                }
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    const float base = top[h] == -INFINITY ? 0.f : top[h];
#pragma unroll
                    for (int t = 0; t < 2; ++t) {
                        const float x = ex2(s[t][2 * h] - base), y = ex2(s[t][2 * h + 1] - base);
                        sum[h] += x + y;
                        p[t * 2 + h] = pack2<T>(x, y);
                    }
                }
            }
            __syncwarp();
            if (lane == 0) mbar_arrive(smem_u32(&empty[k_stg]));
            if (!warp_wait(smem_u32(&full[v_stg]), phase, abort)) break;
            if (valid > 0) {
                if (valid < 16) {
                    // rows that nobody owns may hold anything: zero weights times them must be zero
                    uint8_t *v = raw + (vt - smem_u32(raw));
                    for (int c = 0; c < DP / 64; ++c)
                        for (int u = valid * 8 + lane; u < 16 * 8; u += 32)
                            reinterpret_cast<uint4 *>(v + c * kTileKeys * 128 + warp * 16 * 128)[u] = make_uint4(0, 0, 0, 0);
                    fence_proxy_async_smem();
                    __syncwarp();
                }
#pragma unroll
                for (int c = 0; c < DP / 16; ++c) {
                    uint32_t f[4];  // elements 16c..16c+7 of keys 0-7, 8-15, then 16c+8..
                    const int key = warp * 16 + (lane & 15), u = (c & 3) * 2 + (lane >> 4);
                    ldsm4_t(f, vt + (c >> 2) * kTileKeys * 128 + swizzled(key, u));
                    mma16816<T>(o[2 * c], p, f[0], f[1]);
                    mma16816<T>(o[2 * c + 1], p, f[2], f[3]);
                }
            }
            __syncwarp();
            if (lane == 0) mbar_arrive(smem_u32(&empty[v_stg]));
        }
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            sum[h] += __shfl_xor_sync(0xffffffffu, sum[h], 1);
            sum[h] += __shfl_xor_sync(0xffffffffu, sum[h], 2);
        }
    }
    __syncthreads();  // the ring is free: every copy was waited for,
    if (*abort) {     // or a wait gave up, and the copies in flight land before the ring is reused or released
        if (tid == kWarps * 32)
            for (int i = max(issued_s - ST, 0); i < issued_s; ++i) {
                int never = 0;
                mbar_wait(smem_u32(&full[i % ST]), (i / ST) & 1, &never);
            }
        __syncthreads();
    }
    float *part = reinterpret_cast<float *>(raw + (sm - smem_u32(raw)));
    // weights of the partial rows in the join: the cluster's CTAs and the tensor-core phase's splits
    auto weight_s = reinterpret_cast<float(*)[kMaxCluster + 1]>(part + R::kParts);
    auto pweight_s = reinterpret_cast<float(*)[kMaxSplits + 1]>(weight_s + kMaxRows);
    if (warp < kWarps) {
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const int row = (lane >> 2) + 8 * h;
            if (row >= rows) continue;
            float *dst = part + (warp * kMaxRows + row) * R::kPartStride + (lane & 3) * 2;
#pragma unroll
            for (int c = 0; c < DP / 8; ++c)
                *reinterpret_cast<float2 *>(dst + c * 8) = make_float2(o[c][2 * h], o[c][2 * h + 1]);
            if ((lane & 3) == 0) {
                ml_s[warp][row][0] = top[h];
                ml_s[warp][row][1] = sum[h];
            }
        }
    }
    __syncthreads();
    // the warps' rows joined into the first warp's
    const int quads = d.shape.d / 4;
    for (int e = tid; e < rows * quads; e += kThreads) {
        const int row = e / quads, col = (e - row * quads) * 4;
        float m[kWarps], most = -INFINITY;
#pragma unroll
        for (int w = 0; w < kWarps; ++w) most = fmaxf(most, m[w] = ml_s[w][row][0]);
        const float base = most == -INFINITY ? 0.f : most;
        float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
        float total = 0.f;
#pragma unroll
        for (int w = 0; w < kWarps; ++w) {
            const float f = ex2(m[w] - base);
            const float4 x = *reinterpret_cast<const float4 *>(part + (w * kMaxRows + row) * R::kPartStride + col);
            acc.x += f * x.x;
            acc.y += f * x.y;
            acc.z += f * x.z;
            acc.w += f * x.w;
            total += f * ml_s[w][row][1];
        }
        *reinterpret_cast<float4 *>(part + row * R::kPartStride + col) = acc;
        if (col == 0) {
            joined_s[row][0] = most;
            joined_s[row][1] = total;
        }
    }
    if (ranks > 1) cluster_sync();
    else __syncthreads();
    if (*abort && tid == 0) *a.status = reported = QMM_ERR_DEVICE;

    // ------------------------------------------------ the join
    if (a.parts > 0) grid_dependency_wait();
    const int64_t row0 = b * d.shape.hq + head0, all_rows = d.batch * d.shape.hq;
    for (int row = warp; row < rows; row += kWarps + 1) {
        float m = -INFINITY, l = 0.f, most;
        if (ranks == 1) {
            m = lane == 0 ? joined_s[row][0] : m;
            l = lane == 0 ? joined_s[row][1] : l;
        } else if (lane < ranks) {
            m = peer_f32(smem_u32(&joined_s[row][0]), lane);
            l = peer_f32(smem_u32(&joined_s[row][1]), lane);
        }
        most = m;
        for (int p = lane; p < a.parts; p += 32) {
            const float x = a.part_lse[p * all_rows + row0 + row];
            pweight_s[row][p] = x;
            most = fmaxf(most, x);
        }
#pragma unroll
        for (int s = 16; s > 0; s >>= 1) most = fmaxf(most, __shfl_xor_sync(0xffffffffu, most, s));
        const float base = most == -INFINITY ? 0.f : most;
        const float w = ex2(m - base);
        float total = w * l;
        for (int p = lane; p < a.parts; p += 32) total += pweight_s[row][p] = ex2(pweight_s[row][p] - base);
#pragma unroll
        for (int s = 16; s > 0; s >>= 1) total += __shfl_xor_sync(0xffffffffu, total, s);
        const bool none = !(total != 0.f);
        const float inv = none ? 0.f : 1.f / total;
        if (lane < ranks) weight_s[row][lane] = w * inv;
        for (int p = lane; p < a.parts; p += 32) pweight_s[row][p] *= inv;
        if (d.lse && lane == 0 && rank == 0) d.lse[row0 + row] = none ? -INFINITY : (base + log2f(total)) * kLn2;
    }
    __syncthreads();
    for (int e = rank + tid * ranks; e < rows * quads; e += ranks * kThreads) {
        const int row = e / quads, col = (e - row * quads) * 4;
        float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
        auto add = [&](float w, float4 x) {
            acc.x += w * x.x;
            acc.y += w * x.y;
            acc.z += w * x.z;
            acc.w += w * x.w;
        };
        const uint32_t addr = smem_u32(part + row * R::kPartStride + col);
        if (ranks == 1) {
            add(weight_s[row][0], *reinterpret_cast<const float4 *>(part + row * R::kPartStride + col));
        } else {
#pragma unroll 4
            for (int p = 0; p < ranks; ++p) add(weight_s[row][p], peer_f32x4(addr, p));
        }
        const float *src = a.part + (row0 + row) * d.shape.d + col;
        const int64_t step = all_rows * d.shape.d;
        for (int p0 = 0; p0 < a.parts; p0 += 8) {  // eight loads in flight: the join waits for nothing else
            float4 x[8];
#pragma unroll
            for (int i = 0; i < 8; ++i)
                x[i] = __ldcg(reinterpret_cast<const float4 *>(src + min(p0 + i, a.parts - 1) * step));
#pragma unroll
            for (int i = 0; i < 8; ++i)
                if (p0 + i < a.parts) add(pweight_s[row][p0 + i], x[i]);
        }
        T *out = static_cast<T *>(d.out) + b * d.so.t + (head0 + row) * d.so.h + col;
        *reinterpret_cast<uint2 *>(out) = make_uint2(pack2<T>(acc.x, acc.y), pack2<T>(acc.z, acc.w));
    }
    if (ranks > 1) cluster_sync();  // no CTA leaves while its shared memory may be read
}

size_t align256(size_t x) { return (x + 255) & ~size_t(255); }

// Whether the prefix goes through the tensor-core phase.  Read inline, every request reads it
// again from L2; read once for all, it costs a second launch and the join of partial rows.  Even
// where the rereading comes to about 70 MB (32/8 heads of 128, prefix and requests: 1000 x 8, 33 MB,
// 9.5 us inline and 11.7 on the tensor cores; 1000 x 16, 66 MB, 12.8 and 12.0; 1000 x 32, 131 MB,
// 18.3 and 12.7; 8192 x 64, 190 and 35.  32/32 heads of 64: 1000 x 8, 66 MB, 15.0 and 13.5; 1000 x 16
// 18.9 and 14.2.  32/2 of 128: 1000 x 40, 41 MB, 16.7 and 17.6; 1000 x 80 23.3 and 18.2).  Heads beyond
// 16 of a kv head, which read again as blocks of their own, are not counted: 64/2 heads of 128 are
// even at 20 MB by this count (1000 x 20, 16.6 and 17.6; 1000 x 40 23.3 and 18.2).
bool prefix_on_tensor_cores(const DecodeArgs &d) {
    return 4.0 * double(d.batch) * double(d.shape.hk) * double(d.prefix) * double(d.shape.d) > 80e6;
}

// CTAs of one request and kv head (a power of two, at most one for each key tile): as many as
// leave every CTA resident at once with room to spare (one an SM fewer than fit: a grid of clusters
// that nearly fills the SMs runs its last clusters on their own; 112 pairs of 19 tiles with three
// CTAs an SM: 9.8 us with 2 CTAs each, 13.3 with 4), or, for long caches, parts of at least 32 tiles, which level out ragged
// lengths (48 x 8 pairs of up to 128 tiles: 140 us with 1, 129 with 4).
int cluster_ctas(const DecodeArgs &d, int64_t inline_prefix, int64_t pairs) {
    const int64_t tiles = (inline_prefix + kTileKeys - 1) / kTileKeys + (d.room + kTileKeys - 1) / kTileKeys;
    const int64_t room = int64_t(d.shape.d <= 64 ? Ring<64>::kCtas - 1 : Ring<128>::kCtas - 1) * device_sm_count();
    int c = 1;
    while (c < kMaxCluster && tiles >= 2 * c && (pairs * 2 * c <= room || tiles >= 64 * c)) c *= 2;
    return c;
}

template <typename T, int DP> cudaError_t launch_dp(const DecArgs &a, int64_t pairs, int ctas, cudaStream_t st) {
    auto kern = attn_decode_kernel<T, DP>;
    cudaError_t e = ensure_smem(kern, Ring<DP>::kBytes);
    if (e != cudaSuccess) return e;
    if (ctas > 8) {
        e = cudaFuncSetAttribute(kern, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
        if (e != cudaSuccess) return e;
    }
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3((unsigned)(pairs * ctas));
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = Ring<DP>::kBytes;
    cfg.stream = st;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = ctas;
    attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
    // after the tensor-core phase: start on SMs that it leaves free, and wait for it in the join
    attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[1].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = a.parts > 0 ? 2 : 1;
    return cudaLaunchKernelEx(&cfg, kern, a);
}

}  // namespace

cudaError_t attn_decode_take_error(int *code, cudaStream_t st) { return take_error(code, st); }

size_t attn_decode_workspace_bytes(const DecodeArgs &d) {
    if (!prefix_on_tensor_cores(d)) return 256;
    const size_t splits = attn_prefix_splits(d), rows = size_t(d.batch) * d.shape.hq;
    return 256 + align256(splits * rows * d.shape.d * 4) + align256(splits * rows * 4);
}

cudaError_t launch_attn_decode(const DecodeArgs &d, qmm_float t, void *ws, cudaStream_t st) {
    DecArgs a{};
    a.d = d;
    a.group = d.shape.hq / d.shape.hk;
    a.row_blocks = (a.group + kMaxRows - 1) / kMaxRows;
    a.scale_log2 = d.scale * kLog2e;
    a.status = static_cast<int *>(ws);
    a.fault = test_fault_mode();
    // maps that no tile uses describe q
    const bool cache = d.room > 0, pre = d.prefix > 0;
    if (!attn_make_map(&a.k, t, cache ? d.k : d.q, d.shape.d, cache ? d.shape.hk : 1, cache ? d.room : 1, d.sk, 1,
                       kTileKeys, cache ? d.batch : 1, d.k_batch) ||
        !attn_make_map(&a.v, t, cache ? d.v : d.q, d.shape.d, cache ? d.shape.hk : 1, cache ? d.room : 1, d.sv, 1,
                       kTileKeys, cache ? d.batch : 1, d.v_batch))
        return cudaErrorInvalidValue;
    if (prefix_on_tensor_cores(d)) {
        a.parts = attn_prefix_splits(d);
        const size_t rows = size_t(d.batch) * d.shape.hq;
        float *part = reinterpret_cast<float *>(static_cast<uint8_t *>(ws) + 256);
        float *lse = reinterpret_cast<float *>(static_cast<uint8_t *>(ws) + 256 +
                                               align256(size_t(a.parts) * rows * d.shape.d * 4));
        a.part = part;
        a.part_lse = lse;
        const cudaError_t e = launch_attn_prefix(d, t, a.parts, part, lse, ws, st);
        if (e != cudaSuccess) return e;
    } else if (pre) {
        a.inline_prefix = d.prefix;
        if (!attn_make_map(&a.pk, t, d.pk, d.shape.d, d.shape.hk, d.prefix, d.spk, 1, kTileKeys) ||
            !attn_make_map(&a.pv, t, d.pv, d.shape.d, d.shape.hk, d.prefix, d.spv, 1, kTileKeys))
            return cudaErrorInvalidValue;
    }
    const int64_t pairs = d.batch * d.shape.hk * a.row_blocks;
    const int ctas = cluster_ctas(d, a.inline_prefix, pairs);
    if (pairs * ctas > 0x7fffffff) return cudaErrorInvalidConfiguration;
    if (t == QMM_F16) return d.shape.d <= 64 ? launch_dp<__half, 64>(a, pairs, ctas, st) : launch_dp<__half, 128>(a, pairs, ctas, st);
    return d.shape.d <= 64 ? launch_dp<__nv_bfloat16, 64>(a, pairs, ctas, st)
                           : launch_dp<__nv_bfloat16, 128>(a, pairs, ctas, st);
}

}  // namespace qmm
