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
//   - values: the block's scale multiplies the weights, p d_jb rounded to fp16 (11 bits). The weights are p 2^15 until
//     a value scale of 2 or more comes, then p 2^(15 - E) for scales from 2^E on: the products stay within fp16, and what
//     they lose below its normal range is 2^-40 (times a code) or, where scales are large, 2^-40 of the largest of them.
//     Codes enter as subnormals too, and a second MMA adds -bias times the same weights
//     to the same fp32 sums, at once, so that the sums stay as small as the output.
//   - keys are the MMA's 16 rows and query heads its 8 columns, so that no row is empty; the weights reach the
//     second product's layout by movmatrix.  Codes come by ldmatrix with neighbouring codes in one 16-bit unit,
//     transposed for V, so that a nibble's mask gives the pairs of keys or elements that the MMA wants.
// A warp takes tiles of 32 keys (64 of small heads) on its own: a private ring of bulk copies (a record of 16 tokens is
// contiguous), its running softmax, no barrier with other warps until the join.
//
// Three ways to share the work out.  Many short requests: a warp for each request and kv head, no join.  Calls that fit
// the SMs at once: a cluster of up to 16 CTAs takes one request
// and kv head and joins through distributed shared memory, one launch.  Larger ones: the tiles of all
// requests lie in one row that resident CTAs cut into equal parts (each scans the lengths on the device), and a second
// launch joins the requests that were cut.  mma.sync: 8 query heads would leave tcgen05's 128 rows empty.
//
// 128 caches of up to 8192 tokens, 32/8 heads of 128 in 4 bits: 114 us, 5.3 TB/s (78% of the measured copy rate); 48 of
// them 49 us; one of 131071 (40/8 heads, fp16) 40 us; one of 640 7.5 us.  About 15 us of a large call are launch, first
// tiles and join; each further 200000 tokens take 36 us, 6.4 TB/s (94%), and in 8 bits 400000 tokens 141 us in all (91%).
// Value scales of 2 and more, where every tile looks for the largest, cost 7 to 10%.  More than 8 query heads of a kv head
// are blocks of 8 that each copy and unpack the records again: 131071 tokens of 2 kv heads of 128 take 20.8 us with 16
// query heads, 24.0 with 32, 34.4 with 64 (floor 5.6), of one kv head with 128 query heads 57.4 (floor 2.8).
#include <cuda.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <atomic>

#include "qmm_attn.cuh"
#include "qmm_internal.h"
#include "qmm_kv.h"
#include "qmm_mma.cuh"
#include "qmm_tc_ptx.cuh"

namespace qmm {

namespace {

using namespace ptx;

constexpr int kWarps = 4;
constexpr int kThreads = kWarps * 32;
constexpr int kRows = 8;         // query heads of one CTA: the MMA's N side
constexpr int kMaxCluster = 16;
constexpr int kMaxFlatBatch = 1024, kMaxParts = 1024;
constexpr int kMaxCtas = 4;      // of one SM
constexpr int kPieceUnits = 12;  // what a piece costs beside its tiles, in tiles (128 caches of up to 8192: 114.9 us
                                 // with 8, 111.8 with 12; 256 of up to 2000: 71.9 and 69.1; 48 of 8192 even)
constexpr int kMinUnits = 4;     // units of a CTA at least, a tile for each warp (with max_len 131072, one request of 100
                                 // tokens: 9.0 us with 1, 6.2 with 4, 8.9 with 13; of 640 9.4, 8.9 and 11.2; of 4000
                                 // 10.7, 10.5 and 11.7; 4 of 1000 among 64 places of up to 8192 11.1, 12.0 and 13.1)
template <bool kQ8, int D> struct Tile {
    static constexpr int kSide = kv_side_bytes(kQ8, D), kScales = kv_scales_at(kQ8, D);
    static constexpr int kRec = kv_record_bytes(kQ8, D);
    // Records of a tile: what a tile costs beside its records is spread over 2.3 KB or more
    static constexpr int kRecs = 2 * kRec < 2400 ? 4 : 2, kKeys = kRecs * kKvGroup, kBytes = kRecs * kRec;
    static constexpr int kWindow = 32 / kRecs;  // tiles whose records' places the 32 lanes hold
    // CTAs of an SM: as many as two stages of the ring leave room for, at most four: 16 warps of 128 registers (with
    // five CTAs of 96 registers 128 caches took 122.4 us instead of 115.2, with three 119.3)
    static constexpr int kCtas = std::min(kMaxCtas, 224 * 1024 / (2 * kWarps * kBytes + 4096));
    static constexpr int kStages = std::min(6, (224 * 1024 / kCtas - 4096) / (kWarps * kBytes));
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
    int4 *cuts;             // what to join: the first part's CTA, its piece, the number of parts, the request's place.  An
                            // entry for each request and 8 heads, or, where those are more, for each CTA (the last that begins in it)
    int by_pair;
    int fault;              // as in qmm_attn.cu
};

// A CTA's next piece of the flat form: some tiles of one request and kv head.
struct Piece {
    int64_t b, begin, end, total;  // the request, its first unit, the CTA's last, all units
    int pair, tiles, first;        // its heads, all its tiles, the first of this CTA
    int slot, whole;               // 0 for the CTA's first piece, 1 for a later one; whether it is all tiles
};

__device__ __forceinline__ int request_len(const KvDecodeArgs &d, int64_t b) {
    return (int)min(max(int64_t(d.lens[b]), int64_t(0)), d.max_len);
}
// The flat form's row has kPieceUnits units and one for each tile for every request and kv head, so that
// a CTA of many short pieces gets fewer tiles.  CTA c of those that take part takes the units [total c / ctas,
// total (c + 1) / ctas) of it.  The grid is made for requests of max_len; where the lengths turn out to hold fewer than kMinUnits
// units a CTA, fewer CTAs take part: none is without a unit, so every part that the join counts has been written.
__device__ __forceinline__ int taking_part(int64_t total, int ctas) {
    return (int)min(int64_t(ctas), max(total / kMinUnits, int64_t(1)));
}
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
__device__ __forceinline__ uint32_t lds32(uint32_t addr) {
    uint32_t v;
    asm volatile("ld.shared.u32 %0, [%1];" : "=r"(v) : "r"(addr) : "memory");
    return v;
}
__device__ __forceinline__ float2 halves(uint32_t x) { return __half22float2(*reinterpret_cast<const __half2 *>(&x)); }
__device__ __forceinline__ uint32_t mul2(uint32_t x, uint32_t y) {
    return h2bits(__hmul2(*reinterpret_cast<const __half2 *>(&x), *reinterpret_cast<const __half2 *>(&y)));
}
__device__ __forceinline__ uint32_t fma2(uint32_t x, uint32_t y, uint32_t z) {
    return h2bits(__hfma2(*reinterpret_cast<const __half2 *>(&x), *reinterpret_cast<const __half2 *>(&y),
                          *reinterpret_cast<const __half2 *>(&z)));
}
// Two floats at a time
__device__ __forceinline__ float2 add_f32x2(float2 a, float2 b) {
    float2 y;
    asm("{.reg .b64 x, y;\nmov.b64 x, {%2, %3};\nmov.b64 y, {%4, %5};\nadd.rn.f32x2 x, x, y;\nmov.b64 {%0, %1}, x;}"
        : "=f"(y.x), "=f"(y.y)
        : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
    return y;
}
__device__ __forceinline__ float2 fma_f32x2(float2 a, float2 b, float2 c) {
    float2 y;
    asm("{.reg .b64 x, y, z;\nmov.b64 x, {%2, %3};\nmov.b64 y, {%4, %5};\nmov.b64 z, {%6, %7};\n"
        "fma.rn.f32x2 x, x, y, z;\nmov.b64 {%0, %1}, x;}"
        : "=f"(y.x), "=f"(y.y)
        : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y), "f"(c.x), "f"(c.y));
    return y;
}
// Two 16-bit values of a word
template <typename T> __device__ __forceinline__ float2 values(uint32_t x) {
    if constexpr (std::is_same<T, __half>::value) return halves(x);
    else return make_float2(__uint_as_float(x << 16), __uint_as_float(x & 0xffff0000u));
}
__device__ __forceinline__ uint32_t transpose8x8(uint32_t x) {
    uint32_t y;
    asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
    return y;
}
// c = a b + first
__device__ __forceinline__ void mma_first(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                          uint32_t b1, float4 first) {
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%10,%11,%12,%13};"
        : "=f"(c[0]), "=f"(c[1]), "=f"(c[2]), "=f"(c[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(first.x), "f"(first.y), "f"(first.z), "f"(first.w));
}
__device__ __forceinline__ void mma_more(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0, uint32_t b1) {
    const uint32_t a[4] = {a0, a1, a2, a3};
    mma16816<__half>(c, a, b0, b1);
}

enum Form { kCluster, kFlatRow, kWarpEach };  // how the work is shared out

template <typename T, bool kQ8, int D, Form kForm> __global__ void __launch_bounds__(kThreads, Tile<kQ8, D>::kCtas) kv_decode_kernel(const __grid_constant__ Args a) {
    using L = Tile<kQ8, D>;
    constexpr bool kFlat = kForm == kFlatRow, kAlone = kForm == kWarpEach;  // kAlone: a warp has its own request and kv head
    constexpr int ST = L::kStages, NB = D / 32, kQuads = D / 4, R = L::kRecs;
    extern __shared__ __align__(128) uint8_t ring[];
    __shared__ uint64_t full[kWarps * ST];
    __shared__ int abort_s;
    __shared__ Piece piece_s;                        // kept here while the tiles take the registers
    __shared__ float ml_s[kWarps][kRows][2];         // each warp's maximum and sum (log2 domain)
    __shared__ float joined_s[kRows][2];             // the CTA's
    __shared__ float weight_s[kRows][kMaxCluster];
    __shared__ uint2 qb_s[kAlone ? kWarps : 1][NB][2][32];  // B fragments of two MMAs a block: k 2t, 2t + 1 and 2t + 8, 2t + 9 of head g
    __shared__ float4 qc_s[kAlone ? kWarps : 1][NB][4];     // the accumulators' first values, of heads 2t, 2t + 1
    __shared__ float beyond_s[kWarps][kRows];               // what a head's factor from sums to scores has beyond 2^127
    const KvDecodeArgs &d = a.d;
    auto request_tiles = [&](int64_t b) { return (request_len(d, b) + L::kKeys - 1) / L::kKeys; };
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, g = lane >> 2, t = lane & 3;
    const int rank = kForm == kCluster ? (int)cluster_rank() : 0, ranks = kForm == kCluster ? (int)cluster_size() : 1;
    const int mine = kAlone ? warp : 0;              // of qb_s and qc_s
    const int pairs = d.shape.hk * a.row_blocks;     // of a request

    const uint32_t my_ring = smem_u32(ring) + warp * ST * L::kBytes, my_full = smem_u32(full) + warp * ST * 8;
    if (tid == 0) abort_s = 0;
    if (lane == 0) {
        for (int i = 0; i < ST; ++i) mbar_init(my_full + 8 * i, R);
        fence_mbar_init();
    }
    grid_dependency_wait();    // the kernel before may have written anything that is read from here on
    grid_launch_dependents();  // what follows (the join, the next call) may take the places that become free, and waits there
    Piece piece{};
    if (kFlat) {
        // each warp for itself: the sum of all units, then the request that holds the CTA's first
        int sum = 0;
        for (int i = lane; i < d.batch; i += 32) sum += units_of(request_tiles(i));
#pragma unroll
        for (int s = 16; s > 0; s >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, s);
        const int64_t total = int64_t(sum) * pairs;
        const int ctas = taking_part(total, a.ctas);
        if (!a.by_pair && tid == 0) a.cuts[blockIdx.x] = make_int4(0, 0, 0, 0);
        if (int(blockIdx.x) >= ctas) return;
        const int64_t x = cut(total, blockIdx.x, ctas);
        int before = 0, units = kPieceUnits;  // of one head of the requests before the piece's, of that
        for (int base = 0; base < d.batch; base += 32) {
            const int own = base + lane < d.batch ? units_of(request_tiles(base + lane)) : 0;
            int upto = own;
#pragma unroll
            for (int s = 1; s < 32; s <<= 1) {
                const int u = __shfl_up_sync(0xffffffffu, upto, s);
                if (lane >= s) upto += u;
            }
            const uint32_t after = __ballot_sync(0xffffffffu, int64_t(before + upto) * pairs > x);
            if (after) {
                const int at = __ffs(after) - 1;
                piece.b = base + at;
                units = __shfl_sync(0xffffffffu, own, at);
                before += __shfl_sync(0xffffffffu, upto, at) - units;
                break;
            }
            before += __shfl_sync(0xffffffffu, upto, 31);
        }
        piece.total = total;
        piece.end = cut(total, blockIdx.x + 1, ctas);
        piece.tiles = units - kPieceUnits;
        piece.begin = int64_t(before) * pairs;
        piece.pair = int((x - piece.begin) / units);
        piece.begin += int64_t(piece.pair) * units;
        piece.first = max(int(x - piece.begin) - kPieceUnits, 0);
    } else {
        const int64_t at = kAlone ? int64_t(blockIdx.x) * kWarps + warp : blockIdx.x / ranks;
        if (!kAlone || at < d.batch * pairs) {
            piece.b = at / pairs;
            piece.pair = int(at - piece.b * pairs);
            piece.tiles = request_tiles(piece.b);
        } else {
            piece.b = -1;
        }
    }
    __syncthreads();
    if (kAlone && piece.b < 0) return;
    volatile int *abort = &abort_s;
    int stg = 0, phase = 0;  // the warp's next stage
    bool dead = false;

    while (true) {
        int j0, n;  // tiles of the warp
        if (kFlat) {
            const int count = int(min(piece.end - piece.begin - kPieceUnits, int64_t(piece.tiles))) - piece.first;
            if (count <= 0) break;
            piece.whole = count == piece.tiles;
            if (tid == 0) {
                piece_s = piece;
                if (piece.first == 0 && (!piece.whole || a.by_pair)) {
                    const int64_t place = piece.b * pairs + piece.pair;
                    const int last = cta_of(piece.total, piece.begin + units_of(piece.tiles) - 1, taking_part(piece.total, a.ctas));
                    a.cuts[a.by_pair ? place : blockIdx.x] =
                        make_int4(int(blockIdx.x), piece.slot, piece.whole ? 0 : last - int(blockIdx.x) + 1, int(place));
                }
            }
            j0 = piece.first + int(int64_t(count) * warp / kWarps);
            n = piece.first + int(int64_t(count) * (warp + 1) / kWarps) - j0;
        } else if (kAlone) {
            j0 = 0;
            n = piece.tiles;
        } else {
            if (tid == 0) piece_s = piece;
            const int64_t workers = ranks * kWarps, me = rank * kWarps + warp;
            j0 = int(piece.tiles * me / workers);
            n = int(piece.tiles * (me + 1) / workers) - j0;
        }
        if (dead) n = 0;  // after a wait that gave up the other pieces are empty: the join finds its entries
        const int64_t b = piece.b;
        const int hk = piece.pair / a.row_blocks, block = piece.pair - hk * a.row_blocks;
        const int head0 = hk * a.group + block * kRows, rows = min(a.group - block * kRows, kRows);
        const int len = request_len(d, b);

        // the queries are on their way while the pages are looked up
        uint2 raw[NB][2];
        {
            const T *const src = static_cast<const T *>(d.q) + b * d.sq.t + (head0 + g) * d.sq.h;
#pragma unroll
            for (int i = 0; i < NB; ++i) {
                raw[i][0] = raw[i][1] = make_uint2(0, 0);
                if (g >= rows) continue;
                if (kQ8) {
                    raw[i][0] = *reinterpret_cast<const uint2 *>(src + 32 * i + 4 * t);
                    raw[i][1] = *reinterpret_cast<const uint2 *>(src + 32 * i + 16 + 4 * t);
                } else {
                    const uint4 u = *reinterpret_cast<const uint4 *>(src + 32 * i + 8 * t);
                    raw[i][0] = make_uint2(u.x, u.y);
                    raw[i][1] = make_uint2(u.z, u.w);
                }
            }
        }

        // where the records R (j0 + i).. of the next 32 lie, one a lane, and the pages of the 32 after them: -1 for
        // a page that does not exist, -2 past the last
        const int log2g = d.cache.page_log2 - 4, records = min((len + 15) / 16, R * (j0 + n));
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
        const uint8_t *src = source(R * j0 + lane, page_of(R * j0 + lane));
        int next = page_of(R * j0 + 32 + lane);
        uint32_t missing_ahead = __ballot_sync(0xffffffffu, !src && R * j0 + lane < records), missing = 0;  // records that are not copied
        auto issue = [&](int i, int to) {  // the lanes of its records copy a tile
            if ((i & (L::kWindow - 1)) == 0 && i > 0) {
                const int record = R * (j0 + i) + lane;
                src = source(record, next);
                next = page_of(record + 32);
                missing_ahead = __ballot_sync(0xffffffffu, !src && record < records);
            }
            if (lane / R == (i & (L::kWindow - 1))) {
                const uint32_t bar = my_full + 8 * to;
                if (src) {
                    mbar_arrive_expect_tx(bar, L::kRec);
                    bulk_g2s(my_ring + to * L::kBytes + (lane & (R - 1)) * L::kRec, src, L::kRec, bar);
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
        float up_w = 15.f;               // weights are p 2^up_w, and so are their sum and o
        float out_unit = 0x1p24f;        // of o's columns that hold codes as they are
#pragma unroll
        for (int i = 0; i < D / 16; ++i) o[i][0] = o[i][1] = o[i][2] = o[i][3] = 0.f;
        float factor[2];  // of heads 2t, 2t + 1
        {
            float v[NB][8], most = 0.f;
#pragma unroll
            for (int i = 0; i < NB; ++i) {
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const float2 y = values<T>(j & 1 ? raw[i][j >> 1].y : raw[i][j >> 1].x);
                    v[i][2 * j] = y.x;
                    v[i][2 * j + 1] = y.y;
                    most = fmaxf(most, fmaxf(fabsf(y.x), fabsf(y.y)));
                }
            }
            most = fmaxf(most, __shfl_xor_sync(0xffffffffu, most, 1));
            most = fmaxf(most, __shfl_xor_sync(0xffffffffu, most, 2));
            // times 2^up: the largest element into [2^13, 2^14), -115 at least; a negative scale turns the queries
            const int up = most > 0.f ? min(100, 140 - int(__float_as_uint(most) >> 23)) : 0;
            const float times = copysignf(__int_as_float((127 + up) << 23), a.scale_log2);
            // Not zero, so that a score of minus infinity stays one; 2^127 at most, so that a difference of zero stays one: any
            // other is then far beyond what leaves a weight, and only the scores' maximum takes what lies beyond
            const float f0 = fabsf(a.scale_log2) * __int_as_float((127 + 12 - up / 2) << 23), f1 = __int_as_float((127 + 12 - (up - up / 2)) << 23);
            const float f = fminf(fmaxf(f0 * f1, 1e-37f), 0x1p127f);
            beyond_s[warp][g] = fmaxf(f0 * (f1 * 0x1p-127f), 1.f);
            factor[0] = __shfl_sync(0xffffffffu, f, 8 * t);
            factor[1] = __shfl_sync(0xffffffffu, f, 8 * t + 4);
#pragma unroll
            for (int i = 0; i < NB; ++i) {
                if (!kAlone && i != warp) continue;  // a block a warp
                float total = 0.f;
#pragma unroll
                for (int m = 0; m < 2; ++m) {
                    // nibbles 0, 4 (and 2, 6) as they are, 1, 5 (and 3, 7) 16 times as large; bytes in order
                    const float e[4] = {v[i][kQ8 ? 4 * m : 2 * m] * times, v[i][kQ8 ? 4 * m + 1 : 2 * m + 4] * times,
                                        v[i][kQ8 ? 4 * m + 2 : 2 * m + 1] * (kQ8 ? times : times * 0.0625f),
                                        v[i][kQ8 ? 4 * m + 3 : 2 * m + 5] * (kQ8 ? times : times * 0.0625f)};
                    const uint2 q = make_uint2(pack2<__half>(e[0], e[1]), pack2<__half>(e[2], e[3]));
                    qb_s[mine][i][m][lane] = q;
                    const float2 y = halves(q.x), z = halves(q.y);
                    total += y.x + y.y + (kQ8 ? 1.f : 16.f) * (z.x + z.y);
                }
                total += __shfl_xor_sync(0xffffffffu, total, 1);
                total += __shfl_xor_sync(0xffffffffu, total, 2);
                total *= (kQ8 ? -128.f : -8.f) * 0x1p-24f;
                const float c0 = __shfl_sync(0xffffffffu, total, 8 * t), c1 = __shfl_sync(0xffffffffu, total, 8 * t + 4);
                if (g == 0) qc_s[mine][i][t] = make_float4(c0, c1, c0, c1);
            }
        }
        if (kAlone) __syncwarp();
        else __syncthreads();
        if (n > 0) {
            const uint32_t odd = (g & 1) ? 0x7632u : 0x5410u;  // halves of keys g and g + 8 out of four scales
            // -bias as an A operand, of rows g, g + 8, g, g + 8
            constexpr uint32_t kBias[4] = {kQ8 ? 0x80808080u : 0x80088008u, 0x80808080u, kQ8 ? 0x80808080u : 0x80088008u, 0x80808080u};
            const int plain = min(n, len / L::kKeys - j0);  // tiles without keys past the end
            bool ok = a.fault != 2;
            int i = 0;
            for (; i < n && ok; ++i) {
                ok = warp_wait(my_full + 8 * stg, phase, abort, a.fault ? 100000 : kWaitCycles);
                if (!ok) break;
                const uint32_t tile = my_ring + stg * L::kBytes;
                if ((i & (L::kWindow - 1)) == 0) missing = missing_ahead;
                const bool care = i >= plain || missing;
                uint64_t seen = ~uint64_t(0);
                if (care) {
                    // keys that nobody sees may hold anything: their value scales become zero, their scores minus infinity
                    const int valid = len - (j0 + i) * L::kKeys;
                    if (valid < L::kKeys) seen = (uint64_t(1) << valid) - 1;
#pragma unroll
                    for (int r = 0; r < R; ++r)
                        if (missing >> (R * (i & (L::kWindow - 1)) + r) & 1u) seen &= ~(uint64_t(0xffff) << (16 * r));
                    for (int e = lane; e < R * NB * 16; e += 32) {
                        const int rec = e / (NB * 16), at = e % (NB * 16), place = at & 15;
                        const int token = 2 * (place >> 2) + (place & 1) + 8 * ((place >> 1) & 1);
                        if (!(seen >> (16 * rec + token) & 1u))
                            *reinterpret_cast<uint16_t *>(ring + (tile - smem_u32(ring)) + rec * L::kRec + L::kSide + L::kScales + at * 2) = 0;
                    }
                    fence_proxy_async_smem();
                    __syncwarp();
                }
                // scores of keys g (first two) and g + 8 of the records, heads 2 t and 2 t + 1
                float s[R][4];
                uint32_t f[R][4];  // words of keys 0-7 and 8-15, of two units
#pragma unroll
                for (int blk = 0; blk < NB; ++blk) {
                    const uint2 q0 = qb_s[mine][blk][0][lane], q1 = qb_s[mine][blk][1][lane];
                    const float4 qc = qc_s[mine][blk][t];
#pragma unroll
                    for (int r = 0; r < R; ++r) {
                        const uint32_t codes = tile + r * L::kRec;
                        float acc[4];
                        if constexpr (kQ8) {
                            ldsm4(f[r], codes + blk * 512 + lane * 16);
                            const uint32_t(&w)[4] = f[r];
                            mma_first(acc, __byte_perm(w[0], 0, 0x4140), __byte_perm(w[1], 0, 0x4140), __byte_perm(w[0], 0, 0x4342),
                                      __byte_perm(w[1], 0, 0x4342), q0.x, q0.y, qc);
                            mma_more(acc, __byte_perm(w[2], 0, 0x4140), __byte_perm(w[3], 0, 0x4140), __byte_perm(w[2], 0, 0x4342),
                                     __byte_perm(w[3], 0, 0x4342), q1.x, q1.y);
                        } else {
                            if ((blk & 1) == 0) {
                                if (blk + 1 < NB) ldsm4(f[r], codes + blk * 256 + lane * 16);
                                else ldsm2(f[r], codes + blk * 256 + (lane & 15) * 16);
                            }
                            constexpr uint32_t lo = 0x000f000fu, hi = 0x00f000f0u;
                            const uint32_t y = f[r][(blk & 1) * 2], z = f[r][(blk & 1) * 2 + 1];
                            mma_first(acc, y & lo, z & lo, y & hi, z & hi, q0.x, q0.y, qc);
                            mma_more(acc, y >> 8 & lo, z >> 8 & lo, y >> 8 & hi, z >> 8 & hi, q1.x, q1.y);
                        }
                        const uint2 sc = lds64(codes + L::kScales + blk * 32 + (g >> 1) * 8);
                        const float2 ks = halves(__byte_perm(sc.x, sc.y, odd));
#pragma unroll
                        for (int e = 0; e < 4; ++e) {
                            const float y = e < 2 ? ks.x : ks.y;
                            s[r][e] = blk == 0 ? y * acc[e] : s[r][e] + y * acc[e];
                        }
                    }
                }
                if (care) {
#pragma unroll
                    for (int r = 0; r < R; ++r)
#pragma unroll
                        for (int e = 0; e < 4; ++e)
                            if (!(seen >> (16 * r + g + 8 * (e >> 1)) & 1u)) s[r][e] = -INFINITY;
                }
                float m[2];
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    m[h] = fmaxf(s[0][h], s[0][2 + h]);
#pragma unroll
                    for (int r = 1; r < R; ++r) m[h] = fmaxf(m[h], fmaxf(s[r][h], s[r][2 + h]));
                }
                // the tile's value scales, two or four a lane: is one of them 2 or more?
                constexpr int kScaleWords = R * NB * 8, kPerLane = (kScaleWords + 31) / 32;
                uint2 vs = make_uint2(0, 0);
                if (lane * kPerLane < kScaleWords) {
                    const int rec = lane * kPerLane / (NB * 8), at = lane * kPerLane % (NB * 8);
                    const uint32_t from = tile + rec * L::kRec + L::kSide + L::kScales + at * 4;
                    if constexpr (kPerLane == 2) vs = lds64(from);
                    else vs.x = lds32(from);
                }
                const bool large = ((vs.x | vs.y) & 0x40004000u) != 0;
                if (__any_sync(0xffffffffu, large || m[0] > top[0] || m[1] > top[1])) {
                    const float before = up_w;
                    if (__any_sync(0xffffffffu, large)) {  // fp16 bits of the largest; their exponent is 15 for 1
                        const uint32_t most = max(max(vs.x & 0x7fffu, vs.x >> 16 & 0x7fffu), max(vs.y & 0x7fffu, vs.y >> 16 & 0x7fffu));
                        up_w = fminf(up_w, 30.f - float(__reduce_max_sync(0xffffffffu, most) >> 10));
                    }
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
#pragma unroll
                        for (int y = 4; y < 32; y <<= 1) m[h] = fmaxf(m[h], __shfl_xor_sync(0xffffffffu, m[h], y));
                        const float now = fmaxf(top[h], m[h]);
                        const float f = top[h] == -INFINITY ? 1.f : ex2(fmaf(top[h] - now, factor[h], up_w - before));
                        top[h] = now;
                        sum[h] *= f;
#pragma unroll
                        for (int c = 0; c < D / 16; ++c) {
                            o[c][h] *= f;
                            o[c][2 + h] *= f;
                        }
                    }
                }
                const float2 base = make_float2(top[0] == -INFINITY ? 0.f : -top[0], top[1] == -INFINITY ? 0.f : -top[1]);
#pragma unroll
                for (int r = 0; r < R; ++r)
#pragma unroll
                    for (int e = 0; e < 4; e += 2) {
                        // the difference first: the largest weight is 2^up_w exactly, and no other is larger
                        const float2 x = fma_f32x2(add_f32x2(make_float2(s[r][e], s[r][e + 1]), base), make_float2(factor[0], factor[1]),
                                                   make_float2(up_w, up_w));
                        s[r][e] = ex2(x.x);
                        s[r][e + 1] = ex2(x.y);
                    }
#pragma unroll
                for (int r = 0; r < R; ++r)
#pragma unroll
                    for (int h = 0; h < 2; ++h) sum[h] += s[r][h] + s[r][2 + h];
#pragma unroll
                for (int r = 0; r < R; ++r) {
                    const uint32_t codes = tile + r * L::kRec + L::kSide;
                    // the weights in the second product's layout: head g, keys 2t, 2t + 1 and 2t + 8, 2t + 9.  For fp16
                    // outputs what their rounding leaves goes along, so that weight times scale is rounded once
                    constexpr bool kExact = std::is_same<T, __half>::value;
                    const uint32_t h0 = pack2<__half>(s[r][0], s[r][1]), h1 = pack2<__half>(s[r][2], s[r][3]);
                    const uint32_t p0 = transpose8x8(h0), p1 = transpose8x8(h1);
                    uint32_t l0 = 0, l1 = 0;
                    if (kExact) {
                        const float2 y = halves(h0), z = halves(h1);
                        l0 = transpose8x8(pack2<__half>(s[r][0] - y.x, s[r][1] - y.y));
                        l1 = transpose8x8(pack2<__half>(s[r][2] - z.x, s[r][3] - z.y));
                    }
                    uint32_t f[4];
#pragma unroll
                    for (int blk = 0; blk < NB; ++blk) {
                        const uint2 sc = lds64(codes + L::kScales + blk * 32 + t * 8);
                        uint32_t w0, w1;
                        if (kExact) {
                            w0 = fma2(p0, sc.x, mul2(l0, sc.x));
                            w1 = fma2(p1, sc.y, mul2(l1, sc.y));
                        } else {
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
                                mma_more(o[2 * blk + u], kBias[0], kBias[1], kBias[2], kBias[3], w0, w1);
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
                            mma_more(o[2 * blk], kBias[0], kBias[1], kBias[2], kBias[3], w0, w1);
                            mma_more(o[2 * blk + 1], kBias[0], kBias[1], kBias[2], kBias[3], w0, w1);
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
            top[0] = top[0] * factor[0] * beyond_s[warp][2 * t];
            top[1] = top[1] * factor[1] * beyond_s[warp][2 * t + 1];
            const float down = ex2(-up_w);
            sum[0] *= down;
            sum[1] *= down;
            out_unit *= down;
        }
        if constexpr (kAlone) {  // the warp's rows are whole
            if (n > 0 && *abort && lane == 0) atomicMax(&reported, int(QMM_ERR_DEVICE));
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const int row = 2 * t + h;
                if (row >= rows) continue;
                const bool none = !(sum[h] != 0.f);
                const float inv = none ? 0.f : 1.f / sum[h];
                T *const out = static_cast<T *>(d.out) + b * d.so.t + (head0 + row) * d.so.h;
#pragma unroll
                for (int blk = 0; blk < NB; ++blk) {
                    const float lo = out_unit * inv, hi = (kQ8 ? out_unit : out_unit * 0.0625f) * inv;  // of rows g, of rows g + 8
                    const uint32_t x = pack2<T>(o[2 * blk][h] * lo, o[2 * blk][2 + h] * hi);
                    const uint32_t y = pack2<T>(o[2 * blk + 1][h] * lo, o[2 * blk + 1][2 + h] * hi);
                    if constexpr (kQ8) {
                        *reinterpret_cast<uint32_t *>(out + 32 * blk + 2 * g) = x;
                        *reinterpret_cast<uint32_t *>(out + 32 * blk + 16 + 2 * g) = y;
                    } else {
                        *reinterpret_cast<uint2 *>(out + 32 * blk + 4 * g) = make_uint2(x, y);
                    }
                }
                if (d.lse && g == 0) d.lse[b * d.shape.hq + head0 + row] = none ? -INFINITY : (top[h] + log2f(sum[h])) * kLn2;
            }
            return;
        }
        __syncthreads();  // the ring is free
        const bool gave_up = *abort;
        piece = piece_s;
        const int64_t to = piece.b;  // the piece's request and heads again
        const int to_block = piece.pair % a.row_blocks, to_head = piece.pair / a.row_blocks * a.group + to_block * kRows;
        const int to_rows = min(a.group - to_block * kRows, kRows);
        float *part = reinterpret_cast<float *>(ring);
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const int row = 2 * t + h;
            float *dst = part + (warp * kRows + row) * L::kStride;
            if (row >= to_rows) continue;
#pragma unroll
            for (int blk = 0; blk < NB; ++blk) {
                const float lo = out_unit, hi = kQ8 ? out_unit : out_unit * 0.0625f;  // of rows g, of rows g + 8
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
        const int64_t row0 = to * d.shape.hq + to_head;
        for (int e = tid; e < to_rows * kQuads; e += kThreads) {
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
                const int64_t at = (int64_t(blockIdx.x) * 2 + piece.slot) * kRows + row;
                if (piece.whole) {
                    T *out = static_cast<T *>(d.out) + to * d.so.t + (to_head + row) * d.so.h + col;
                    *reinterpret_cast<uint2 *>(out) = make_uint2(pack2<T>(acc.x, acc.y), pack2<T>(acc.z, acc.w));
                } else {
                    *reinterpret_cast<float4 *>(a.part + at * D + col) = acc;
                }
                if (col == 0) {
                    if (!piece.whole) a.part_lse[at] = log2_total;
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
            dead |= gave_up;
            piece.begin += units_of(piece.tiles);
            if (piece.begin >= piece.end) break;
            piece.first = 0;
            piece.slot = 1;
            if (++piece.pair == pairs) {
                piece.pair = 0;
                do piece.tiles = request_tiles(++piece.b);
                while (piece.tiles == 0 && piece.b + 1 < d.batch);
            }
            continue;
        }
        if (ranks > 1) cluster_sync();
        else __syncthreads();

        // ------------------------------------------------ the cluster's rows
        for (int row = warp; row < to_rows; row += kWarps) {
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
        for (int e = rank + tid * ranks; e < to_rows * kQuads; e += ranks * kThreads) {
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
            T *out = static_cast<T *>(d.out) + to * d.so.t + (to_head + row) * d.so.h + col;
            *reinterpret_cast<uint2 *>(out) = make_uint2(pack2<T>(acc.x, acc.y), pack2<T>(acc.z, acc.w));
        }
        if (ranks > 1) cluster_sync();  // no CTA leaves while its shared memory may be read
        break;
    }
}

// The flat form's requests that were cut, joined: a block for each entry of a.cuts, whose warps share out the
// rows and then the parts of a row.  Requests without tiles, which no CTA has seen, give zeros.
constexpr int kJoinWarps = 32;
template <typename T> __global__ void __launch_bounds__(kJoinWarps * 32) kv_join_kernel(const __grid_constant__ Args a) {
    __shared__ float lse_s[kRows * kMaxParts];
    __shared__ float4 acc_s[kJoinWarps][32];
    grid_dependency_wait();
    grid_launch_dependents();
    const KvDecodeArgs &d = a.d;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, D = d.shape.d, col = lane * 4, pairs = d.shape.hk * a.row_blocks;
    for (int64_t b = blockIdx.x; b < d.batch && blockIdx.y == 0; b += gridDim.x) {
        if (request_len(d, b) > 0) continue;
        for (int e = tid; e < d.shape.hq * (D / 4); e += blockDim.x) {
            T *out = static_cast<T *>(d.out) + b * d.so.t + e / (D / 4) * d.so.h + e % (D / 4) * 4;
            *reinterpret_cast<uint2 *>(out) = make_uint2(0, 0);
        }
        if (d.lse)
            for (int h = tid; h < d.shape.hq; h += blockDim.x) d.lse[b * d.shape.hq + h] = -INFINITY;
    }
    if (a.by_pair && request_len(d, blockIdx.x / pairs) == 0) return;  // no CTA has written its entry
    const int4 info = __ldcg(a.cuts + blockIdx.x);
    const int parts = info.z, b = info.w / pairs, pair = info.w - b * pairs;
    // (lengths that changed under the call would leave an entry unwritten)
    if (parts <= 0 || info.x < 0 || parts > a.ctas - info.x || info.w < 0 || info.w >= d.batch * pairs) return;
    const int hk = pair / a.row_blocks, block = pair - hk * a.row_blocks;
    const int head0 = hk * a.group + block * kRows, rows = min(a.group - block * kRows, kRows);
    // a warp's row, and which of the row's parts: the first part is the CTA's last piece, the others are the
    // first pieces of the CTAs after it
    const bool by_row = gridDim.y > 1;  // or a block's one row
    if (by_row && (int)blockIdx.y >= rows) return;
    const int groups = by_row ? int(blockDim.x >> 5) : int(blockDim.x >> 5) / rows;
    const int row = by_row ? blockIdx.y : warp % rows, group = by_row ? warp : warp / rows;
    auto at = [&](int p) { return (int64_t(info.x + p) * 2 + (p == 0 ? info.y : 0)) * kRows; };
    float4 y[8], acc = make_float4(0.f, 0.f, 0.f, 0.f);
    auto load = [&](int p0) {
#pragma unroll
        for (int i = 0; i < 8; ++i)
            y[i] = col < D && p0 + i * groups < parts
                       ? __ldcg(reinterpret_cast<const float4 *>(a.part + (at(p0 + i * groups) + row) * D + col))
                       : make_float4(0.f, 0.f, 0.f, 0.f);
    };
    if (group < groups) load(group);
    for (int e = tid; e < parts * rows; e += blockDim.x) {
        const int p = e / rows;
        if (!by_row || e - p * rows == row) lse_s[e] = __ldcg(a.part_lse + at(p) + e - p * rows);
    }
    __syncthreads();
    float most = -INFINITY, sum = 0.f;
    for (int p = lane; p < parts; p += 32) most = fmaxf(most, lse_s[p * rows + row]);
#pragma unroll
    for (int s = 16; s > 0; s >>= 1) most = fmaxf(most, __shfl_xor_sync(0xffffffffu, most, s));
    const float base = most == -INFINITY ? 0.f : most;
    for (int p = lane; p < parts; p += 32) sum += ex2(lse_s[p * rows + row] - base);
#pragma unroll
    for (int s = 16; s > 0; s >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, s);
    const float inv = sum != 0.f ? 1.f / sum : 0.f;
    if (group < groups)
        for (int p0 = group; p0 < parts; p0 += 8 * groups) {
            if (p0 != group) load(p0);
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const int p = p0 + i * groups;
                const float w = p < parts ? ex2(lse_s[p * rows + row] - base) * inv : 0.f;
                acc.x += w * y[i].x;
                acc.y += w * y[i].y;
                acc.z += w * y[i].z;
                acc.w += w * y[i].w;
            }
        }
    if (groups > 1) {
        acc_s[warp][lane] = acc;
        __syncthreads();
    }
    if (group != 0) return;
    for (int i = 1; i < groups; ++i) {
        const float4 z = acc_s[by_row ? i : i * rows + row][lane];
        acc.x += z.x;
        acc.y += z.y;
        acc.z += z.z;
        acc.w += z.w;
    }
    T *out = static_cast<T *>(d.out) + int64_t(b) * d.so.t + (head0 + row) * d.so.h + col;
    if (col < D) *reinterpret_cast<uint2 *>(out) = make_uint2(pack2<T>(acc.x, acc.y), pack2<T>(acc.z, acc.w));
    if (d.lse && lane == 0) d.lse[int64_t(b) * d.shape.hq + head0 + row] = sum != 0.f ? (base + log2f(sum)) * kLn2 : -INFINITY;
}

size_t align256(size_t x) { return (x + 255) & ~size_t(255); }

// How a call is shared out: a warp for each request and kv head (both 0), clusters of `ranks` CTAs, or the flat form's
// CTAs (ranks == 0).
//
// A warp for each, four of them a CTA without any join, from one of them for every resident CTA and 8 tiles of the longest
// request on (and where there is a single tile; no further than 64, which one warp takes about 60 us for), CTAs and
// warps, 32/8 heads of 128: 2000 requests of 100 tokens 133.7 and 48.3 us; 256 of 30 20.7 and 7.5, of 100 22.0 and 11.5,
// of 250 25.3 and 18.6, of 1000 (32 tiles) 43.6 and 52.4; 128 of 100 12.8 and 9.1; 64 of 30 7.0 and 5.7, of 100 7.4 and
// 8.0; 1100 of 1000 158.9 and 130.9, of 2000 253.1 and 242.2.
//
// A cluster has a power of two CTAs, at most one for every four tiles, three an SM in all.  The flat form pays for its
// cuts (about 4 us and the join's launch) and wins where a warp of a cluster would get 12 tiles of the longest request or
// more, clusters and flat: 35 requests of up to 1001, 16 heads of 64 in 8 bits (8 tiles) 14.5 and 19.7 us; 256 of 500,
// 32/8 heads of 128 (4) 30.9 and 36.4; 1 of 12500 (6) 16.1 and 17.3, of 25000 (12) 22.7 and 21.7; 64 of 2000 (16) 26.8
// and 27.2; 16 of 8000 (31) 40.8 and 25.8; 48 of up to 8192 (32) 83.8 and 50.4.  Its CTAs get 16 tiles at least, so that
// the join stays small.  Beyond 1024 requests, whose lengths each warp would scan, there is no flat form: one long request
// among them is one CTA's or cluster's work (1000 requests of 100 tokens and one of 65536 107 us, 1100 and one 523).
struct Plan {
    int ranks, ctas;
};
Plan plan(const KvDecodeArgs &d) {
    const int64_t group = d.shape.hq / d.shape.hk, pairs = d.batch * d.shape.hk * ((group + kRows - 1) / kRows);
    const int64_t tiles = (d.max_len + 31) / 32, sms = device_sm_count();
    if (tiles == 1 || (tiles <= 64 && pairs >= kMaxCtas * sms && 8 * pairs >= kMaxCtas * sms * tiles)) return {0, 0};
    int ranks = 1;
    while (ranks < kMaxCluster && tiles >= 2 * ranks * kWarps && pairs * 2 * ranks <= 3 * sms) ranks *= 2;
    if (tiles >= 12 * ranks * kWarps && d.batch <= kMaxFlatBatch && d.batch * (tiles + kPieceUnits) < (int64_t(1) << 30))
        return {0, (int)std::min({pairs * tiles / 16, kMaxCtas * sms, int64_t(kMaxParts)})};
    return {ranks, 0};
}

template <typename T, bool kQ8, int D> cudaError_t launch(const Args &a, Plan p, int64_t pairs, cudaStream_t st) {
    using L = Tile<kQ8, D>;
    auto kern = p.ranks ? kv_decode_kernel<T, kQ8, D, kCluster> : p.ctas ? kv_decode_kernel<T, kQ8, D, kFlatRow> : kv_decode_kernel<T, kQ8, D, kWarpEach>;
    cudaError_t e = ensure_smem(kern, L::kSmem);
    if (e != cudaSuccess) return e;
    if (!p.ranks && !p.ctas) return launch_pdl(kern, dim3((unsigned)((pairs + kWarps - 1) / kWarps)), dim3(kThreads), L::kSmem, st, a);
    if (!p.ranks) {
        Args flat = a;
        flat.ctas = std::min(p.ctas, L::kCtas * device_sm_count());  // what the type and head size let stand at once
        flat.by_pair = pairs <= flat.ctas;
        e = launch_pdl(kern, dim3(flat.ctas), dim3(kThreads), L::kSmem, st, flat);
        if (e != cudaSuccess) return e;
        // few entries may have many parts each: a block of 32 warps for each row, else one of 8 warps for all
        const int entries = flat.by_pair ? (int)pairs : flat.ctas;
        const bool few = entries * kRows <= 2 * device_sm_count();
        return launch_pdl(kv_join_kernel<T>, dim3(entries, few ? std::min(flat.group, kRows) : 1),
                          dim3(32 * (few ? kJoinWarps : 8)), 0, st, flat);
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
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = p.ranks;
    attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
    attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[1].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 2;
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

namespace {
std::atomic<bool> launched{false};  // a kernel that may report has been launched (or captured) by this process
}

cudaError_t kv_decode_take_error(int *code, cudaStream_t st) {
    *code = QMM_OK;
    return launched ? take_error(code, st) : cudaSuccess;
}

size_t kv_decode_workspace_bytes(const KvDecodeArgs &d) {
    const size_t ctas = plan(d).ctas, rows = ctas * 2 * kRows;
    return align256(rows * d.shape.d * 4) + align256(rows * 4) + align256(ctas * sizeof(int4));
}

cudaError_t launch_kv_decode(const KvDecodeArgs &d, qmm_float t, void *ws, cudaStream_t st) {
    launched = true;
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
