// qmm_attn_tc.cu -- attention on the tensor cores: packed prompts, and a batch's queries over
// a prefix that all its requests share.
//
//   out = sum_j p_j v_j,  p = softmax_j(scale q.k_j) over the keys j that a row sees.
//
// A piece of work is 2 x 128 rows of one key/value head: the query heads that share it are rows of
// the same tile (row = token * G + g), so a tile of K and V is read once for all of them.  It walks
// the keys in tiles of 128 with the running maximum and sum of a softmax:
//   S_i = Q_i K_j^T (tcgen05, fp32 in tensor memory)   -> P_i = exp2(scale' (S_i - top)), rounded
//   to the inputs' type, in tensor memory              -> O_i += P_i V_j (A from tensor memory).
// The weights are rounded because a 16-bit product takes both operands in one type, V's: that adds
// an error of the size of the output's own rounding (against 64 bits 1.2 to 1.4 times what one
// rounding at the end leaves).  The sum of the weights is taken before the rounding, in fp32.
// While the softmax threads of one half (128 threads, one row each) work, the tensor cores run
// the other half's two products.  A row's maximum is only moved when a score passes it by more than
// 2^8 (weights then stay below 256, exact in the fp32 sums), so O_i is rarely rescaled.
//
// CTAs stay: each takes its next piece from the blocks of the grid that have not started, so that
// copies and scores of the next piece overlap the output of the last one.  Where the query tiles
// leave SMs without work, the keys are split and the parts joined by a second launch.
//
// Warps: 0-3 and 4-7 softmax of half 0 and 1, 8 copies (TMA), 9 products, 10 gate (it adds the
// copies' arrival to the weights' barrier), 11 pieces of work.
//
// 8192 causal tokens of 32/8 heads of 128, bf16: 336 us in a short graph, 1640 TFLOP/s, 85% of the
// measured bf16 rate; 361 us, 1520 TFLOP/s, 79%, where calls follow one another for long.
// Of a key tile's 2900 cycles the tensor pipe works on 2048; the rest is the issuing thread (its
// waits, and products that issue no faster than they run).  24 prompts of 9 to 2048 tokens: 239 us,
// 1060 TFLOP/s (248 in a row of calls): a piece's last softmax, output and change of piece take about 7000 cycles in which
// the tensor cores run little.  With heads up to 64 a tile takes about 2300 cycles for 1024 of products
// and as many of exponentials.
#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <type_traits>

#include "qmm_attn.cuh"
#include "qmm_internal.h"
#include "qmm_tc_common.cuh"
#include "qmm_tc_ptx.cuh"

namespace qmm {

namespace {

using namespace ptx;

constexpr int kRows = 128;    // rows of one half
constexpr int kKeys = 128;    // keys of one tile
constexpr int kTcThreads = 384;  // 168 registers each at launch: 64512 in all
constexpr int kSoftmaxRegs = 224, kOtherRegs = 56;  // 256 * 224 + 128 * 56 = 64512
constexpr float kSlack = 8.0f;  // how far (in powers of two) a row's scores may pass its maximum

// Shared-memory plan for a padded head size DP: Q_0, Q_1, then a ring of K and V tiles.  A tile
// is DP/64 blocks of 128 rows x 128 bytes, 128-byte swizzled.
template <int DP> struct Plan {
    static constexpr int kTile = kRows * DP * 2;
    static constexpr int kStages = DP == 128 ? 5 : 8;
    static constexpr size_t kBytes = size_t(2 + kStages) * kTile + 1024;
};

struct TcArgs {
    CUtensorMap q, k, v;
    void *out;              // direct output (part == nullptr)
    float *lse;             // [tokens][hq] natural log, or nullptr (part == nullptr)
    float *part;            // else normalised fp32 partial rows [split][tokens * hq][d]
    float *part_lse;        // and their log2 denominators [split][tokens * hq]
    const void *v_data;     // V again, for the rare rows with non-finite values
    HeadStrides so, sv;
    HeadShape shape;
    const int32_t *cu_q, *cu_k;  // nullptr: one sequence of tokens_q queries and tokens_k keys
    int64_t n_seqs, tokens_q, tokens_k;
    int group, per_half;    // query heads of a kv head, tokens of one half
    int causal, splits;
    float scale_log2;       // |scale| * log2(e)
    uint32_t idesc_qk, idesc_pv;
    int fault;              // qmm_set_test_fault: 1 no copy is issued, and the first wait for one is short;
                            // 2 the copies are issued, and the first wait for one gives up at once
    int *status;
};

// One piece of work: kv head hk, the query tokens from t0 on of a sequence of lq (row q0 first)
// with lk keys (row k0 first), and which of the key splits.
struct Item {
    int q0, lq, k0, lk, t0, hk, split;
    int valid;
    int odd;  // set while it is worked on: a non-finite value was taken out of a V tile
    // its key tiles, [ja, jb0) and [ja, jb1) for the halves, [ja, jb) for either; the keys that all
    // of its rows, and all rows of the second half, see
    int ja, jb0, jb1, jb, vis_lo, vis_lo1;
};

__device__ __forceinline__ float max3(float a, float b, float c) {
    float d;
    asm("max.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
    return d;
}
// Two fp32 fused multiply-adds / additions in one instruction.
__device__ __forceinline__ void fma2(float &x, float &y, float a0, float a1, float b, float c) {
    asm("{\n.reg .b64 p, q, r;\nmov.b64 p, {%2, %3};\nmov.b64 q, {%4, %4};\nmov.b64 r, {%5, %5};\n"
        "fma.rn.f32x2 p, p, q, r;\nmov.b64 {%0, %1}, p;\n}"
        : "=f"(x), "=f"(y)
        : "f"(a0), "f"(a1), "f"(b), "f"(c));
}
__device__ __forceinline__ void add2(float &x, float &y, float a0, float a1) {
    asm("{\n.reg .b64 p, q;\nmov.b64 p, {%0, %1};\nmov.b64 q, {%2, %3};\nadd.rn.f32x2 p, p, q;\nmov.b64 {%0, %1}, p;\n}"
        : "+f"(x), "+f"(y)
        : "f"(a0), "f"(a1));
}
// The registers of earlier tensor-memory loads may be used from here on.
template <int N> __device__ __forceinline__ void loaded(float (&v)[N]) {
#pragma unroll
    for (int i = 0; i < N; ++i) asm volatile("" : "+f"(v[i]));
}

__device__ __forceinline__ void tma_load_3d(uint32_t dst, const CUtensorMap *map, int x, int y, int z, uint32_t bar) {
    asm volatile(
        "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4}], "
        "[%5];" ::"r"(dst),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(z), "r"(bar)
        : "memory");
}

// Lane l holds N 16-byte units of row l, unit u in x[u]; afterwards x[e] of lane l is unit
// l * N / 32 of row (32 / N) * e + l % (32 / N), so that a warp's store of x[e] writes whole pieces
// of N units of 32 / N rows (a lane that writes its own row touches a line of its own with every
// store, and the tile takes 3 to 4 times as long).  An N x N transposition: the unit's bits change
// places with the row's upper bits, one a step.
template <int N> __device__ __forceinline__ void rows_to_pieces(uint4 (&x)[N], int lane) {
#pragma unroll
    for (int bit = N / 2; bit; bit >>= 1) {
        const int other = bit * (32 / N);
        const bool upper = lane & other;
#pragma unroll
        for (int u = 0; u < N; ++u) {
            if (u & bit) continue;
            uint4 &lo = x[u], &hi = x[u | bit];
            uint4 give = upper ? lo : hi;
            give.x = __shfl_xor_sync(0xffffffffu, give.x, other);
            give.y = __shfl_xor_sync(0xffffffffu, give.y, other);
            give.z = __shfl_xor_sync(0xffffffffu, give.z, other);
            give.w = __shfl_xor_sync(0xffffffffu, give.w, other);
            if (upper) lo = give;
            else hi = give;
        }
    }
}

// Operand whose rows run along the MMA's K and whose contiguous side is M or N (V): 64-element
// blocks lbo bytes apart, groups of 8 rows 1024 bytes apart, 128-byte swizzle.
__device__ __forceinline__ uint64_t smem_desc_mn(uint32_t addr, uint32_t lbo_bytes) {
    return uint64_t((addr & 0x3FFFFu) >> 4) | (uint64_t((lbo_bytes >> 4) & 0x3FFFu) << 16) |
           (uint64_t(1024 >> 4) << 32) | (uint64_t(1) << 46) | (uint64_t(2) << 61);
}

// One lane of the converged warp, always the same one.
__device__ __forceinline__ bool elect_one() {
    uint32_t yes;
    asm volatile("{\n.reg .pred p;\nelect.sync _|p, 0xffffffff;\nselp.u32 %0, 1, 0, p;\n}" : "=r"(yes));
    return yes != 0;
}
// mbar_wait_spin by a whole warp: all lanes go on, or all give up.
__device__ __forceinline__ bool spin_wait(uint32_t bar, uint32_t parity, volatile int *abort) {
    return __all_sync(0xffffffffu, mbar_wait_spin(bar, parity, abort));
}

// Clamped [cu[s], cu[s + 1]) as (first, length).
__device__ __forceinline__ void seq_bounds(const int32_t *cu, int64_t s, int64_t most, int &first, int &len) {
    const int64_t a = min(max(int64_t(cu[s]), int64_t(0)), most), b = min(max(int64_t(cu[s + 1]), int64_t(0)), most);
    first = int(a);
    len = int(max(b - a, int64_t(0)));
}

// One sequence's query tiles of `span` tokens.
struct Tiles {
    int q0, lq, k0, lk, count;

    // The first of its tiles whose last token sees keys of at least x key tiles, `count` if there is
    // none; the tiles after it see at least as many.
    __device__ __forceinline__ int first_with(int x, int span, int causal) const {
        const int64_t keys = int64_t(kKeys) * (x - 1) + 1;
        if (x <= 0) return 0;
        if (lk < keys) return count;
        const int64_t last = causal ? keys - lk + lq : 0;  // the last token that a tile has to reach, less 1: at most lq
        return last <= span ? 0 : int((unsigned(last) + unsigned(span) - 1) / unsigned(span)) - 1;
    }
};

__device__ __forceinline__ Tiles tiles_of(const TcArgs &a, int64_t s, int span) {
    Tiles t = {0, 0, 0, 0, 0};
    if (a.cu_q && s < a.n_seqs) {
        seq_bounds(a.cu_q, s, a.tokens_q, t.q0, t.lq);
        seq_bounds(a.cu_k, s, a.tokens_k, t.k0, t.lk);
        t.count = int((unsigned(t.lq) + unsigned(span) - 1) / unsigned(span));
    }
    return t;
}

// The rank'th tile of `span` tokens, most key tiles first (so that the last items to start are
// short ones; a lane holds a sequence), or for more sequences than lanes the last sequence's last
// tile first.  One warp; false when there is no such tile.  24 prompts of up to 2048 tokens, 32/8 heads
// of 128: 222 us sorted, 230 not; 32 of up to 1000: 102.2, 103.3; 8 of up to 500: even.
constexpr int kSortedSeqs = 32;
// Where the last search among many sequences ended: a CTA's ranks rise, so that it passes each
// sequence once (from the last sequence for every piece, 8192 prompts of 4 tokens took 4.8 ms).
struct Walk {
    int64_t chunk, before;  // first of 32 sequences, tiles of the chunks after it
};
__device__ __forceinline__ Walk walk_start(const TcArgs &a) { return {(a.n_seqs - 1) / 32 * 32, 0}; }
__device__ __forceinline__ bool find_item(const TcArgs &a, unsigned rank, int span, int lane, const Tiles &own, Walk &w,
                                          Item &it) {
    if (!a.cu_q) {
        it.q0 = it.k0 = 0;
        it.lq = int(a.tokens_q);
        it.lk = int(a.tokens_k);
        it.t0 = int(rank) * span;
        return int64_t(rank) * span < a.tokens_q;
    }
    if (a.n_seqs <= kSortedSeqs) {  // lane l holds sequence l
        const Tiles &t = own;
        if (rank >= __reduce_add_sync(0xffffffffu, unsigned(t.count))) return false;
        // the largest x for which more than `rank` tiles see at least x key tiles
        int lo = 0, hi = int(__reduce_max_sync(0xffffffffu, unsigned(t.lk)) / kKeys) + 2;
        while (hi - lo > 1) {
            const int mid = lo + (hi - lo) / 2;
            const unsigned n = __reduce_add_sync(0xffffffffu, unsigned(t.count - t.first_with(mid, span, a.causal)));
            if (n > rank) lo = mid;
            else hi = mid;
        }
        const int first = t.first_with(lo, span, a.causal), next = t.first_with(hi, span, a.causal);
        // rank among the tiles with exactly lo key tiles, sequence by sequence
        const unsigned left = unsigned(rank) - __reduce_add_sync(0xffffffffu, unsigned(t.count - next));
        unsigned incl = unsigned(next - first);
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const unsigned x = __shfl_up_sync(0xffffffffu, incl, o);
            if (lane >= o) incl += x;
        }
        const unsigned before = incl - unsigned(next - first);
        const int src = __ffs(__ballot_sync(0xffffffffu, left >= before && left < incl)) - 1;
        it.q0 = __shfl_sync(0xffffffffu, t.q0, src);
        it.lq = __shfl_sync(0xffffffffu, t.lq, src);
        it.t0 = int(__shfl_sync(0xffffffffu, unsigned(first) - before, src) + left) * span;
        it.k0 = __shfl_sync(0xffffffffu, t.k0, src);
        it.lk = __shfl_sync(0xffffffffu, t.lk, src);
        return true;
    }
    if (rank < w.before) w = walk_start(a);
    for (; w.chunk >= 0; w.chunk -= 32) {  // lane l: the l'th sequence from the chunk's end
        const Tiles t = tiles_of(a, w.chunk + 31 - lane, span);
        unsigned incl = unsigned(t.count);
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const unsigned x = __shfl_up_sync(0xffffffffu, incl, o);
            if (lane >= o) incl += x;
        }
        const int64_t last = w.before + incl, first = last - t.count;
        const unsigned hit = __ballot_sync(0xffffffffu, rank >= first && rank < last);
        if (hit) {
            const int src = __ffs(hit) - 1;
            it.q0 = __shfl_sync(0xffffffffu, t.q0, src);
            it.lq = __shfl_sync(0xffffffffu, t.lq, src);
            it.t0 = int(__shfl_sync(0xffffffffu, int(last - 1 - rank), src)) * span;
            it.k0 = __shfl_sync(0xffffffffu, t.k0, src);
            it.lk = __shfl_sync(0xffffffffu, t.lk, src);
            return true;
        }
        w.before += __shfl_sync(0xffffffffu, incl, 31);
    }
    return false;
}

// Keys that query token t of the sequence sees.
__device__ __forceinline__ int visible(const TcArgs &a, const Item &it, int t) {
    if (!a.causal) return it.lk;
    const int64_t n = int64_t(t) + 1 + it.lk - it.lq;
    return int(min(max(n, int64_t(0)), int64_t(it.lk)));
}

__device__ __forceinline__ void set_range(const TcArgs &a, Item &it) {
    it.vis_lo = visible(a, it, it.t0);
    it.vis_lo1 = visible(a, it, it.t0 + a.per_half);
    int n[2];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const int first = it.t0 + i * a.per_half, last = min(first + a.per_half, it.lq) - 1;
        n[i] = last >= first ? (visible(a, it, last) + kKeys - 1) / kKeys : 0;
    }
    const int most = max(n[0], n[1]), per_split = a.splits > 1 ? (most + a.splits - 1) / a.splits : most;
    const int end = min((it.split + 1) * per_split, most);
    it.ja = min(it.split * per_split, most);
    it.jb0 = max(min(end, n[0]), it.ja);
    it.jb1 = max(min(end, n[1]), it.ja);
    it.jb = max(it.jb0, it.jb1);
}

template <typename T> struct Pair;
template <> struct Pair<__half> {
    using type = __half2;
    static constexpr uint32_t kExp = 0x7c007c00u, kOne = 0x04000400u;
};
template <> struct Pair<__nv_bfloat16> {
    using type = __nv_bfloat162;
    static constexpr uint32_t kExp = 0x7f807f80u, kOne = 0x00800080u;
};
// acc + 0 * u: stays zero until an infinity or NaN comes by, and is NaN from then on.
template <typename T> __device__ __forceinline__ void taint(uint32_t &acc, uint32_t u) {
    using P = typename Pair<T>::type;
    const uint32_t zero = 0;
    const P r = __hfma2(*reinterpret_cast<const P *>(&u), *reinterpret_cast<const P *>(&zero),
                        *reinterpret_cast<const P *>(&acc));
    acc = *reinterpret_cast<const uint32_t *>(&r);
}
// The packed pair without its infinite and NaN values.
template <typename T> __device__ __forceinline__ uint32_t finite2(uint32_t u) {
    const uint32_t bad = (u & Pair<T>::kExp) + Pair<T>::kOne;  // bits 15 and 31: exponent all ones
    if (bad & 0x8000u) u &= 0xffff0000u;
    if (bad & 0x80000000u) u &= 0x0000ffffu;
    return u;
}

// A tile's V rows [from, end) may be unseen by some rows, and the rows from `end` on belong to
// nobody: a weight of zero times what they hold must stay zero.  Rows from `end` on become
// zeros; an infinity or NaN before `end` becomes zero and is reported (the rows that see it
// take it in at the end).  One warp, on a tile of DP/64 blocks of 128 x 128 bytes; eight loads
// in flight and one instruction a pair, or the tile's product would wait for this.
template <typename T, int DP> __device__ __forceinline__ bool clean_values(uint8_t *tile, int from, int end, int lane) {
    uint32_t acc[4] = {0, 0, 0, 0};
    for (int b = 0; b < DP / 64; ++b) {
        uint4 *rows = reinterpret_cast<uint4 *>(tile + b * kKeys * 128);
        for (int i0 = from * 8 + lane; i0 < end * 8; i0 += 32 * 8) {
            uint4 u[8];
#pragma unroll
            for (int e = 0; e < 8; ++e) u[e] = rows[min(i0 + 32 * e, end * 8 - 1)];
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                taint<T>(acc[0], u[e].x);
                taint<T>(acc[1], u[e].y);
                taint<T>(acc[2], u[e].z);
                taint<T>(acc[3], u[e].w);
            }
        }
        for (int i = end * 8 + lane; i < kKeys * 8; i += 32) rows[i] = make_uint4(0, 0, 0, 0);
    }
    const bool odd = __any_sync(0xffffffffu, (acc[0] | acc[1] | acc[2] | acc[3]) & 0x7fff7fffu);
    if (odd) {
        for (int b = 0; b < DP / 64; ++b) {
            uint32_t *rows = reinterpret_cast<uint32_t *>(tile + b * kKeys * 128);
#pragma unroll 1
            for (int i = from * 32 + lane; i < end * 32; i += 32) rows[i] = finite2<T>(rows[i]);
        }
    }
    fence_proxy_async_smem();
    __syncwarp();  // one lane arrives for all: the others' rows come first
    return odd;
}

constexpr int kItemRoles = 11;  // warps that read an item: softmax, copies, products, gate

struct Bars {
    uint64_t full[8], empty[8];           // the ring's stages; empty and q_empty: one arrival a half
    uint64_t q, q_empty;
    uint64_t s[2], l[2], p[2][2], o[2];    // scores complete, scores loaded, weights stored, output complete
    uint64_t item[2], item_empty[2], want, next, drain;
};

// Ask the hardware for the next block of the grid that has not started: its index, or -1.  One warp.
__device__ __forceinline__ int64_t take_next_block(uint4 *answer, uint32_t bar, uint32_t parity, int lane,
                                                   volatile int *abort) {
    if (lane == 0) {
        fence_proxy_async_smem();
        mbar_arrive_expect_tx(bar, 16);
        asm volatile("clusterlaunchcontrol.try_cancel.async.shared::cta.mbarrier::complete_tx::bytes.b128 [%0], [%1];" ::"r"(
                         smem_u32(answer)),
                     "r"(bar)
                     : "memory");
    }
    __syncwarp();
    if (!warp_wait(bar, parity, abort)) {
        int never = 0;
        warp_wait(bar, parity, &never);  // the answer lands before shared memory is released
        return -1;
    }
    uint32_t yes, id;
    asm volatile(
        "{\n.reg .b128 r;\n.reg .pred p;\nld.shared.b128 r, [%2];\n"
        "clusterlaunchcontrol.query_cancel.is_canceled.pred.b128 p, r;\nselp.u32 %0, 1, 0, p;\nmov.u32 %1, 0;\n"
        "@p clusterlaunchcontrol.query_cancel.get_first_ctaid::x.b32.b128 %1, r;\n}"
        : "=r"(yes), "=r"(id)
        : "r"(smem_u32(answer))
        : "memory");
    __syncwarp();
    return yes ? int64_t(id) : -1;
}

// kPartial: fp32 partial rows of a key split instead of the output.
template <typename T, int DP, bool kPartial>
__global__ void __launch_bounds__(kTcThreads, 1) attn_tc_kernel(const __grid_constant__ TcArgs a) {
    using P = Plan<DP>;
    constexpr int ST = P::kStages;
    // Tensor memory (512 columns): S_0, S_1 (128 each), O_0, O_1 (DP each).  With DP = 128 it is full and
    // the weights take the place of their scores, so that S(j + 1) waits for the product with V_j.  With
    // DP = 64 they have columns of their own: S(j + 1) is formed as soon as the softmax has loaded S(j),
    // and the softmax is never without scores (5 prompt chunks of up to 509 tokens after 3500, 32 heads
    // of 64: 47.6 -> 42 us).
    constexpr bool kOwnP = DP == 64;
    constexpr int kPCol = kOwnP ? 256 + 2 * DP : 0, kPStep = kOwnP ? kKeys / 2 : kKeys;
    constexpr int kParts = kOwnP ? 1 : 2;  // parts of a tile's weights that are handed over one by one
    extern __shared__ uint8_t raw[];
    __shared__ Bars bars;
    __shared__ Item items[2];
    __shared__ __align__(16) uint4 answer;
    __shared__ uint32_t tmem_s;
    __shared__ int abort_s;
    __shared__ uint32_t issued_s, q_issued_s;  // ring copies and items' Q copies so far
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    grid_launch_dependents();  // a launch that waits for this one's end may take free SMs

    if (tid == 0) {
        abort_s = 0;
        issued_s = q_issued_s = 0;
        for (int i = 0; i < ST; ++i) {
            mbar_init(smem_u32(&bars.full[i]), 1);
            mbar_init(smem_u32(&bars.empty[i]), 2);
        }
        mbar_init(smem_u32(&bars.q), 1);
        mbar_init(smem_u32(&bars.q_empty), 2);
        for (int i = 0; i < 2; ++i) {
            mbar_init(smem_u32(&bars.s[i]), 1);
            mbar_init(smem_u32(&bars.l[i]), 5);
            for (int h = 0; h < kParts; ++h) mbar_init(smem_u32(&bars.p[i][h]), h == 0 ? 5 : 4);
            mbar_init(smem_u32(&bars.o[i]), 1);
            mbar_init(smem_u32(&bars.item[i]), 1);
            mbar_init(smem_u32(&bars.item_empty[i]), kItemRoles);
        }
        mbar_init(smem_u32(&bars.want), 1);
        mbar_init(smem_u32(&bars.next), 1);
        mbar_init(smem_u32(&bars.drain), 1);
        fence_mbar_init();
    }
    if (warp == 8) {
        tmem_alloc(smem_u32(&tmem_s), 512);
        tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = tmem_s;
    volatile int *abort = &abort_s;

    const uint32_t sm0 = (smem_u32(raw) + 1023u) & ~1023u;
    const uint32_t sq = sm0, skv = sm0 + 2 * P::kTile;

    // The k'th item of this CTA, for a whole warp; false at the end.
    auto get_item = [&](int k, Item &it) -> bool {
        if (!warp_wait(smem_u32(&bars.item[k & 1]), (k >> 1) & 1, abort)) return false;
        it = items[k & 1];
        return it.valid;
    };
    auto done_with_item = [&](int k) {
        __syncwarp();
        if (lane == 0) mbar_arrive(smem_u32(&bars.item_empty[k & 1]));
    };
    // Parities: an item's first ring stage, tile of half i, ... is counted over all items of the CTA.
    uint32_t base = 0, tiles0 = 0, tiles1 = 0, worked = 0;  // stages, tiles of each half, items with keys
    auto advance = [&](const Item &r) {
        base += 2 * (r.jb - r.ja);
        tiles0 += r.jb0 - r.ja;
        tiles1 += r.jb1 - r.ja;
        worked += r.jb > r.ja;
    };

    if (warp >= 8) {
    regs_dec<kOtherRegs>();
    if (warp == 11) {
        // ------------------------------------------------ items: this block's, then blocks that have not started
        int64_t id = blockIdx.x;
        int asked = 0;
        const Tiles own = tiles_of(a, lane, 2 * a.per_half);
        Walk walk = walk_start(a);
        for (int k = 0;; ++k) {
            if (k >= 2 && !warp_wait(smem_u32(&bars.item_empty[k & 1]), ((k >> 1) - 1) & 1, abort)) break;
            Item it;
            it.valid = 0;
            if (id >= 0) {
                if (id == 0 && lane == 0) *a.status = QMM_OK;  // long before a wait can give up
                // blocks in order: all heads and splits of a tile, then the next tile
                const unsigned rest = unsigned(id) / unsigned(a.shape.hk), rank = rest / unsigned(a.splits);
                it.hk = int(unsigned(id) - rest * unsigned(a.shape.hk));
                it.split = int(rest - rank * unsigned(a.splits));
                it.valid = find_item(a, rank, 2 * a.per_half, lane, own, walk, it);  // no tile: no later block has one
            }
            if (it.valid) set_range(a, it);
            if (lane == 0) {
                it.odd = 0;
                items[k & 1] = it;
                mbar_arrive(smem_u32(&bars.item[k & 1]));
            }
            __syncwarp();
            if (!it.valid) {
                // the grid counts a tile for every sequence that may hold tokens: the blocks past the
                // last tile are taken here, or each would start a CTA that searches all sequences
                while (id >= 0 && !*abort) id = take_next_block(&answer, smem_u32(&bars.next), asked++ & 1, lane, abort);
                break;
            }
            // the next one once this one's copies are under way: not earlier, or the last items
            // would wait behind long ones
            if (!warp_wait(smem_u32(&bars.want), k & 1, abort)) break;
            id = take_next_block(&answer, smem_u32(&bars.next), asked++ & 1, lane, abort);
        }
    } else if (warp == 8) {
        // ------------------------------------------------ copies
        bool ok = true;
        if (lane == 0) {
            prefetch_tmap(&a.q);
            prefetch_tmap(&a.k);
            prefetch_tmap(&a.v);
        }
        Item it;
        for (int k = 0; get_item(k, it); ++k) {
            if (it.jb > it.ja) {
                if (worked > 0) ok = warp_wait(smem_u32(&bars.q_empty), (worked - 1) & 1, abort);
                if (ok && lane == 0 && a.fault != 1) {
                    const uint32_t bar = smem_u32(&bars.q), box = uint32_t(a.group * a.per_half) * 128;
                    const bool half[2] = {it.jb0 > it.ja, it.jb1 > it.ja};
                    mbar_arrive_expect_tx(bar, box * (DP / 64) * (uint32_t(half[0]) + uint32_t(half[1])));
                    for (int i = 0; i < 2; ++i)
                        for (int b = 0; b < DP / 64; ++b)
                            if (half[i])
                                tma_load_3d(sq + i * P::kTile + b * kRows * 128, &a.q, b * 64, it.hk * a.group,
                                            it.q0 + it.t0 + i * a.per_half, bar);
                    q_issued_s = worked + 1;
                }
                __syncwarp();
            }
            for (int j = it.ja; j < it.jb && ok; ++j) {
                for (int kv = 0; kv < 2 && ok; ++kv) {
                    const uint32_t n = base + 2 * (j - it.ja) + kv, stg = n % ST;
                    if (n >= ST) ok = warp_wait(smem_u32(&bars.empty[stg]), (n / ST - 1) & 1, abort);
                    if (ok && lane == 0 && a.fault != 1) {
                        const uint32_t bar = smem_u32(&bars.full[stg]);
                        mbar_arrive_expect_tx(bar, P::kTile);
                        for (int b = 0; b < DP / 64; ++b)
                            tma_load_3d(skv + stg * P::kTile + b * kKeys * 128, kv ? &a.v : &a.k, b * 64, it.hk,
                                        it.k0 + j * kKeys, bar);
                        issued_s = n + 1;
                    }
                    __syncwarp();
                }
            }
            if (lane == 0) mbar_arrive(smem_u32(&bars.want));
            advance(it);
            if (!ok) break;
            done_with_item(k);
        }
    } else if (warp == 9) {
        // ------------------------------------------------ products, issued by one elected lane
        // The lane runs an item's whole loop: elected, so that the operands are uniform, and without
        // the votes and synchronisations of a warp, which would cost as much as the issue.
        bool ok = true;
        const uint64_t qd = smem_desc(sq, 1024, 2), kd0 = smem_desc(skv, 1024, 2), vd0 = smem_desc_mn(skv, kKeys * 128);
        auto qk = [&](int i, uint32_t n) {
            const uint64_t kd = kd0 + uint32_t((n % ST) * P::kTile >> 4);
#pragma unroll
            for (int s = 0; s < DP / 16; ++s) {
                const uint32_t off = (uint32_t(s / 4) * kRows * 128 + uint32_t(s % 4) * 32) >> 4;
                mma_f16(tmem + i * kKeys, qd + uint32_t(i * P::kTile >> 4) + off, kd + off, a.idesc_qk, s != 0);
            }
            mma_commit(smem_u32(&bars.s[i]));
        };
        Item it;
        for (int k = 0; ok && get_item(k, it); ++k) {
            if (elect_one()) {
                if (it.jb > it.ja) {
                    if (a.fault == 2) *abort = 1;
                    ok = a.fault != 2 && mbar_wait_spin(smem_u32(&bars.q), worked & 1, abort, a.fault ? 100000 : kWaitCycles) &&
                         mbar_wait_spin(smem_u32(&bars.full[base % ST]), (base / ST) & 1, abort);
                    tc_fence_after();
                    if (ok && it.jb0 > it.ja) qk(0, base);
                    if (ok && it.jb1 > it.ja) qk(1, base);
                }
#pragma unroll 1
                for (int turn = 0; ok && turn < 2 * (it.jb - it.ja); ++turn) {
                    const int i = turn & 1, j = turn >> 1, left = (i ? it.jb1 : it.jb0) - it.ja - j;
                    if (left <= 0) continue;
                    const uint32_t n = base + 2 * j + 1, tile = (i ? tiles1 : tiles0) + j;
                    const uint64_t vd = vd0 + uint32_t((n % ST) * P::kTile >> 4);
                    if (kOwnP) {
                        ok = mbar_wait_spin(smem_u32(&bars.l[i]), tile & 1, abort);
                        if (!ok) break;
                        tc_fence_after();
                        if (left > 1) qk(i, n + 1);
                    }
#pragma unroll
                    for (int h = 0; h < kParts; ++h) {
                        ok = ok && mbar_wait_spin(smem_u32(&bars.p[i][h]), tile & 1, abort);
                        if (!ok) break;
                        tc_fence_after();
#pragma unroll
                        for (int s = h * 8 / kParts; s < (h + 1) * 8 / kParts; ++s)
                            mma_f16_tmem_a(tmem + 256 + i * DP, tmem + kPCol + i * kPStep + s * 8,
                                           vd + uint32_t(s * 16 * 128 >> 4), a.idesc_pv, j > 0 || s > 0);
                    }
                    if (!ok) break;
                    if (!kOwnP && left > 1) qk(i, n + 1);
                    else mma_commit(smem_u32(&bars.o[i]));
                }
            }
            __syncwarp();
            ok = !*abort;
            advance(it);
            if (ok) done_with_item(k);
        }
    } else {
        // ------------------------------------------------ gate (warp 10): V_j and K_{j+1} have arrived
        // One arrival of each half's weight barrier (and of that of loaded scores, where S(j + 1) waits
        // for it), so that the issuer waits for nothing else, after
        // V rows that not every row sees are cleaned, and the releases of a half that takes no part.
        bool ok = true;
        Item it;
        for (int k = 0; ok && get_item(k, it); ++k) {
            auto arrived = [&](uint32_t n) {
                ok = ok && warp_wait(smem_u32(&bars.full[n % ST]), (n / ST) & 1, abort);
            };
            if (it.jb > it.ja) {
                arrived(base);
                if (it.jb0 == it.ja || it.jb1 == it.ja) {
                    ok = ok && warp_wait(smem_u32(&bars.q), worked & 1, abort);
                    if (ok && lane == 0) mbar_arrive(smem_u32(&bars.q_empty));
                }
            }
            for (int j = it.ja; j < it.jb && ok; ++j) {
                const uint32_t n = base + 2 * (j - it.ja) + 1, stg = n % ST;
                arrived(n);
                if (ok && (j + 1) * kKeys > it.vis_lo &&
                    clean_values<T, DP>(raw + (sm0 - smem_u32(raw)) + (2 + stg) * P::kTile,
                                        max(it.vis_lo - j * kKeys, 0), min(it.lk - j * kKeys, kKeys), lane) &&
                    lane == 0)
                    items[k & 1].odd = 1;
                if (j + 1 < it.jb) arrived(n + 1);
                for (int i = 0; i < 2 && ok; ++i) {
                    if (j >= (i ? it.jb1 : it.jb0)) {
                        if (lane == 0) {
                            mbar_arrive(smem_u32(&bars.empty[(n - 1) % ST]));
                            mbar_arrive(smem_u32(&bars.empty[stg]));
                        }
                        continue;
                    }
                    const uint32_t tile = (i ? tiles1 : tiles0) + (j - it.ja);
                    auto add = [&](uint64_t &bar) {  // to this tile's phase: the last tile's is complete
                        if (tile > 0) ok = ok && warp_wait(smem_u32(&bar), (tile - 1) & 1, abort);
                        if (ok && lane == 0) mbar_arrive(smem_u32(&bar));
                    };
                    if (kOwnP) add(bars.l[i]);
                    add(bars.p[i][0]);
                }
                __syncwarp();
            }
            advance(it);
            if (ok) done_with_item(k);
        }
    }
    } else {
        // ------------------------------------------------ softmax, one row a thread
        regs_inc<kSoftmaxRegs>();
        // Little is kept over the tile loop next to the 128 scores: what the output needs of the
        // item is read again (a spilled register costs hundreds of cycles: shared memory leaves
        // next to no L1 cache).
        const int i = warp >> 2;
        const uint32_t lanes = uint32_t((warp & 3) * 32) << 16;
        const uint32_t s_addr = tmem + lanes + i * kKeys, o_addr = tmem + lanes + 256 + i * DP;
        const uint32_t p_addr = tmem + lanes + kPCol + i * kPStep;
        const bool releases = (tid & 127) == 0;
        const int mine = (tid & 127) / a.group;  // this row's token within the half
        uint32_t tiles = 0, outputs = 0;  // tiles of this half so far, items in which it took part
        bool ok = true;
        for (int k = 0; ok; ++k) {
            ok = warp_wait(smem_u32(&bars.item[k & 1]), (k >> 1) & 1, abort);
            if (!ok || !items[k & 1].valid) break;
            // tiles to do and to count for the ring; keys from the first tile on that this row,
            // and that every row of the half, sees
            int count, stages, vis, vis_half;
            {
                const Item it = items[k & 1];
                count = (i ? it.jb1 : it.jb0) - it.ja;
                stages = 2 * (it.jb - it.ja);
                const int t = it.t0 + i * a.per_half + mine;
                vis = (mine < a.per_half && t < it.lq ? visible(a, it, t) : 0) - it.ja * kKeys;
                vis_half = (i ? it.vis_lo1 : it.vis_lo) - it.ja * kKeys;
            }
            float top = -INFINITY, sum0 = 0.f, sum1 = 0.f;
#pragma unroll 1
            for (int j = 0; j < count; ++j) {
                ok = warp_wait(smem_u32(&bars.s[i]), (tiles + j) & 1, abort);
                if (!ok) break;
                // S_i(j) is complete: so are the reads of K_j and, unless it was issued before it, O_i's
                // product with V_{j-1}
                auto release = [&](uint32_t n) {
                    if (releases) mbar_arrive(smem_u32(&bars.empty[n % ST]));
                };
                release(base + 2 * j);
                if (!kOwnP && j > 0) release(base + 2 * j - 1);
                if (releases && j + 1 == count) mbar_arrive(smem_u32(&bars.q_empty));
                tc_fence_after();
                float s[kKeys];
#pragma unroll
                for (int c = 0; c < 4; ++c) tmem_ld_32x32b_x32(s_addr + c * 32, *reinterpret_cast<float(*)[32]>(s + c * 32));
                tmem_ld_wait();
                loaded(s);
                if (kOwnP) {
                    tc_fence_before();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(smem_u32(&bars.l[i]));
                }
                if ((j + 1) * kKeys > vis_half) {
                    const int left = vis - j * kKeys;
#pragma unroll
                    for (int c = 0; c < kKeys; ++c)
                        if (c >= left) s[c] = -INFINITY;
                }
                float m0 = s[0], m1 = s[1], m2 = s[2], m3 = s[3];
#pragma unroll
                for (int c = 4; c < kKeys; c += 8) {
                    m0 = max3(m0, s[c], s[c + 1]);
                    m1 = max3(m1, s[c + 2], s[c + 3]);
                    if (c + 4 < kKeys) {
                        m2 = max3(m2, s[c + 4], s[c + 5]);
                        m3 = max3(m3, s[c + 6], s[c + 7]);
                    }
                }
                const float most = fmaxf(fmaxf(m0, m1), fmaxf(m2, m3));
                if (kOwnP && j > 0) {  // the last weights are read and O_i is at rest
                    ok = warp_wait(smem_u32(&bars.o[i]), (tiles + j - 1) & 1, abort);
                    if (!ok) break;
                    tc_fence_after();
                    release(base + 2 * j - 1);
                }
                // move the maximum when a score passes it by more than the slack
                const bool move = (most - top) * a.scale_log2 > kSlack || (top == -INFINITY && most > -INFINITY);
                if (j == 0) {
                    if (move) top = most;
                } else if (__any_sync(0xffffffffu, move)) {
                    const float now = move ? most : top;
                    const float f = top == -INFINITY ? 1.f : ex2((top - now) * a.scale_log2);
                    top = now;
                    sum0 *= f;
                    sum1 *= f;
                    // O_i's last product is done: awaited, or issued before S_i(j)
#pragma unroll 1
                    for (int c = 0; c < DP / 16; ++c) {
                        float o[16];
                        tmem_ld_32x32b_x16(o_addr + c * 16, o);
                        tmem_ld_wait();
                        loaded(o);
#pragma unroll
                        for (int e = 0; e < 16; ++e) o[e] *= f;
                        tmem_st_32x32b_x16(o_addr + c * 16, o);
                    }
                }
                const float shift = top == -INFINITY ? 0.f : -top * a.scale_log2;
#pragma unroll
                for (int c = 0; c < kKeys / 32; ++c) {
                    uint32_t p[16];
#pragma unroll
                    for (int e = 0; e < 16; ++e) {
                        const int x = c * 32 + 2 * e;
                        fma2(s[x], s[x + 1], s[x], s[x + 1], a.scale_log2, shift);
                        s[x] = ex2(s[x]);
                        s[x + 1] = ex2(s[x + 1]);
                        p[e] = pack2<T>(s[x], s[x + 1]);
                        add2(sum0, sum1, s[x], s[x + 1]);
                    }
                    tmem_st_32x32b_x16(p_addr + c * 16, p);
                    if (c % (4 / kParts) == 4 / kParts - 1) {  // a part of the keys: its product may begin
                        tmem_st_wait();
                        tc_fence_before();
                        __syncwarp();
                        if (lane == 0) mbar_arrive(smem_u32(&bars.p[i][c / (4 / kParts)]));
                    }
                }
            }
            if (ok && count > 0) {
                ok = warp_wait(smem_u32(&bars.o[i]), (kOwnP ? tiles + count - 1 : outputs) & 1, abort);
                ++outputs;
                if (ok && releases) mbar_arrive(smem_u32(&bars.empty[(base + 2 * count - 1) % ST]));
            }
            if (ok) {
                tc_fence_after();
                const Item it = items[k & 1];
                const int t = it.t0 + i * a.per_half + mine;
                const bool row_valid = mine < a.per_half && t < it.lq;
                const float sum = count > 0 ? sum0 + sum1 : 0.f;
                const bool none = !(sum != 0.f);  // no key seen (a NaN sum is not none)
                const float inv = none ? 0.f : 1.f / sum;
                const int head = it.hk * a.group + (tid & 127) - mine * a.group;
                const int64_t row = (int64_t(it.q0) + t) * a.shape.hq + head;
                const bool odd = count > 0 && it.odd;
                // where this lane's row goes, in elements of what is stored; of the rows that it helps to write
                using Out = typename std::conditional<kPartial, float, T>::type;
                constexpr int kUnits = 32 * int(sizeof(Out)) / 16;  // of 32 elements
                Out *const out = kPartial ? reinterpret_cast<Out *>(a.part) : static_cast<Out *>(a.out);
                const int64_t out_row = !row_valid ? -1
                                        : kPartial ? (int64_t(it.split) * a.tokens_q * a.shape.hq + row) * a.shape.d
                                                   : (int64_t(it.q0) + t) * a.so.t + head * a.so.h;
                int64_t to[kUnits];
#pragma unroll
                for (int e = 0; e < kUnits; ++e)
                    to[e] = __shfl_sync(0xffffffffu, out_row, (32 / kUnits) * e + (lane & (32 / kUnits - 1)));
#pragma unroll 1
                for (int c = 0; c < DP && __any_sync(0xffffffffu, row_valid); c += 32) {  // rolled: code that runs once an item is fetched anew each time
                    float o[32];
                    tmem_ld_32x32b_x32(o_addr + c, o);
                    tmem_ld_wait();
                    loaded(o);
#pragma unroll
                    for (int e = 0; e < 32; ++e) o[e] = none ? 0.f : o[e] * inv;
                    uint4 x[kUnits];
#pragma unroll
                    for (int e = 0; e < kUnits; ++e) {
                        if (kPartial)
                            x[e] = make_uint4(__float_as_uint(o[4 * e]), __float_as_uint(o[4 * e + 1]),
                                              __float_as_uint(o[4 * e + 2]), __float_as_uint(o[4 * e + 3]));
                        else
                            x[e] = make_uint4(pack2<T>(o[8 * e], o[8 * e + 1]), pack2<T>(o[8 * e + 2], o[8 * e + 3]),
                                              pack2<T>(o[8 * e + 4], o[8 * e + 5]), pack2<T>(o[8 * e + 6], o[8 * e + 7]));
                    }
                    rows_to_pieces(x, lane);
                    const int col = c + lane / (32 / kUnits) * (32 / kUnits);
#pragma unroll
                    for (int e = 0; e < kUnits; ++e)
                        if (to[e] >= 0 && col < a.shape.d) *reinterpret_cast<uint4 *>(out + to[e] + col) = x[e];
                }
                if (odd) {
                    // Non-finite values that were taken out of V: a row that sees one adds it to what the
                    // rest came to, which may be an infinity or NaN itself (a NaN score, a value of a tile
                    // that every row sees).  After the warp's stores above, which other lanes made.
                    __syncwarp();
                    const int from = max(it.vis_lo, it.ja * kKeys);
                    const int end = row_valid ? min(visible(a, it, t), (it.ja + count) * kKeys) : from;
                    const T *v = static_cast<const T *>(a.v_data) + it.hk * a.sv.h;
#pragma unroll 1
                    for (int e = 0; e < a.shape.d; ++e) {
                        float total = 0.f;
#pragma unroll 1
                        for (int key = from; key < end; ++key) {
                            const float x = float(v[(int64_t(it.k0) + key) * a.sv.t + e]);
                            if (!isfinite(x)) total += x;
                        }
                        if (!isfinite(total)) out[out_row + e] = Out(float(out[out_row + e]) + total);
                    }
                }
                if (row_valid) {
                    const float l2 = none ? -INFINITY : top * a.scale_log2 + log2f(sum);
                    if (kPartial) a.part_lse[int64_t(it.split) * a.tokens_q * a.shape.hq + row] = l2;
                    else if (a.lse) a.lse[row] = l2 * kLn2;
                }
            }
            tc_fence_before();
            base += stages;
            tiles += count;
            if (ok) done_with_item(k);
        }
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (*abort) {  // a wait gave up: what was issued ends before shared and tensor memory are released
        int never = 0;
        if (warp == 8) {
            if (q_issued_s > 0) warp_wait(smem_u32(&bars.q), (q_issued_s - 1) & 1, &never);
            for (uint32_t n = issued_s > ST ? issued_s - ST : 0; n < issued_s; ++n) {
                never = 0;
                warp_wait(smem_u32(&bars.full[n % ST]), (n / ST) & 1, &never);
            }
        } else if (warp == 9) {
            if (elect_one()) mma_commit(smem_u32(&bars.drain));
            spin_wait(smem_u32(&bars.drain), 0, &never);
        }
        if (tid == 0) *a.status = gave_up = QMM_ERR_DEVICE;
        __syncthreads();
    }
    if (warp == 8) tmem_dealloc(tmem, 512);
}

// The joined output row of a prompt call with key splits: out = sum_s 2^(lse_s) part_s / sum_s 2^(lse_s),
// one warp a row, four elements a lane.
template <typename T> __global__ void __launch_bounds__(128) attn_join_kernel(const __grid_constant__ TcArgs a) {
    grid_dependency_wait();  // in every block: this launch ends after the parts' launch
    const int lane = threadIdx.x & 31, d = a.shape.d;
    const int64_t rows = a.tokens_q * a.shape.hq, row = int64_t(blockIdx.x) * 4 + (threadIdx.x >> 5);
    if (row >= rows) return;
    const int64_t t = row / a.shape.hq;
    const int h = int(row - t * a.shape.hq);
    bool mine = false;  // whether some sequence holds this query: other rows are not written
    for (int64_t s = lane; s < a.n_seqs; s += 32) {
        int q0, lq;
        seq_bounds(a.cu_q, s, a.tokens_q, q0, lq);
        mine |= t >= q0 && t < int64_t(q0) + lq;
    }
    if (!__any_sync(0xffffffffu, mine)) return;
    float l[2], top = -INFINITY;  // of splits lane and lane + 32
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const int s = lane + 32 * i;
        l[i] = s < a.splits ? a.part_lse[s * rows + row] : -INFINITY;
        top = fmaxf(top, l[i]);
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
    const float base = top == -INFINITY ? 0.f : top;
    float sum = 0.f;
#pragma unroll
    for (int i = 0; i < 2; ++i) sum += l[i] = ex2(l[i] - base);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
    const bool none = !(sum != 0.f);
    const float inv = none ? 0.f : 1.f / sum;
    float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
    const bool live = 4 * lane < d;
    const float *src = a.part + row * d + (live ? 4 * lane : 0);
    for (int s0 = 0; s0 < a.splits; s0 += 8) {
        float4 x[8];
#pragma unroll
        for (int i = 0; i < 8; ++i)
            x[i] = __ldcg(reinterpret_cast<const float4 *>(src + int64_t(min(s0 + i, a.splits - 1)) * rows * d));
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const float w = __shfl_sync(0xffffffffu, s0 < 32 ? l[0] : l[1], (s0 + i) & 31) * inv;
            if (s0 + i >= a.splits) continue;
            acc.x += w * x[i].x;
            acc.y += w * x[i].y;
            acc.z += w * x[i].z;
            acc.w += w * x[i].w;
        }
    }
    if (live)
        *reinterpret_cast<uint2 *>(static_cast<T *>(a.out) + t * a.so.t + h * a.so.h + 4 * lane) =
            make_uint2(pack2<T>(acc.x, acc.y), pack2<T>(acc.z, acc.w));
    if (a.lse && lane == 0) a.lse[row] = none ? -INFINITY : (base + log2f(sum)) * kLn2;
}

template <typename T, int DP> cudaError_t launch_dp(const TcArgs &a, int64_t blocks, cudaStream_t st) {
    auto kern = a.part ? attn_tc_kernel<T, DP, true> : attn_tc_kernel<T, DP, false>;
    cudaError_t e = ensure_smem(kern, Plan<DP>::kBytes);
    if (e != cudaSuccess) return e;
    kern<<<(unsigned)blocks, kTcThreads, Plan<DP>::kBytes, st>>>(a);
    return cudaGetLastError();
}

// What the two launches have in common.
TcArgs common_args(const HeadShape &shape, qmm_float t, float scale, void *ws) {
    TcArgs a{};
    a.shape = shape;
    a.group = shape.hq / shape.hk;
    a.per_half = kRows / a.group;
    a.splits = 1;
    // a scale of 0 (all keys alike) as the smallest one, so that a hidden key's -infinity stays one;
    // a negative scale negates Q in the product
    a.scale_log2 = std::max(std::abs(scale) * kLog2e, 1.2e-38f);
    const uint32_t type_bits = t == QMM_F16 ? 0u : (1u << 7) | (1u << 10);
    a.idesc_qk = idesc_f16_f32(kRows, kKeys) | type_bits | (scale < 0.f ? 1u << 13 : 0u);
    a.idesc_pv = idesc_f16_f32(kRows, shape.d <= 64 ? 64 : 128) | type_bits | (1u << 16);
    a.status = static_cast<int *>(ws);
    a.fault = test_fault_mode();
    return a;
}

cudaError_t launch_tc(const TcArgs &a, qmm_float t, int64_t blocks, cudaStream_t st) {
    if (blocks > 0x7fffffff) return cudaErrorInvalidConfiguration;
    if (t == QMM_F16)
        return a.shape.d <= 64 ? launch_dp<__half, 64>(a, blocks, st) : launch_dp<__half, 128>(a, blocks, st);
    return a.shape.d <= 64 ? launch_dp<__nv_bfloat16, 64>(a, blocks, st)
                           : launch_dp<__nv_bfloat16, 128>(a, blocks, st);
}

}  // namespace

namespace {

// Upper bound of a prompt call's query tiles: n sequences of l_i > 0 tokens have
// sum (floor((l_i - 1) / span) + 1) <= floor((tokens - n) / span) + n, which grows with n.
int64_t prompt_tiles(const PromptArgs &p) {
    const int64_t span = 2 * (kRows / (p.shape.hq / p.shape.hk)), n = std::min(p.n_seqs, p.tokens_q);
    return (p.tokens_q - n) / span + n;
}

// Key splits of a prompt call: where the tiles would leave half of the SMs or more without work, as
// many as give each SM an item, of at least four key tiles (counted for sequences of equal lengths:
// the host does not know theirs; a long chunk beside short prompts is not split).  With parts of at
// least 2, 4 and 8 tiles, 32/8 heads of 128: 64 tokens on 1300 keys 16.6, 20.0, 22.9 us; on 2100 17.1,
// 19.2, 24.0; on 4096 19.7, 18.7, 23.5; 128 on 2000 18.5, 21.6, 29.9; 256 on 4000 27.7, 27.6, 30.9: two
// would be the better bound for most of these.
int prompt_splits(const PromptArgs &p) {
    const int64_t items = prompt_tiles(p) * p.shape.hk;
    if (items == 0 || p.n_seqs == 0) return 1;
    const int64_t key_tiles = p.tokens_k / p.n_seqs / kKeys;
    return int(std::max<int64_t>(1, std::min<int64_t>({device_sm_count() / items, key_tiles / 4, kMaxSplits})));
}

size_t align256(size_t x) { return (x + 255) & ~size_t(255); }

}  // namespace

cudaError_t attn_tc_take_gave_up(bool *yes, cudaStream_t st) { return take_gave_up(yes, st); }

size_t attn_prompt_workspace_bytes(const PromptArgs &p) {
    const size_t splits = prompt_splits(p), rows = size_t(p.tokens_q) * p.shape.hq;
    return splits == 1 ? 256 : 256 + align256(splits * rows * p.shape.d * 4) + align256(splits * rows * 4);
}

cudaError_t launch_attn_prompt(const PromptArgs &p, qmm_float t, void *ws, cudaStream_t st) {
    TcArgs a = common_args(p.shape, t, p.scale, ws);
    if (!attn_make_map(&a.q, t, p.q, p.shape.d, p.shape.hq, p.tokens_q, p.sq, a.group, a.per_half))
        return cudaErrorInvalidValue;
    // without any key the maps are not used; they describe q then
    const bool keys = p.tokens_k > 0;
    if (!attn_make_map(&a.k, t, keys ? p.k : p.q, p.shape.d, keys ? p.shape.hk : 1, keys ? p.tokens_k : 1, p.sk, 1, kKeys) ||
        !attn_make_map(&a.v, t, keys ? p.v : p.q, p.shape.d, keys ? p.shape.hk : 1, keys ? p.tokens_k : 1, p.sv, 1, kKeys))
        return cudaErrorInvalidValue;
    a.out = p.out;
    a.lse = p.lse;
    a.v_data = p.v;
    a.so = p.so;
    a.sv = p.sv;
    a.cu_q = p.cu_q;
    a.cu_k = p.cu_k;
    a.n_seqs = p.n_seqs;
    a.tokens_q = p.tokens_q;
    a.tokens_k = p.tokens_k;
    a.causal = p.causal;
    a.splits = prompt_splits(p);
    const int64_t rows = p.tokens_q * p.shape.hq;
    if (a.splits > 1) {
        uint8_t *at = static_cast<uint8_t *>(ws) + 256;
        a.part = reinterpret_cast<float *>(at);
        a.part_lse = reinterpret_cast<float *>(at + align256(size_t(a.splits) * rows * p.shape.d * 4));
    }
    const cudaError_t e = launch_tc(a, t, prompt_tiles(p) * a.splits * p.shape.hk, st);
    if (e != cudaSuccess || a.splits == 1) return e;
    auto join = t == QMM_F16 ? attn_join_kernel<__half> : attn_join_kernel<__nv_bfloat16>;
    return launch_pdl(join, dim3((unsigned)((rows + 3) / 4)), dim3(128), 0, st, a);
}

// The prefix's key splits: enough CTAs (tiles of queries x kv heads x splits) for every SM, at
// least two key tiles each.  With at least 1, 2 and 4, 32/8 heads of 128, requests x prefix: 32 x 700
// 11.4, 12.6, 17.0 us; 16 x 1300 12.0, 12.8, 16.3; 8 x 2600 13.0, 12.9, 15.3; 4 x 5200 14.0, 14.1, 16.0.
int attn_prefix_splits(const DecodeArgs &d) {
    const int64_t span = 2 * (kRows / (d.shape.hq / d.shape.hk));
    const int64_t pairs = (d.batch + span - 1) / span * d.shape.hk, tiles = (d.prefix + kKeys - 1) / kKeys;
    const int64_t most = std::max<int64_t>(1, std::min<int64_t>({device_sm_count() / pairs, tiles / 2, int64_t(kMaxSplits)}));
    const int64_t per = (tiles + most - 1) / most;
    return int((tiles + per - 1) / per);
}

cudaError_t launch_attn_prefix(const DecodeArgs &d, qmm_float t, int splits, float *part, float *part_lse, void *ws,
                               cudaStream_t st) {
    TcArgs a = common_args(d.shape, t, d.scale, ws);
    if (!attn_make_map(&a.q, t, d.q, d.shape.d, d.shape.hq, d.batch, d.sq, a.group, a.per_half) ||
        !attn_make_map(&a.k, t, d.pk, d.shape.d, d.shape.hk, d.prefix, d.spk, 1, kKeys) ||
        !attn_make_map(&a.v, t, d.pv, d.shape.d, d.shape.hk, d.prefix, d.spv, 1, kKeys))
        return cudaErrorInvalidValue;
    a.part = part;
    a.part_lse = part_lse;
    a.v_data = d.pv;
    a.sv = d.spv;
    a.n_seqs = 1;
    a.tokens_q = d.batch;
    a.tokens_k = d.prefix;
    a.splits = splits;
    const int64_t tiles = (d.batch + 2 * a.per_half - 1) / (2 * a.per_half);
    return launch_tc(a, t, tiles * splits * d.shape.hk, st);
}

}  // namespace qmm
