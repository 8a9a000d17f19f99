// Attention of a tree of drafted tokens over a paged cache, on the 5th-generation tensor cores of sm_103a.
//
// What it computes: the newest tree_len[b] cached tokens of sequence b are the nodes of a drafted tree (several
// continuations verified in one pass over their positions; speculative decoding paragraph of "Tornar a inferência
// barata", neuralialabs.com).  Node t's query row attends to the whole history before the tree and to the nodes whose
// bit is set in its mask (its ancestors and itself, normally):
//   out = softmax(q K^T * scale + mask) V,   a row whose mask leaves nothing gives 0,
// with the running-max / exp-sum rule of the FlashAttention article over key tiles and over chunks of the context.
//
// Layout.  The tree_len * G query rows of a (sequence, KV head), G = Hq / Hkv, are the M = 128 side of both products
// in tiles of 128 rows (row = node * G + head of the group; a TMEM lane and a softmax thread each), the keys the other
// side in tiles of 128 (8 cache blocks), worked on in halves of 64.  A CTA works on two streams A and B, each with four
// row warps, two buffers of scores / weights and an output accumulator in TMEM:
//   two row tiles     the streams are the row tiles and share every K/V tile (the tile is read once for 256 rows);
//   one row tile      the streams are the two halves of every key tile for the same rows, merged at the end.
// Per stream X and step of 64 keys:  S_X = Q_X K^T (both K-major in shared memory, 128-byte swizzle, as TMA writes the
// blocks); the row warps take S_X from TMEM, keep the running max lazily (it moves when it has grown by 2^4; O_X is
// then rescaled in TMEM) and write P_X over S_X in fp16;  O_X += P_X V with P_X from TMEM and V MN-major.  Two buffers
// let S of the next step run under this step's softmax; steps of 64 keys instead of 128 make room for both.
// Warps.  Eight row warps; one product warp per stream and product (S_A, S_B, PV_A, PV_B: a wait costs a warp about 200
// clocks and a product 40 to 90, so that one warp for all of them was the bound); a copy warp each for K and V.  The
// two buffers and the four product warps together took 8 x 4096 keys, 64 nodes, 32 / 8 heads, D = 128 from 57 to 37 us.
// Sixteen row warps, two to a row, are slower (40.2 against 38.3 us), and so is one row tile per CTA (42 us).
// P.  With an fp16 output the weights are one fp16 value and the row sums add the rounded weights, so a row is a
// convex combination of V rows; with an fp32 output they are an fp16 high part plus residual (two products).  A weight
// is within 2^-11 / 2^-20 of itself, or 2^-36 of its row's largest one where that is more (see kWeightLog2).
// Split.  The context is cut into chunks where (sequence, KV head, row tile pair) units are fewer than SMs.  Up to
// eight CTAs of a unit are a cluster: each leaves its states (max, sum, O) in its shared memory and merges a share of
// the rows from all of them.  Where a unit has several clusters their states go through the workspace to the combine
// kernel below.  A merge reads about 15 bytes per clock and SM from the other CTAs, whatever the instruction (loads,
// stores, asynchronous stores and bulk copies: 4.3 to 4.9 K clocks for 64 KB): half of the 9 K clocks between the last
// product of a CTA with two row tiles and its end.  Through global memory instead that step took 47.6 us.
// What bounds it (us; bytes and products at the card's measured rates in parentheses):
//   4 x 65,536 keys, 16 nodes, 32 / 8 heads, D = 128    156   (158)  memory
//   8 x 4096 keys, 64 nodes, 32 / 8 heads, D = 128      37.0   (21)  3.0 K clocks per key tile for two row tiles, of
//                                                       which the products alone take 2.05 K, and the merge
//   32 x <= 2048 keys, 16 nodes, 14 / 2 heads, D = 64   15.0  (4.6)  start (2.2), 1.5 K clocks per key tile (memory,
//                                                       on 128 of the SMs), end (3.5: last product, barriers, merge)
//   1 x 2048 keys, 8 nodes, 14 / 2 heads, D = 64         8.1  (0.2)  start, two key tiles, end
// With fp32 outputs (twice the P V products) 160, 46.0, 16.4 and 8.6.
// Every wait is bounded.
#include <algorithm>
#include <cfloat>
#include <type_traits>

#include "../../include/kvc.h"
#include "decode_common.cuh"
#include "kvc_internal.h"
#include "ptx.cuh"
#include "tcgen05.cuh"

namespace kvc {
namespace tree {

constexpr int kRows = 128;  // rows of a row tile
constexpr int kKeys = 128;  // keys of a key tile
constexpr int kHalf = 64;   // keys of one step of a stream
constexpr int kPages = kKeys / kBlockSize;
constexpr int kRowWarps = 8;
constexpr int kSWarp = kRowWarps;        // S products of stream A, of stream B
constexpr int kPvWarp = kRowWarps + 2;   // P V products of stream A, of stream B
constexpr int kLoadKWarp = kRowWarps + 4;
constexpr int kLoadVWarp = kRowWarps + 5;
constexpr int kThreads = (kRowWarps + 6) * 32;
constexpr int kMaxTreeCluster = 8;
constexpr uint64_t kWaitNs = 1000000000ull;
// a scale of 0 is taken as this: the scores of fp16 rows (below 2^40) still vanish next to 1, and a masked score of
// -inf times it stays -inf
constexpr float kMinScaleLog2 = 0x1p-100f;
// A weight is 2^(x - m) for a score of exponent x.  The running m lies 2^11 below the largest score so far and moves
// when a score is 2^15 above it, inside fp16's 2^16: a weight keeps fp16's 11 bits down to 2^-25 of its row's largest one
// and 2^-36 of that below.  The factor is in the row's sum too and costs no time.  (With the largest weight at 1, a key
// 2^25 below another one was lost, and 65,536 of those are 1.4e-3 of a row.)
constexpr float kWeightLog2 = 11.f;
constexpr float kRescaleLog2 = 15.f;
// Scores of finite fp16 rows reach 2^41, where neighbouring fp32 exponents x lie 2^18 apart: x - m, exact in the
// weights' multiply-add, can then be any number although m came from the same score.  So m is rounded down (the largest
// score's x - m is never negative: no row is lost), and weights are cut off at fp16's largest value: scores as close as
// their own rounding count as equal.  The conversion of an fp16-output weight does that by itself (a branch over the
// scores in its place cost 2 % of 8 x 4096 keys with 64 nodes); the split weights' exponents are cut off where a row's m
// is beyond kFar, from where on a step is no longer small against fp16's range.
constexpr float kFar = 0x1p22f;

template <int D>
struct Geom {
    static constexpr int kChunks = D / 64;  // 64-dim (128-byte) column chunks
    static constexpr int kKStages = D == 64 ? 5 : 3;
    static constexpr int kVStages = D == 64 ? 5 : 2;
    static constexpr int kChunkBytes = kRows * 128;  // 128 rows or keys x 64 dims
    static constexpr int kTileBytes = kChunks * kChunkBytes;
    // Q_A, Q_B, V ring, K ring.  With one row tile Q_B's place is one more V stage (V is freed last: its product waits
    // for the softmax).
    static constexpr int kQOff = 0;
    static constexpr int kVOff = kQOff + 2 * kTileBytes;
    static constexpr int kKOff = kVOff + kVStages * kTileBytes;
    static constexpr int kBarOff = kKOff + kKStages * kTileBytes;
    static constexpr int kMaxVStages = kVStages + 1;
    static constexpr int kSmemBytes = kBarOff + 512 + 1024;  // barriers, TMEM address, flags; alignment
    static_assert(kSmemBytes <= 227 * 1024, "shared memory of one CTA");
    // at the end the row threads leave their states in the idle V and K rings: per thread (max, sum), and a row of O,
    // padded so that eight rows lie on distinct banks
    static constexpr int kOStride = D + 4;  // floats
    static constexpr int kStateOff = kVOff;
    static constexpr int kMlOff = kStateOff + 2 * kRows * kOStride * 4;
    static constexpr int kWeightOff = kMlOff + 2 * kRows * 8;  // the states' weights of the rows this CTA merges
    // (rows / CTAs, rounded up, times CTAs: at most 2 * 128 and one more row's)
    static_assert(kWeightOff + (2 * kRows + kMaxTreeCluster) * 8 <= kBarOff, "state area");
    // TMEM columns: two buffers of S / P per stream, A [0, 128) and B [128, 256), then O_A and O_B, D columns each
    static constexpr int kTmemO = 4 * kHalf;
    static constexpr uint32_t kTmemCols = 512;
};

struct Params {
    const __half* q;
    const int32_t* block_table;
    const int32_t* context_lens;
    const int32_t* tree_lens;
    const uint64_t* masks;
    const __half* v_cache;
    void* out;
    float* part_ml;
    float* part_acc;
    unsigned* err;
    int T, Hq, Hkv, G, max_blocks, num_blocks, max_ctx, out_f32;
    int chunk;      // key tiles per CTA
    int cluster;    // CTAs per cluster: consecutive chunks of one unit, merged in distributed shared memory
    int nclus;      // clusters along the longest context: stride of the partial states
    int row_pairs;  // pairs of row tiles of the widest tree
    uint32_t g_magic;  // ceil(2^18 / G): row * g_magic >> 18 = row / G for rows below 4096
    int negate;      // scale < 0: the query rows change sign as they are loaded
    float scale_log2;  // |scale| * log2 e, at least kMinScaleLog2 and finite
};

__device__ __forceinline__ uint32_t sw128(int row, int c) {
    return static_cast<uint32_t>(row * 128 + ((c ^ (row & 7)) << 4));
}

// acc + the two fp16 halves of h (each converted exactly), as two rounded fp32 additions
__device__ __forceinline__ float add_halves(uint32_t h, float acc) {
    asm("{\n\t.reg .f16 lo, hi;\n\tmov.b32 {lo, hi}, %1;\n\tadd.rn.f32.f16 %0, lo, %0;\n\t"
        "add.rn.f32.f16 %0, hi, %0;\n\t}"
        : "+f"(acc)
        : "r"(h));
    return acc;
}
__device__ __forceinline__ float max3f(float a, float b, float c) {
    float r;
    asm("max.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
    return r;
}
__device__ __forceinline__ bool try_wait_sleep(uint64_t* bar, uint32_t parity) {
    uint32_t ok;
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2, %3;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(ok)
        : "r"(smem_u32(bar)), "r"(parity), "r"(20000u)
        : "memory");
    return ok != 0;
}
// Wait for a phase; gives up when another thread of the CTA has given up (abort flag) or after the limit, in which
// case it raises the flag itself.
__device__ __forceinline__ bool wait(uint64_t* bar, uint32_t parity, volatile int* abort_flag) {
    if (mbar_try_wait(bar, parity)) return true;
    const uint64_t t0 = global_timer_ns();
    for (;;) {
        if (try_wait_sleep(bar, parity)) return true;
        if (*abort_flag) return false;
        if (global_timer_ns() - t0 > kWaitNs) {
            *abort_flag = 1;
            return false;
        }
    }
}
// The same for a whole warp whose waits sit between two products: it polls instead of sleeping.
__device__ __forceinline__ bool wait_poll(uint64_t* bar, uint32_t parity, volatile int* abort_flag) {
    if (__all_sync(0xffffffffu, mbar_test(bar, parity))) return true;
    const uint64_t t0 = global_timer_ns();
    for (uint32_t i = 1;; ++i) {
        if (__all_sync(0xffffffffu, mbar_test(bar, parity))) return true;
        if ((i & 255u) == 0u) {
            if (__any_sync(0xffffffffu, *abort_flag != 0)) return false;
            if (__any_sync(0xffffffffu, global_timer_ns() - t0 > kWaitNs)) {
                *abort_flag = 1;
                return false;
            }
        }
    }
}
__device__ __forceinline__ void bar_sync(int id, int threads) {
    asm volatile("bar.sync %0, %1;" ::"r"(id), "r"(threads) : "memory");
}
__device__ __forceinline__ void bar_arrive(int id, int threads) {
    asm volatile("bar.arrive %0, %1;" ::"r"(id), "r"(threads) : "memory");
}
__device__ __forceinline__ void row_warps_sync() { asm volatile("bar.sync 1, %0;" ::"n"(kRowWarps * 32) : "memory"); }

// an infinity or NaN among the 8 fp16 values of a chunk
__device__ __forceinline__ bool half_nonfinite(uint32_t h) { return (h & 0x7C00u) == 0x7C00u; }
__device__ __forceinline__ uint32_t finite_halves(uint32_t w, bool& found) {
    if (half_nonfinite(w)) {
        w &= 0xFFFF0000u;
        found = true;
    }
    if (half_nonfinite(w >> 16)) {
        w &= 0x0000FFFFu;
        found = true;
    }
    return w;
}

__device__ __forceinline__ uint32_t cluster_addr(uint32_t addr, int rank) {
    uint32_t r;
    asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(addr), "r"(rank));
    return r;
}
__device__ __forceinline__ float2 ld_cluster_f32x2(uint32_t addr) {
    float2 v;
    asm volatile("ld.shared::cluster.v2.f32 {%0, %1}, [%2];" : "=f"(v.x), "=f"(v.y) : "r"(addr) : "memory");
    return v;
}
__device__ __forceinline__ float4 ld_cluster_f32x4(uint32_t addr) {
    float4 v;
    asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];"
                 : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w)
                 : "r"(addr)
                 : "memory");
    return v;
}

__device__ __forceinline__ bool lengths_fit(const Params& p, int tree, int ctx) {
    return tree >= 0 && tree <= p.T && ctx >= tree && ctx <= p.max_ctx &&
           ctx <= static_cast<int64_t>(p.max_blocks) * kBlockSize;
}
__device__ __forceinline__ int key_tiles(int ctx) { return (ctx + kKeys - 1) / kKeys; }

template <int D, bool kSplitP>
__global__ void __launch_bounds__(kThreads, 1) paged_decode_tree_kernel(const __grid_constant__ CUtensorMap tmK,
                                                                         const __grid_constant__ CUtensorMap tmV,
                                                                         const Params p) {
    using Geo = Geom<D>;
    constexpr int KS = Geo::kKStages, MVS = Geo::kMaxVStages;
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    uint64_t* bars = reinterpret_cast<uint64_t*>(smem + Geo::kBarOff);
    uint64_t* q_full = bars;                 // query rows in shared memory (one arrival per row warp)
    uint64_t* k_full = bars + 1;             // [KS] K tile landed
    uint64_t* k_empty = k_full + KS;         // [KS] S products of the stage's tile done
    uint64_t* v_full = k_empty + KS;         // [MVS] V tile landed
    uint64_t* v_empty = v_full + MVS;        // [MVS] P V products of the stage's tile done
    uint64_t* s_full = v_empty + MVS;        // [2][2] S of stream x's buffer i in TMEM (index 2 x + i)
    uint64_t* p_full = s_full + 4;           // [2][2] P of the buffer in TMEM (4 arrivals)
    uint64_t* o_full = p_full + 4;           // [2][2] P V of the buffer done
    uint64_t* fin = o_full + 4;              // [4] every product that a product warp issued is done
    uint64_t* v_land = fin + 4;              // [2] the V tiles that reach into the tree landed (then mended)
    uint32_t* s_tmem = reinterpret_cast<uint32_t*>(v_land + 2);
    volatile int* s_abort = reinterpret_cast<volatile int*>(s_tmem + 1);
    volatile int* s_bad_block = s_abort + 1;  // a block id out of range: the chunk is left out
    volatile int* s_bad_v = s_abort + 2;      // an infinity or NaN among the tree's V values
    volatile int* s_bad_of = s_abort + 3;     // bit q: CTA q of the cluster has noted such values
    static_assert((1 + 2 * KS + 2 * MVS + 18) * 8 + 20 <= 512, "barrier area");

    // (the shuffle tells the compiler that the warp index is the same in all lanes: the product warp's descriptors and
    // counters then live in uniform registers, as its instructions want them)
    const int warp = __shfl_sync(0xffffffffu, static_cast<int>(threadIdx.x >> 5), 0), lane = threadIdx.x & 31;
    // blockIdx.x = (cluster along the context * row pairs + row pair) * CTAs per cluster + rank
    const int rank = static_cast<int>(blockIdx.x) % p.cluster;
    const int pair = static_cast<int>(blockIdx.x) / p.cluster % p.row_pairs;
    const int clus = static_cast<int>(blockIdx.x) / p.cluster / p.row_pairs;
    const int hk = blockIdx.y, b = blockIdx.z;
    const int r0 = pair * 2 * kRows;
    const int per_clus = p.chunk * p.cluster, c0 = clus * per_clus + rank * p.chunk;
    auto node_of = [&](int rr) { return static_cast<int>(static_cast<uint32_t>(rr) * p.g_magic >> 18); };  // rr / G

    // Loads that do not depend on the lengths go out together with them: the block ids of the first four key tiles
    // (entries past the context are not used) and the query rows (rows past the tree are not used).
    const int32_t* const table_row = p.block_table + static_cast<int64_t>(b) * p.max_blocks;
    auto block_ids = [&](int j) {  // of tiles j .. j + 3, eight lanes each
        const int page = (c0 + j) * kPages + lane;
        return page < p.max_blocks ? table_row[page] : 0;
    };
    grid_dependency_wait();  // nothing is read or written before the kernel in front is done
    const int tree = p.tree_lens != nullptr ? p.tree_lens[b] : p.T, ctx = p.context_lens[b];
    int ids = 0;
    constexpr int kQLoads = D / 8;  // 16-byte chunks of two row tiles per row thread
    constexpr int kQStep = kRowWarps * 32 / (D / 8);
    uint4 qv[kQLoads];
    if (warp < kRowWarps) {
#pragma unroll
        for (int i = 0; i < kQLoads; ++i) {
            const int rr = r0 + threadIdx.x / (D / 8) + i * kQStep, t = node_of(rr);
            qv[i] = make_uint4(0u, 0u, 0u, 0u);
            if (rr < p.T * p.G)
                qv[i] = *reinterpret_cast<const uint4*>(
                    p.q + ((static_cast<int64_t>(b) * p.T + t) * p.Hq + hk * p.G + rr - t * p.G) * D +
                    threadIdx.x % (D / 8) * 8);
        }
    } else if (warp >= kLoadKWarp) {
        ids = block_ids(0);
    }
    if (!lengths_fit(p, tree, ctx)) {
        if (blockIdx.x == 0) {
            if (threadIdx.x == 0) atomicOr(p.err, KVC_DEVERR_CONTEXT);
            const int rows = min(max(tree, 0), p.T) * p.G;
            for (int e = threadIdx.x; e < rows * D; e += kThreads) {
                const int r = e / D;
                store_out(p.out, p.out_f32,
                          ((static_cast<int64_t>(b) * p.T + r / p.G) * p.Hq + hk * p.G + r % p.G) * D + e % D, 0.f);
            }
        }
        return;
    }
    const int rows = tree * p.G, all_tiles = key_tiles(ctx);
    if (r0 >= rows || clus * per_clus >= all_tiles) return;  // the whole cluster
    const int n = max(0, min(p.chunk, all_tiles - c0));  // key tiles of this CTA
    const bool two_rows = rows - r0 > kRows;             // two row tiles: they are the streams
    const int units = two_rows ? 2 * n : n;              // 64-key steps of each stream
    const int hist = ctx - tree;                         // keys before the tree
    const int pages = (ctx + kBlockSize - 1) / kBlockSize;
    const bool whole = all_tiles <= per_clus;            // one cluster covers the context: no partial states
    const uint32_t VS = two_rows ? Geo::kVStages : MVS;
    // unit u of stream x: key tile and half of the tile
    auto tile_of = [&](int u) { return two_rows ? u >> 1 : u; };
    auto half_of = [&](int u, int x) { return two_rows ? u & 1 : x; };

    auto qs = [&](int x) { return smem + Geo::kQOff + x * Geo::kTileBytes; };
    auto kst = [&](uint32_t st) { return smem + Geo::kKOff + st * Geo::kTileBytes; };
    uint8_t* const vring = smem + (two_rows ? Geo::kVOff : Geo::kVOff - Geo::kTileBytes);
    auto vst = [&](uint32_t st) { return vring + st * Geo::kTileBytes; };

    // The copy warps start as soon as the barriers are there; the others also need the tensor memory.
    uint32_t tmem = 0;
    if (warp >= kLoadKWarp) {
        if (warp == kLoadKWarp && lane == 0) {
            mbar_init(q_full, kRowWarps);
            for (int i = 0; i < KS; ++i) {
                mbar_init(&k_full[i], 1);
                mbar_init(&k_empty[i], 2);  // both streams' products
            }
            for (int i = 0; i < MVS; ++i) {
                mbar_init(&v_full[i], 1);
                mbar_init(&v_empty[i], 2);
            }
            for (int i = 0; i < 4; ++i) {
                mbar_init(&s_full[i], 1);
                mbar_init(&p_full[i], 4);
                mbar_init(&o_full[i], 1);
                mbar_init(&fin[i], 1);
            }
            mbar_init(&v_land[0], 1);
            mbar_init(&v_land[1], 1);
            *s_abort = 0;
            *s_bad_block = 0;
            *s_bad_v = 0;
            *s_bad_of = 0;
            fence_barrier_init();
        }
        __syncwarp();
        bar_sync(2, 64);  // the two copy warps
        bar_arrive(3, kThreads);
    } else {
        if (warp == 0) {
            tmem_alloc(s_tmem, Geo::kTmemCols);
            tmem_relinquish();
            tc_fence_before();
        }
        bar_sync(3, kThreads);
        tc_fence_after();
        tmem = *s_tmem;
    }

    if (warp >= kLoadKWarp) {
        // ====== copies: a warp for K and one for V, each as far ahead as its ring allows; lane i copies block i ======
        const bool is_v = warp == kLoadVWarp;
        // one pair of row tiles reads its K and V once; several pairs meet them in L2
        const uint64_t policy = p.row_pairs == 1 ? l2_policy_evict_first() : l2_policy_evict_normal();
        uint64_t* const full = is_v ? v_full : k_full;
        uint64_t* const empty = is_v ? v_empty : k_empty;
        const CUtensorMap* const map = is_v ? &tmV : &tmK;
        const uint32_t stages = is_v ? VS : KS;
        const int mend0 = min(n, max(0, hist / kKeys - c0));  // first tile that reaches into the tree; at most two do
        uint32_t st = 0, ph = 0;  // stage and use of tile j
        int issued = 0, ids_next = 0;
        bool ok = true;
        for (int j = 0; j < n; ++j) {
            if ((j & 3) == 0) {
                if (j > 0) ids = ids_next;
                if (j + 4 < n) ids_next = block_ids(j + 4);
            }
            const int np = min(kPages, pages - (c0 + j) * kPages);
            int phys = __shfl_sync(0xffffffffu, ids, (j & 3) * kPages + (lane & (kPages - 1)));
            if (lane < np && (phys < 0 || phys >= p.num_blocks)) {
                // flagged, and block 0 copied in its place; the chunk's values are then not used
                atomicOr(p.err, KVC_DEVERR_BLOCK_ID);
                *s_bad_block = 1;  // seen by the row warps behind this tile's barriers
                phys = 0;
            }
            if (ph > 0) ok = __all_sync(0xffffffffu, wait(&empty[st], (ph - 1) & 1, s_abort));
            if (!ok) break;
            // V tiles that reach into the tree are mended before the products may read them
            const bool mend = is_v && (c0 + j + 1) * kKeys > hist;
            uint64_t* const bar = mend ? &v_land[j - mend0] : &full[st];
            if (lane == 0) mbar_arrive_expect_tx(bar, np * (kBlockSize * D * 2));
            __syncwarp();
            if (lane < np) {
                uint8_t* tile = is_v ? vst(st) : kst(st);
#pragma unroll
                for (int c = 0; c < Geo::kChunks; ++c)
                    tma_load_2d(tile + c * Geo::kChunkBytes + lane * (kBlockSize * 128), map, bar, c * 64,
                                (phys * p.Hkv + hk) * kBlockSize, policy);
            }
            issued = j + 1;
            if (++st == stages) {
                st = 0;
                ++ph;
            }
        }
        if (!is_v) {
            // copies still in flight land before the shared memory is used otherwise or released (immediate unless
            // aborted: the products consumed every tile)
            if (lane == 0)
                for (int t = max(0, issued - KS); t < issued; ++t)
                    mbar_wait_bounded(&k_full[t % KS], (t / KS) & 1, kWaitNs / 8);
        } else {
            if (lane == 0) {
                for (int t = max(0, issued - static_cast<int>(VS)); t < min(issued, mend0); ++t)
                    mbar_wait_bounded(&v_full[t % VS], (t / VS) & 1, kWaitNs / 8);
                for (int t = mend0; t < issued; ++t) mbar_wait_bounded(&v_land[t - mend0], 0, kWaitNs / 8);
            }
            __syncwarp();
        }
        // V rows past the context are zeroed, so that whatever they hold cannot reach an output through a zero weight;
        // so are infinities and NaN among the tree's V rows, which not every row sees (the rows that do get them back
        // at the end).  Both copy warps work on it, the K warp's copies being done.
        for (int t = mend0; t < n; ++t) {
            if (ok) ok = __all_sync(0xffffffffu, wait(&v_land[t - mend0], 0, s_abort));
            if (ok) {
                uint8_t* vt = vst(t % VS);
                const int k0 = (c0 + t) * kKeys, from = max(hist - k0, 0), end = ctx - k0;
                bool found = false;
                constexpr int U = 4;
                for (int e0 = (warp - kLoadKWarp) * 32 + lane; e0 < (kKeys - from) * 8 * Geo::kChunks; e0 += 64 * U) {
                    uint4 v[U];
                    uint4* at[U];
#pragma unroll
                    for (int i = 0; i < U; ++i) {
                        const int e = e0 + i * 64, r = from + e / (8 * Geo::kChunks), rest = e % (8 * Geo::kChunks);
                        at[i] = reinterpret_cast<uint4*>(vt + (rest / 8) * Geo::kChunkBytes + sw128(r, rest % 8));
                        if (r >= kKeys) at[i] = nullptr;
                        v[i] = make_uint4(0u, 0u, 0u, 0u);
                        if (r < min(end, kKeys)) v[i] = *at[i];
                    }
#pragma unroll
                    for (int i = 0; i < U; ++i) {
                        if (at[i] == nullptr) continue;
                        bool bad = false;
                        *at[i] = make_uint4(finite_halves(v[i].x, bad), finite_halves(v[i].y, bad),
                                            finite_halves(v[i].z, bad), finite_halves(v[i].w, bad));
                        found = found || bad;
                    }
                }
                if (found) *s_bad_v = 1;
                fence_proxy_async_smem();  // visible to the tensor cores (async proxy)
            }
            __syncwarp();
            bar_sync(2, 64);
            if (is_v && lane == 0) mbar_arrive(&v_full[t % VS]);
        }
    } else if (warp >= kSWarp) {
        // ====== tensor-core products: a warp per stream for S and one for P V.  A warp waits as one, its elected lane
        // issues.  (One warp for all of them was bound by its own instruction stream: every wait is about 200 clocks
        // and every product about 40.) ======
        const int x = (warp - kSWarp) & 1;
        bool ok = true;
        uint32_t st = 0, ph = 0;  // stage and use of the unit's tile
        if (warp < kPvWarp) {
            // S of unit u = Q K^T over D / 16 steps of 16 dims (with one row tile both streams use Q_A), once the P of
            // unit u - 2 in the same buffer is consumed
            constexpr uint32_t idS = umma_idesc_f16(kRows, kHalf, 0, 0);
            const uint64_t dQ = umma_smem_desc(smem_u32(qs(two_rows ? x : 0)), 16, 1024);
            const uint64_t dK = umma_smem_desc(smem_u32(kst(0)), 16, 1024);
            if (n > 0) ok = wait_poll(q_full, 0, s_abort);
            for (int u = 0; ok && u < units; ++u) {
                const int buf = 2 * x + (u & 1);
                const bool last = !two_rows || (u & 1);  // the tile's last unit
                ok = wait_poll(&k_full[st], ph & 1, s_abort);
                if (ok && u >= 2) ok = wait_poll(&o_full[buf], ((u - 2) >> 1) & 1, s_abort);
                if (!ok) break;
                tc_fence_after();
                const uint64_t b0 = dK + static_cast<uint64_t>((st * Geo::kTileBytes + half_of(u, x) * kHalf * 128) >> 4);
                const uint32_t tS = tmem + buf * kHalf;
                if (elect_one()) {
#pragma unroll
                    for (int i = 0; i < D / 16; ++i) {
                        const int c = i >> 2, kk = i & 3;
                        umma_f16_ss(tS, dQ + ((c * Geo::kChunkBytes + kk * 32) >> 4),
                                    b0 + ((c * Geo::kChunkBytes + kk * 32) >> 4), idS, i > 0);
                    }
                    umma_commit(&s_full[buf]);
                    if (last) umma_commit(&k_empty[st]);
                }
                __syncwarp();
                if (last && ++st == KS) {
                    st = 0;
                    ++ph;
                }
            }
        } else {
            // O_X += P V of unit u: 4 steps of 16 keys, P from TMEM (fp16, or its high part and residual); V as the
            // MN-major B operand: 8-key groups 1024 bytes apart, 64-dim atoms one chunk apart
            constexpr uint32_t idPV = umma_idesc_f16(kRows, D, 0, 1);
            const uint64_t dV = umma_smem_desc(smem_u32(vring), Geo::kChunkBytes, 1024);
            const uint32_t tO = tmem + Geo::kTmemO + x * D;
            for (int u = 0; u < units; ++u) {
                const int buf = 2 * x + (u & 1);
                const bool last = !two_rows || (u & 1);
                ok = wait_poll(&v_full[st], ph & 1, s_abort) && wait_poll(&p_full[buf], (u >> 1) & 1, s_abort);
                if (!ok) break;
                tc_fence_after();
                const uint64_t v0 = dV + static_cast<uint64_t>((st * Geo::kTileBytes + half_of(u, x) * kHalf * 128) >> 4);
                const uint32_t tP = tmem + buf * kHalf;
                if (elect_one()) {
#pragma unroll
                    for (int kk = 0; kk < kHalf / 16; ++kk) {
                        const uint64_t bd = v0 + ((kk * 2048) >> 4);
                        umma_f16_ts(tO, tP + kk * 8, bd, idPV, (u > 0 || kk > 0) ? 1u : 0u);
                        if constexpr (kSplitP) umma_f16_ts(tO, tP + kHalf / 2 + kk * 8, bd, idPV, 1u);
                    }
                    umma_commit(&o_full[buf]);
                    if (last) umma_commit(&v_empty[st]);
                }
                __syncwarp();
                if (last && ++st == VS) {
                    st = 0;
                    ++ph;
                }
            }
        }
        // every product issued is complete before the tensor memory is released
        if (elect_one()) umma_commit(&fin[warp - kSWarp]);
        __syncwarp();
        mbar_wait_bounded(&fin[warp - kSWarp], 0, kWaitNs);
        if (!ok && lane == 0) atomicOr(p.err, KVC_DEVERR_TIMEOUT);
    } else {
        // ================= row warps: query rows, softmax; thread = query row = TMEM lane =================
        const int x = warp / 4, wq = warp & 3;
        const int row = wq * 32 + lane;
        {
            const uint32_t flip = p.negate ? 0x80008000u : 0u;
            const int c = threadIdx.x % (D / 8);
#pragma unroll
            for (int i = 0; i < kQLoads; ++i) {
                const int r = threadIdx.x / (D / 8) + i * kQStep;
                if (i < kQLoads / 2 || two_rows) {
                    const uint4 v = make_uint4(qv[i].x ^ flip, qv[i].y ^ flip, qv[i].z ^ flip, qv[i].w ^ flip);
                    *reinterpret_cast<uint4*>(qs(r / kRows) + (c / 8) * Geo::kChunkBytes + sw128(r % kRows, c % 8)) = v;
                }
            }
            fence_proxy_async_smem();  // visible to the tensor cores (async proxy)
            __syncwarp();
            if (lane == 0) mbar_arrive(q_full);
        }
        const int rr = r0 + (two_rows ? x * kRows : 0) + row;  // row of the (sequence, KV head)
        const bool live = rr < rows;
        const bool live_warp = __any_sync(0xffffffffu, live);
        const uint64_t tree_bits = tree >= 64 ? ~0ull : (1ull << tree) - 1;
        const uint64_t mask = live ? p.masks[static_cast<int64_t>(b) * p.T + node_of(rr)] & tree_bits : 0;
        const uint32_t lane_base = static_cast<uint32_t>(wq * 32) << 16;
        const uint32_t tO = tmem + Geo::kTmemO + x * D + lane_base;
        const float sl2 = p.scale_log2;
        const uint64_t sc2 = pack_f32x2(sl2, sl2);
        float m_used = -INFINITY, l = 0.f;
        bool far = false;  // some row of the warp has its m beyond kFar, or sees nothing yet
        bool ok = true;
        for (int u = 0; u < units; ++u) {
            const int buf = 2 * x + (u & 1);
            const uint32_t tS = tmem + buf * kHalf + lane_base;
            ok = __all_sync(0xffffffffu, wait(&s_full[buf], (u >> 1) & 1, s_abort));
            if (!ok) break;
            tc_fence_after();
            const int k0 = (c0 + tile_of(u)) * kKeys + half_of(u, x) * kHalf;  // the unit's first key
            const bool masked = k0 + kHalf > hist;  // it reaches into the tree or past the context
            if (live_warp) {
                float s[kHalf];
                tmem_ld64(tS, s);
                if (masked) {
                    // bit i of w = key i is seen: history keys all, tree keys by the row's mask
                    const int d = hist - k0;  // history keys from here on, below 64
                    const uint64_t w = (d > 0 ? (1ull << d) - 1 : 0ull) |
                                       (d >= 0 ? mask << d : d > -64 ? mask >> -d : 0ull);
                    const uint32_t w0 = static_cast<uint32_t>(w), w1 = static_cast<uint32_t>(w >> 32);
#pragma unroll
                    for (int c = 0; c < kHalf; ++c)
                        if (!(((c < 32 ? w0 : w1) >> (c & 31)) & 1u)) s[c] = -INFINITY;
                }
                float e[4];
#pragma unroll
                for (int i = 0; i < 4; ++i) e[i] = max3f(s[i], s[4 + i], s[8 + i]);
#pragma unroll
                for (int c = 12; c + 8 <= kHalf; c += 8)
#pragma unroll
                    for (int i = 0; i < 4; ++i) e[i] = max3f(e[i], s[c + i], s[c + 4 + i]);
#pragma unroll
                for (int i = 0; i < 4; ++i) e[i] = fmaxf(e[i], s[kHalf - 4 + i]);
                const float mx = __fmul_rd(max3f(e[0], e[1], fmaxf(e[2], e[3])), sl2);  // -inf: nothing seen
                float alpha = 1.f;
                if (mx > m_used + kRescaleLog2) {  // includes the first finite max (m_used = -inf)
                    const float m_new = __fsub_rd(mx, kWeightLog2);
                    alpha = m_used == -INFINITY ? 0.f : ex2(m_used - m_new);
                    m_used = m_new;
                }
                if (__any_sync(0xffffffffu, alpha != 1.f)) {
                    if constexpr (kSplitP) far = __any_sync(0xffffffffu, fabsf(m_used) >= kFar);
                    // rescale O_X, which idles once the stream's previous product is complete (this unit's P is not
                    // there yet)
                    if (u > 0) ok = __all_sync(0xffffffffu, wait(&o_full[buf ^ 1], ((u - 1) >> 1) & 1, s_abort));
                    if (!ok) break;
                    tc_fence_after();
#pragma unroll 1
                    for (int c = 0; u > 0 && c < D; c += 32) {
                        float o[32];
                        tmem_ld32(tO + c, o);
#pragma unroll
                        for (int i = 0; i < 32; ++i) o[i] *= alpha;
                        tmem_st32(tO + c, o);
                    }
                }
                const float neg_m = m_used == -INFINITY ? 0.f : -m_used;
                float ls[4] = {0.f, 0.f, 0.f, 0.f};
                uint64_t by2 = sc2, nm2 = pack_f32x2(neg_m, neg_m);
                if (kSplitP && far) {
#pragma unroll
                    for (int c = 0; c < kHalf; ++c) {
                        const float d = fmaf(s[c], sl2, neg_m);
                        s[c] = d > kRescaleLog2 ? kRescaleLog2 : d;
                    }
                    by2 = pack_f32x2(1.f, 1.f);
                    nm2 = 0;
                }
#pragma unroll
                for (int hh = 0; hh < 2; ++hh) {  // 32 keys at a time
                    uint32_t hv[16], lv[16];
#pragma unroll
                    for (int i = 0; i < 16; ++i) {
                        const int c = hh * 32 + 2 * i;
                        float x0, x1;
                        unpack_f32x2(fma_f32x2(pack_f32x2(s[c], s[c + 1]), by2, nm2), x0, x1);
                        x0 = ex2(x0);
                        x1 = ex2(x1);
                        hv[i] = kSplitP ? pack_half2(x0, x1) : pack_half2_finite(x0, x1);
                        if constexpr (kSplitP) {
                            const float2 f = unpack_half2(hv[i]);
                            lv[i] = pack_half2(x0 - f.x, x1 - f.y);
                            ls[i & 3] += x0 + x1;
                        } else {
                            ls[i & 3] = add_halves(hv[i], ls[i & 3]);
                        }
                    }
                    tmem_st16(tS + hh * 16, hv);
                    if constexpr (kSplitP) tmem_st16(tS + kHalf / 2 + hh * 16, lv);
                }
                l = l * alpha + ((ls[0] + ls[1]) + (ls[2] + ls[3]));
            }
            tmem_wait_st();
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(&p_full[buf]);
        }
        if (ok && units > 0)
            ok = __all_sync(0xffffffffu, wait(&o_full[2 * x + ((units - 1) & 1)], ((units - 1) >> 1) & 1, s_abort));
        tc_fence_after();
        row_warps_sync();  // both streams done: the rings are idle, the notes on bad blocks and values complete
        // the rows' states into the state area: slot x * 128 + row with two row tiles; with one the streams' states of
        // a row are merged first, each of its two threads for half of the columns
        const bool drop = *s_bad_block != 0 || *s_abort != 0 || units == 0;  // the same in every thread
        float2* const ml = reinterpret_cast<float2*>(smem + Geo::kMlOff);
        float* const states = reinterpret_cast<float*>(smem + Geo::kStateOff);
        ml[x * kRows + row] = drop ? make_float2(-INFINITY, 0.f) : make_float2(m_used, l);
        if (two_rows) {
            if (live_warp && !drop) {
                float* const mine = states + (x * kRows + row) * Geo::kOStride;
#pragma unroll
                for (int c = 0; c < D; c += 64) {
                    float o[64];
                    tmem_ld64(tO + c, o);
#pragma unroll
                    for (int i = 0; i < 64; i += 4)
                        *reinterpret_cast<float4*>(mine + c + i) = make_float4(o[i], o[i + 1], o[i + 2], o[i + 3]);
                }
            }
        } else {
            tc_fence_before();
            row_warps_sync();
            tc_fence_after();  // the other stream's accumulator
            const float2 sa = ml[row], sb = ml[kRows + row];
            const bool ha = sa.y != 0.f, hb = sb.y != 0.f;  // a state with sum 0 holds nothing
            const float m = fmaxf(ha ? sa.x : -INFINITY, hb ? sb.x : -INFINITY);
            const float wa = !ha ? 0.f : sa.x == m ? 1.f : ex2(sa.x - m);
            const float wb = !hb ? 0.f : sb.x == m ? 1.f : ex2(sb.x - m);
            row_warps_sync();
            if (x == 0) ml[row] = make_float2(m, (ha ? sa.y * wa : 0.f) + (hb ? sb.y * wb : 0.f));
            if (live_warp && !drop) {
                float* const mine = states + row * Geo::kOStride + x * (D / 2);
#pragma unroll
                for (int c = 0; c < D / 2; c += 32) {
                    float oa[32], ob[32];
                    tmem_ld32(tmem + Geo::kTmemO + lane_base + x * (D / 2) + c, oa);
                    tmem_ld32(tmem + Geo::kTmemO + D + lane_base + x * (D / 2) + c, ob);
#pragma unroll
                    for (int i = 0; i < 32; ++i) oa[i] = (ha ? oa[i] * wa : 0.f) + (hb ? ob[i] * wb : 0.f);
#pragma unroll
                    for (int i = 0; i < 32; i += 4)
                        *reinterpret_cast<float4*>(mine + c + i) = make_float4(oa[i], oa[i + 1], oa[i + 2], oa[i + 3]);
                }
            }
        }
    }
    // every TMEM access of the CTA is complete; the allocating warp frees it
    __syncwarp();
    tc_fence_before();
    __syncthreads();
    if (warp == 0) {
        tc_fence_after();
        tmem_dealloc(tmem, Geo::kTmemCols);
    }
    // ================= the cluster's states merged: each CTA takes a share of the rows =================
    const int live_rows = min(two_rows ? 2 * kRows : kRows, rows - r0);
    const int share = (live_rows + p.cluster - 1) / p.cluster;
    const int ra = min(rank * share, live_rows), nr = min(share, live_rows - ra);
    const int ncta = min(p.cluster, (all_tiles - clus * per_clus + p.chunk - 1) / p.chunk);  // CTAs with tiles
    auto out_row = [&](int rr) {
        const int t = node_of(rr);
        return (static_cast<int64_t>(b) * p.T + t) * p.Hq + hk * p.G + rr - t * p.G;
    };
    if (*s_bad_block != 0) *s_bad_v = 0;  // the chunk is left out
    if (p.cluster > 1) {
        __syncwarp();
        cluster_sync_all();  // every CTA's states are in its shared memory
    } else {
        __syncthreads();
    }
    // weights of a row's states, s_w[row][state] = (weight, sum): a group of `group` lanes takes a row, a lane a state
    float2* const s_w = reinterpret_cast<float2*>(smem + Geo::kWeightOff);
    {
        const uint32_t ml0 = smem_u32(smem + Geo::kMlOff), flag0 = smem_u32(const_cast<int*>(s_bad_v));
        int group = 1;
        while (group < ncta) group *= 2;
        const int s = threadIdx.x & (group - 1);
        for (int rbase = 0; rbase < nr; rbase += kThreads / group) {  // (group divides 32: whole warps)
            const int r = rbase + threadIdx.x / group;
            float2 st = make_float2(-INFINITY, 0.f);
            if (r < nr && s < ncta) st = ld_cluster_f32x2(cluster_addr(ml0, s) + (ra + r) * 8);
            float m = st.y != 0.f ? st.x : -INFINITY;  // a state with sum 0 holds nothing
            for (int off = group / 2; off > 0; off >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, off));
            const float w = st.y == 0.f ? 0.f : st.x == m ? 1.f : ex2(st.x - m);
            float l = st.y != 0.f ? st.y * w : 0.f;
            for (int off = group / 2; off > 0; off >>= 1) l += __shfl_xor_sync(0xffffffffu, l, off);
            const float inv = whole ? (l > 0.f || l != l ? 1.f / l : 0.f) : 1.f;
            if (r < nr && s < ncta) {
                s_w[r * ncta + s] = make_float2(w * inv, st.y);
                if (!whole && s == 0)
                    *reinterpret_cast<float2*>(p.part_ml + (out_row(r0 + ra + r) * p.nclus + clus) * 2) = make_float2(m, l);
            }
        }
        if (threadIdx.x < ncta && ld_cluster_u32(cluster_addr(flag0, threadIdx.x)) != 0)
            atomicOr(const_cast<int*>(s_bad_of), 1 << threadIdx.x);
    }
    __syncthreads();
    const uint32_t bad_of = static_cast<uint32_t>(*s_bad_of);
    // output rows: a thread per four columns; U items of S states are read at a time
    auto merge_rows = [&](auto u_items, auto s_states) {
        constexpr int U = decltype(u_items)::value, S = decltype(s_states)::value;
        constexpr int kCols = D / 4;
        const uint32_t state0 = smem_u32(smem + Geo::kStateOff);
        for (int e0 = threadIdx.x; e0 < nr * kCols; e0 += U * kThreads) {
            float4 o[U];
#pragma unroll
            for (int i = 0; i < U; ++i) o[i] = make_float4(0.f, 0.f, 0.f, 0.f);
            for (int s0 = 0; s0 < ncta; s0 += S) {
                float4 a[U][S];
#pragma unroll
                for (int j = 0; j < S; ++j) {
                    if (s0 + j >= ncta) break;
                    const uint32_t base = cluster_addr(state0, s0 + j) + ra * (Geo::kOStride * 4);
#pragma unroll
                    for (int i = 0; i < U; ++i) {
                        const int e = min(e0 + i * kThreads, nr * kCols - 1);
                        a[i][j] = ld_cluster_f32x4(base + (e / kCols * Geo::kOStride + e % kCols * 4) * 4);
                    }
                }
#pragma unroll
                for (int i = 0; i < U; ++i) {
                    const int r = min(e0 + i * kThreads, nr * kCols - 1) / kCols;
#pragma unroll
                    for (int j = 0; j < S; ++j) {
                        if (s0 + j >= ncta) break;
                        const float2 w = s_w[r * ncta + s0 + j];
                        if (w.y != 0.f) o[i] = fma4(w.x, a[i][j], o[i]);  // (O of a state that holds nothing: unwritten)
                    }
                }
            }
#pragma unroll
            for (int i = 0; i < U; ++i) {
                const int e = e0 + i * kThreads;
                if (e >= nr * kCols) break;
                const int rr = r0 + ra + e / kCols, c = e % kCols * 4;
                const int64_t orow = out_row(rr);
                if (bad_of != 0) {
                    // infinities and NaN of the tree's V rows that this row sees, in the noted CTAs' keys
                    const uint64_t mask = p.masks[static_cast<int64_t>(b) * p.T + node_of(rr)];
                    for (int t = 0; t < tree; ++t) {
                        const int pos = hist + t, q = pos / kKeys / p.chunk - clus * p.cluster;
                        if (!((mask >> t) & 1) || q < 0 || q >= ncta || !((bad_of >> q) & 1u)) continue;
                        const int64_t blk = table_row[pos / kBlockSize];
                        const __half* v = p.v_cache + ((blk * p.Hkv + hk) * kBlockSize + pos % kBlockSize) * D + c;
                        const float y[4] = {__half2float(v[0]), __half2float(v[1]), __half2float(v[2]),
                                            __half2float(v[3])};
                        if (!(fabsf(y[0]) < INFINITY)) o[i].x += y[0];
                        if (!(fabsf(y[1]) < INFINITY)) o[i].y += y[1];
                        if (!(fabsf(y[2]) < INFINITY)) o[i].z += y[2];
                        if (!(fabsf(y[3]) < INFINITY)) o[i].w += y[3];
                    }
                }
                if (whole)
                    store_out4(p.out, p.out_f32, orow * D + c, o[i]);
                else
                    *reinterpret_cast<float4*>(p.part_acc + (orow * p.nclus + clus) * D + c) = o[i];
            }
        }
    };
    if (ncta <= 2)
        merge_rows(std::integral_constant<int, 4>(), std::integral_constant<int, 2>());
    else if (ncta <= 4)
        merge_rows(std::integral_constant<int, 2>(), std::integral_constant<int, 4>());
    else
        merge_rows(std::integral_constant<int, 1>(), std::integral_constant<int, 8>());
    if (p.cluster > 1) {
        __syncwarp();
        cluster_sync_all();  // no CTA leaves while another reads its shared memory
    }
}

// Partial states of the chunks merged: a warp per (32 / (D / 4)) output rows, a lane per four columns.
constexpr int kCombineWarps = 8;

template <int D>
__global__ void __launch_bounds__(kCombineWarps * 32) tree_combine_kernel(const Params p, int64_t nrows) {
    constexpr int kLanes = D / 4, kPer = 32 / kLanes;
    grid_dependency_wait();
    const int lane = threadIdx.x & 31;
    const int64_t row = (static_cast<int64_t>(blockIdx.x) * kCombineWarps + (threadIdx.x >> 5)) * kPer + lane / kLanes;
    if (row >= nrows) return;
    const int c = (lane % kLanes) * 4;
    const int64_t bt = row / p.Hq;
    const int b = static_cast<int>(bt / p.T), t = static_cast<int>(bt % p.T);
    const int tree = p.tree_lens != nullptr ? p.tree_lens[b] : p.T, ctx = p.context_lens[b];
    if (!lengths_fit(p, tree, ctx) || t >= tree) return;
    const int per_clus = p.chunk * p.cluster, nclus = (key_tiles(ctx) + per_clus - 1) / per_clus;
    if (nclus <= 1) return;  // the attention kernel wrote the row
    float m = -INFINITY, l = 0.f;
    float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 4
    for (int s = 0; s < nclus; ++s) {
        const int64_t at = row * p.nclus + s;
        const float2 ml = *reinterpret_cast<const float2*>(p.part_ml + at * 2);
        const float4 a = *reinterpret_cast<const float4*>(p.part_acc + at * D + c);
        if (ml.y == 0.f) continue;  // the row saw none of the part's keys
        const float mn = fmaxf(m, ml.x);
        const float f_old = m == mn ? 1.f : ex2(m - mn), f_new = ml.x == mn ? 1.f : ex2(ml.x - mn);
        o = fma4(f_new, a, scale4(o, f_old));
        l = l * f_old + ml.y * f_new;
        m = mn;
    }
    store_out4(p.out, p.out_f32, row * D + c, scale4(o, l > 0.f || l != l ? 1.f / l : 0.f));
}

}  // namespace tree

// What a split of the contexts costs, in units of 0.01 us, by [D = 128][two row tiles]: a CTA's start and end, a key
// tile, and a merge in a cluster.  Fitted to 56 shapes (1 to 128 sequences, 1 to 65,536 keys, every head layout of the
// tests) measured with every split: the split chosen is 0.5 % slower than the best one on average, 5 % at worst.
constexpr int kCtaCost[2][2] = {{480, 580}, {680, 1000}};
constexpr int kTileCost[2][2] = {{70, 130}, {100, 135}};
constexpr int kMergeCost[2][2] = {{60, 200}, {30, 30}};
constexpr int kMergeCtaCost = 5;     // per CTA of the cluster
constexpr int kCombineCost = 300;    // the second launch
constexpr int kStateCost = 35;       // a partial state of a row: they are read one after another
constexpr int kPartialCost = 100;    // per partial state and unit, over the SMs

template <int D, bool kSplitP>
static cudaError_t tree_setup() {
    static std::atomic<bool> done[128];  // by device
    int dev = 0;
    cudaError_t err = cudaGetDevice(&dev);
    if (err != cudaSuccess) return err;
    const bool kept = dev >= 0 && dev < 128;
    if (kept && done[dev].load(std::memory_order_relaxed)) return cudaSuccess;
    err = cudaFuncSetAttribute(tree::paged_decode_tree_kernel<D, kSplitP>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                               tree::Geom<D>::kSmemBytes);
    if (err == cudaSuccess && kept) done[dev].store(true, std::memory_order_relaxed);
    return err;
}

// Clusters of cs CTAs (one per SM) that the device holds at a time; the SMs of a GPC that no whole cluster fills stay
// idle.  Asked once per device and size.
static int resident_clusters(int dev, int D, int cs, int sms) {
    static std::atomic<int> cache[128][2][tree::kMaxTreeCluster + 1];
    if (cs == 1) return sms;
    if (dev < 0 || dev >= 128) return std::max(1, sms / cs);
    std::atomic<int>& slot = cache[dev][D == 128][cs];
    int n = slot.load(std::memory_order_relaxed);
    if (n > 0) return n;
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute attr;
    attr.id = cudaLaunchAttributeClusterDimension;
    attr.val.clusterDim.x = cs;
    attr.val.clusterDim.y = attr.val.clusterDim.z = 1;
    cfg.gridDim = dim3(cs);
    cfg.blockDim = dim3(tree::kThreads);
    cfg.attrs = &attr;
    cfg.numAttrs = 1;
    cudaError_t e;
    if (D == 64) {
        cfg.dynamicSmemBytes = tree::Geom<64>::kSmemBytes;
        e = tree_setup<64, false>();
        if (e == cudaSuccess) e = cudaOccupancyMaxActiveClusters(&n, tree::paged_decode_tree_kernel<64, false>, &cfg);
    } else {
        cfg.dynamicSmemBytes = tree::Geom<128>::kSmemBytes;
        e = tree_setup<128, false>();
        if (e == cudaSuccess) e = cudaOccupancyMaxActiveClusters(&n, tree::paged_decode_tree_kernel<128, false>, &cfg);
    }
    if (e != cudaSuccess || n < 1) {
        cudaGetLastError();
        n = std::max(1, sms / cs);
    }
    slot.store(n, std::memory_order_relaxed);
    return n;
}

cudaError_t tree_plan(int B, int Hq, int Hkv, int D, int max_ctx, int T, TreePlan* plan) {
    const int sms = sm_count();
    int dev = 0;
    if (sms <= 0 || cudaGetDevice(&dev) != cudaSuccess) return cudaErrorNoDevice;
    if (D != 64 && D != 128) return cudaErrorInvalidValue;
    const int G = Hq / Hkv;
    const int row_tiles = (T * G + tree::kRows - 1) / tree::kRows;
    plan->row_pairs = (row_tiles + 1) / 2;
    const int tiles = std::max(1, (max_ctx + tree::kKeys - 1) / tree::kKeys);
    const int64_t units = std::max<int64_t>(1, static_cast<int64_t>(B) * Hkv * plan->row_pairs);
    const int d = D == 128, two = row_tiles > 1;
    // The split with the shortest run: waves of clusters times a CTA's tiles, start and end; then the merges.  The
    // clusters are of 1, 2, 4 or 8 CTAs, or of all chunks of a context.
    const int cta = kCtaCost[d][two], tile = kTileCost[d][two], merge = kMergeCost[d][two];
    const uint32_t all = static_cast<uint32_t>(std::min<int64_t>(units, 1 << 30));
    int64_t best_cost = INT64_MAX;
    // numbers of chunks in turn that chunks of one size divide a context into
    for (int chunk = tiles, nc = 1;;) {
        for (int cs = nc <= tree::kMaxTreeCluster ? nc : tree::kMaxTreeCluster; cs > 0;) {
            const uint32_t nclus = static_cast<uint32_t>(nc + cs - 1) / cs;  // (all * nclus: below 8 * SMs + all)
            const uint32_t resident = static_cast<uint32_t>(resident_clusters(dev, D, cs, sms));
            const int64_t waves = (all * nclus + resident - 1) / resident;
            int64_t cost = waves * (cta + static_cast<int64_t>(chunk) * tile);
            if (cs > 1) cost += merge + kMergeCtaCost * cs;
            if (nclus > 1) cost += kCombineCost + kStateCost * nclus + kPartialCost * nclus * all / sms;
            if (cost < best_cost) {
                best_cost = cost;
                plan->chunk = chunk;
                plan->cluster = cs;
                plan->nclus = static_cast<int>(nclus);
            }
            cs = cs > 4 ? 4 : cs > 2 ? 2 : cs > 1 ? 1 : 0;  // all of up to eight, then 4, 2, 1
        }
        if (units * nc > 8 * sms || chunk == 1) break;  // every SM has its share: more chunks only cost
        nc = (tiles + chunk - 2) / (chunk - 1);         // the next number with smaller chunks
        chunk = (tiles + nc - 1) / nc;
        if (nc > 128) break;
    }
    plan->workspace_bytes = plan->nclus > 1 ? partials_bytes(static_cast<size_t>(B) * T * Hq * plan->nclus, D) : 0;
    return cudaSuccess;
}

template <int D, bool kSplitP>
static cudaError_t launch_tree_d(const TreeArgs& a, const TreePlan& plan, cudaStream_t stream) {
    using Geo = tree::Geom<D>;
    cudaError_t e = tree_setup<D, kSplitP>();
    if (e != cudaSuccess) return e;
    const int64_t rows = static_cast<int64_t>(a.num_blocks) * a.Hkv * kBlockSize;
    CUtensorMap tmK, tmV;
    e = make_tile_map(&tmK, a.k_cache, D, rows);
    if (e == cudaSuccess) e = make_tile_map(&tmV, a.v_cache, D, rows);
    if (e != cudaSuccess) return e;
    const size_t nrow = static_cast<size_t>(a.B) * a.T * a.Hq * plan.nclus;
    tree::Params p;
    p.q = a.q;
    p.block_table = a.block_table;
    p.context_lens = a.context_lens;
    p.tree_lens = a.tree_lens;
    p.masks = a.masks;
    p.v_cache = a.v_cache;
    p.out = a.out;
    p.part_ml = static_cast<float*>(a.workspace);
    p.part_acc = plan.nclus > 1 ? partials_acc(p.part_ml, nrow) : nullptr;
    p.err = a.err;
    p.T = a.T;
    p.Hq = a.Hq;
    p.Hkv = a.Hkv;
    p.G = a.Hq / a.Hkv;
    p.g_magic = ((1u << 18) + p.G - 1) / p.G;
    p.max_blocks = a.max_blocks;
    p.num_blocks = a.num_blocks;
    p.max_ctx = a.max_context_len;
    p.out_f32 = a.out_f32;
    p.chunk = plan.chunk;
    p.cluster = plan.cluster;
    p.nclus = plan.nclus;
    p.row_pairs = plan.row_pairs;
    p.negate = a.scale < 0.f;
    p.scale_log2 = std::min(std::max(std::fabs(a.scale) * kLog2e, tree::kMinScaleLog2), FLT_MAX);
    const dim3 grid(static_cast<unsigned>(plan.row_pairs * plan.nclus * plan.cluster), a.Hkv, a.B);
    e = launch(tree::paged_decode_tree_kernel<D, kSplitP>, grid, dim3(tree::kThreads), Geo::kSmemBytes, stream, true,
               static_cast<unsigned>(plan.cluster), tmK, tmV, p);
    if (e != cudaSuccess || plan.nclus == 1) return e;
    const int64_t nrows = static_cast<int64_t>(a.B) * a.T * a.Hq;
    constexpr int per_cta = tree::kCombineWarps * 128 / D;
    return launch(tree::tree_combine_kernel<D>, dim3(static_cast<unsigned>((nrows + per_cta - 1) / per_cta)),
                  dim3(tree::kCombineWarps * 32), 0, stream, true, 1u, p, nrows);
}

cudaError_t launch_tree(const TreeArgs& a, cudaStream_t stream) {
    TreePlan plan;
    cudaError_t e = tree_plan(a.B, a.Hq, a.Hkv, a.D, a.max_context_len, a.T, &plan);
    if (e != cudaSuccess) return e;
    if (plan.workspace_bytes > a.workspace_bytes) return cudaErrorInvalidValue;
    switch (a.D * 2 + (a.out_f32 ? 1 : 0)) {
        case 128: return launch_tree_d<64, false>(a, plan, stream);
        case 129: return launch_tree_d<64, true>(a, plan, stream);
        case 256: return launch_tree_d<128, false>(a, plan, stream);
        case 257: return launch_tree_d<128, true>(a, plan, stream);
        default: return cudaErrorInvalidValue;
    }
}

}  // namespace kvc
