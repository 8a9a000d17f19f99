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
// side in tiles of 128 (8 cache blocks).  A CTA works on two streams A and B of (row tile, key tile) pairs, each with
// four row warps, its scores / weights and its output accumulator in TMEM:
//   two row tiles     the streams are the row tiles and share every K/V tile (the tile is read once for 256 rows);
//   one row tile      the streams are the even and the odd key tiles of the same rows, merged at the end, so that one
//                     stream's softmax runs while the tensor cores work for the other.
// Per stream X and tile:  S_X = Q_X K^T (both K-major in shared memory, 128-byte swizzle, as TMA writes the blocks);
// the row warps take S_X from TMEM, keep the running max lazily (it moves when it has grown by 2^8; O_X is then
// rescaled in TMEM) and write P_X over S_X in fp16;  O_X += P_X V with P_X from TMEM and V MN-major.
// P.  With an fp16 output the weights are one fp16 value and the row sums add the rounded weights, so a row is a
// convex combination of V rows with weights within 2^-11 relative, which is the output's own rounding; with an fp32
// output they are an fp16 high part plus residual (two products), ~22 bits.
// The context is cut into chunks where (sequence, KV head, row tile pair) units are fewer than SMs; a chunk's state
// (max, sum, O) goes through the workspace to the combine kernel below.
// Lane 0 of warp 8 issues the products, warp 9 the copies (lane i the block i of a tile).  Every wait is bounded.
#include <algorithm>

#include "../../include/kvc.h"
#include "decode_common.cuh"
#include "kvc_internal.h"
#include "ptx.cuh"
#include "tcgen05.cuh"

namespace kvc {
namespace tree {

constexpr int kRows = 128;  // rows of a row tile
constexpr int kKeys = 128;  // keys of a key tile
constexpr int kPages = kKeys / kBlockSize;
constexpr int kRowWarps = 8;
constexpr int kMmaWarp = kRowWarps;
constexpr int kLoadKWarp = kRowWarps + 1;
constexpr int kLoadVWarp = kRowWarps + 2;
constexpr int kThreads = (kRowWarps + 3) * 32;
constexpr int kMaxTreeCluster = 8;
constexpr uint64_t kWaitNs = 1000000000ull;
// a scale of 0 is taken as this: the scores of fp16 rows (below 2^40) still vanish next to 1, and a masked score of
// -inf times it stays -inf
constexpr float kMinScaleLog2 = 0x1p-100f;
constexpr float kRescaleLog2 = 8.f;  // P stays below 2^8, far inside fp16

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
    static_assert(kMlOff + 2 * kRows * 8 <= kBarOff, "state area");
    // TMEM columns: S_A / P_A [0, 128), S_B / P_B [128, 256), O_A [256, 256 + D), O_B [256 + D, 256 + 2D)
    static constexpr int kTmemO = 2 * kKeys;
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
    int negate;      // scale < 0: the query rows change sign as they are loaded
    float scale_log2;  // |scale| * log2 e, at least kMinScaleLog2
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

// Sizes of sequence b; false where its lengths do not fit (tree_len and ctx stay as read).
__device__ __forceinline__ bool lengths(const Params& p, int b, int& tree, int& ctx) {
    tree = p.tree_lens != nullptr ? p.tree_lens[b] : p.T;
    ctx = p.context_lens[b];
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
    uint64_t* s_full = v_empty + MVS;        // [2] S_X of the stream's tile in TMEM
    uint64_t* p_full = s_full + 2;           // [2] P_X of the stream's tile in TMEM (4 arrivals)
    uint64_t* o_full = p_full + 2;           // [2] P_X V of the stream's tile done
    uint64_t* fin = o_full + 2;              // every MMA issued so far done
    uint32_t* s_tmem = reinterpret_cast<uint32_t*>(fin + 1);
    volatile int* s_abort = reinterpret_cast<volatile int*>(s_tmem + 1);
    volatile int* s_bad_block = s_abort + 1;  // a block id out of range: the chunk is left out
    volatile int* s_bad_v = s_abort + 2;      // an infinity or NaN among the tree's V values
    static_assert((1 + 2 * KS + 2 * MVS + 7) * 8 + 16 <= 512, "barrier area");

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    // blockIdx.x = (cluster along the context * row pairs + row pair) * CTAs per cluster + rank
    const int rank = static_cast<int>(blockIdx.x) % p.cluster;
    const int pair = static_cast<int>(blockIdx.x) / p.cluster % p.row_pairs;
    const int clus = static_cast<int>(blockIdx.x) / p.cluster / p.row_pairs;
    const int hk = blockIdx.y, b = blockIdx.z;
    int tree, ctx;
    if (!lengths(p, b, tree, ctx)) {
        if (blockIdx.x == 0) {
            if (threadIdx.x == 0) atomicOr(p.err, KVC_DEVERR_CONTEXT);
            const int rows = min(max(tree, 0), p.T);
            for (int e = threadIdx.x; e < rows * p.G * D; e += kThreads) {
                const int r = e / D;
                store_out(p.out, p.out_f32,
                          ((static_cast<int64_t>(b) * p.T + r / p.G) * p.Hq + hk * p.G + r % p.G) * D + e % D, 0.f);
            }
        }
        return;
    }
    const int rows = tree * p.G, r0 = pair * 2 * kRows;
    const int all_tiles = key_tiles(ctx), per_clus = p.chunk * p.cluster;
    if (r0 >= rows || clus * per_clus >= all_tiles) return;  // the whole cluster
    const int c0 = clus * per_clus + rank * p.chunk;
    const int n = max(0, min(p.chunk, all_tiles - c0));  // key tiles of this CTA
    const bool two_rows = rows - r0 > kRows;             // two row tiles: they are the streams
    const int step = two_rows ? 1 : 2;                   // key tiles between two of a stream's
    const int hist = ctx - tree;                         // keys before the tree
    const int pages = (ctx + kBlockSize - 1) / kBlockSize;
    const bool whole = all_tiles <= per_clus;            // one cluster covers the context: no partial states
    const uint32_t VS = two_rows ? Geo::kVStages : MVS;

    auto qs = [&](int x) { return smem + Geo::kQOff + x * Geo::kTileBytes; };
    auto kst = [&](uint32_t st) { return smem + Geo::kKOff + st * Geo::kTileBytes; };
    uint8_t* const vring = smem + (two_rows ? Geo::kVOff : Geo::kVOff - Geo::kTileBytes);
    auto vst = [&](uint32_t st) { return vring + st * Geo::kTileBytes; };

    // Copies of key tile j: lane i of the calling warp takes block i.
    const int32_t* const table_row = p.block_table + static_cast<int64_t>(b) * p.max_blocks;
    auto block_of = [&](int j) {
        const int page = (c0 + j) * kPages + lane;
        return lane < kPages && page < pages ? table_row[page] : 0;
    };
    // a block id out of range is flagged and block 0 copied in its place; the chunk's values are then not used
    auto checked_block = [&](int phys) {
        if (phys >= 0 && phys < p.num_blocks) return phys;
        atomicOr(p.err, KVC_DEVERR_BLOCK_ID);
        *s_bad_block = 1;  // seen by the row warps behind this tile's barriers
        return 0;
    };
    auto load = [&](uint8_t* tile, const CUtensorMap* map, uint64_t* bar, int j, int phys, uint64_t policy) {
        const int np = min(kPages, pages - (c0 + j) * kPages);
        if (lane == 0) mbar_arrive_expect_tx(bar, np * (kBlockSize * D * 2));
        __syncwarp();
        if (lane < np) {
#pragma unroll
            for (int c = 0; c < Geo::kChunks; ++c)
                tma_load_2d(tile + c * Geo::kChunkBytes + lane * (kBlockSize * 128), map, bar, c * 64,
                            (phys * p.Hkv + hk) * kBlockSize, policy);
        }
    };
    // one pair of row tiles reads its K and V once; several pairs meet them in L2
    uint64_t policy = 0;
    const int pre = min(n, Geo::kVStages);  // tiles whose copies start before the CTA's other preparations
    if (warp == kLoadKWarp) {
        if (lane == 0) {
            mbar_init(q_full, kRowWarps);
            for (int i = 0; i < KS; ++i) {
                mbar_init(&k_full[i], 1);
                mbar_init(&k_empty[i], 1);
            }
            for (int i = 0; i < MVS; ++i) {
                mbar_init(&v_full[i], 1);
                mbar_init(&v_empty[i], 1);
            }
            for (int x = 0; x < 2; ++x) {
                mbar_init(&s_full[x], 1);
                mbar_init(&p_full[x], 4);
                mbar_init(&o_full[x], 1);
            }
            mbar_init(fin, 1);
            *s_abort = 0;
            *s_bad_block = 0;
            *s_bad_v = 0;
            fence_barrier_init();
        }
        __syncwarp();
        policy = p.row_pairs == 1 ? l2_policy_evict_first() : l2_policy_evict_normal();
        static_assert(Geo::kVStages <= KS, "the first copies find every stage free");
        for (int j = 0; j < pre; ++j) {
            const int phys = checked_block(block_of(j));
            load(kst(j), &tmK, &k_full[j], j, phys, policy);
            load(vst(j), &tmV, &v_full[j], j, phys, policy);
        }
    }
    if (warp == 0) {
        tmem_alloc(s_tmem, Geo::kTmemCols);
        tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *s_tmem;

    if (warp == kLoadKWarp || warp == kLoadVWarp) {
        // ================= copies: a warp for K and one for V, each as far ahead as its ring allows =================
        const bool is_v = warp == kLoadVWarp;
        if (is_v) policy = p.row_pairs == 1 ? l2_policy_evict_first() : l2_policy_evict_normal();
        uint64_t* const full = is_v ? v_full : k_full;
        uint64_t* const empty = is_v ? v_empty : k_empty;
        const uint32_t stages = is_v ? VS : KS;
        uint32_t st = static_cast<uint32_t>(pre) % stages, ph = static_cast<uint32_t>(pre) / stages;  // of tile j
        int issued = pre;
        bool ok = true;
        int next = pre < n ? block_of(pre) : 0;
        for (int j = pre; j < n; ++j) {
            const int phys = checked_block(next);
            if (j + 1 < n) next = block_of(j + 1);
            if (ph > 0) ok = __all_sync(0xffffffffu, wait(&empty[st], (ph - 1) & 1, s_abort));
            if (!ok) break;
            load(is_v ? vst(st) : kst(st), is_v ? &tmV : &tmK, &full[st], j, phys, policy);
            issued = j + 1;
            if (++st == stages) {
                st = 0;
                ++ph;
            }
        }
        // copies still in flight land before the shared memory is used otherwise or released (immediate unless
        // aborted: the products consumed every tile)
        if (lane == 0)
            for (int t = max(0, issued - static_cast<int>(stages)); t < issued; ++t)
                mbar_wait_bounded(&full[t % stages], (t / stages) & 1, kWaitNs / 8);
    } else if (warp == kMmaWarp) {
        // ================= tensor-core products (one thread) =================
        if (lane == 0) {
            constexpr uint32_t idS = umma_idesc_f16(kRows, kKeys, 0, 0);
            constexpr uint32_t idPV = umma_idesc_f16(kRows, D, 0, 1);
            const uint64_t dQ = umma_smem_desc(smem_u32(qs(0)), 16, 1024);
            const uint64_t dK = umma_smem_desc(smem_u32(kst(0)), 16, 1024);
            // V as the MN-major B operand: 8-key groups 1024 bytes apart, 64-dim atoms one chunk apart
            const uint64_t dV = umma_smem_desc(smem_u32(vring), Geo::kChunkBytes, 1024);
            // S_X = Q_X K^T over D / 16 steps of 16 dims (with one row tile both streams use it)
            auto mma_s = [&](int x, uint32_t st) {
                const uint64_t a0 = dQ + static_cast<uint64_t>(two_rows ? x * (Geo::kTileBytes >> 4) : 0);
                const uint64_t b0 = dK + static_cast<uint64_t>(st * (Geo::kTileBytes >> 4));
#pragma unroll
                for (int ks = 0; ks < D / 16; ++ks) {
                    const int c = ks >> 2, kk = ks & 3;
                    umma_f16_ss(tmem + x * kKeys, a0 + ((c * Geo::kChunkBytes + kk * 32) >> 4),
                                b0 + ((c * Geo::kChunkBytes + kk * 32) >> 4), idS, ks > 0);
                }
                umma_commit(&s_full[x]);
            };
            // O_X += P_X V: 8 steps of 16 keys, P from TMEM (fp16, or its high part and residual)
            auto mma_pv = [&](int x, uint32_t st, bool first) {
                const uint64_t v0 = dV + static_cast<uint64_t>(st * (Geo::kTileBytes >> 4));
                const uint32_t tP = tmem + x * kKeys, tO = tmem + Geo::kTmemO + x * D;
#pragma unroll
                for (int kk = 0; kk < kKeys / 16; ++kk) {
                    const uint64_t bd = v0 + ((kk * 2048) >> 4);
                    umma_f16_ts(tO, tP + kk * 8, bd, idPV, (!first || kk > 0) ? 1u : 0u);
                    if constexpr (kSplitP) umma_f16_ts(tO, tP + 64 + kk * 8, bd, idPV, 1u);
                }
                umma_commit(&o_full[x]);
            };
            bool ok = n == 0 || wait(q_full, 0, s_abort);
            // the first tile of each stream: tile 0 for both, or tiles 0 and 1
            for (int x = 0; ok && x < 2; ++x) {
                const int j = two_rows ? 0 : x;
                if (j >= n) break;
                if (!(ok = wait(&k_full[j], 0, s_abort))) break;
                tc_fence_after();
                mma_s(x, j);
                if (!two_rows || x == 1) umma_commit(&k_empty[j]);
            }
            uint32_t vs = 0, vph = 0;                                                    // V stage and phase of tile j
            uint32_t ks = static_cast<uint32_t>(step) % KS, kph = static_cast<uint32_t>(step) / KS;  // K: of tile j + step
            for (int j = 0; ok && j < n; ++j) {
                if (!(ok = wait(&v_full[vs], vph & 1, s_abort))) break;
                const int jn = j + step;
                const uint32_t it = static_cast<uint32_t>(two_rows ? j : j >> 1);  // the streams' tile count
                // per stream of this tile: P_X V once P_X is in TMEM; then the stream's next S_X into the same
                // columns once that product has read P_X
                for (int x = two_rows ? 0 : (j & 1), left = two_rows ? 2 : 1; ok && left > 0; ++x, --left) {
                    if (!(ok = wait(&p_full[x], it & 1, s_abort))) break;
                    tc_fence_after();
                    mma_pv(x, vs, it == 0);
                    if (jn < n) {
                        if (!(ok = wait(&k_full[ks], kph & 1, s_abort))) break;
                        if (!(ok = wait(&o_full[x], it & 1, s_abort))) break;
                        tc_fence_after();
                        mma_s(x, ks);
                    }
                }
                if (!ok) break;
                umma_commit(&v_empty[vs]);
                if (jn < n) umma_commit(&k_empty[ks]);
                if (++vs == VS) {
                    vs = 0;
                    ++vph;
                }
                if (++ks == KS) {
                    ks = 0;
                    ++kph;
                }
            }
            // every product issued is complete before the tensor memory is released
            umma_commit(fin);
            mbar_wait_bounded(fin, 0, kWaitNs);
            if (!ok) atomicOr(p.err, KVC_DEVERR_TIMEOUT);
        }
    } else {
        // ================= row warps: query rows, softmax, output; thread = query row = TMEM lane =================
        const int x = warp / 4, wq = warp & 3;
        const int row = wq * 32 + lane;
        {
            const int nrows = two_rows ? 2 * kRows : kRows;
            const uint32_t flip = p.negate ? 0x80008000u : 0u;
            for (int e = threadIdx.x; e < nrows * (D / 8); e += kRowWarps * 32) {
                const int r = e / (D / 8), c = e % (D / 8), rr = r0 + r;
                uint4 v = make_uint4(0u, 0u, 0u, 0u);
                if (rr < rows) {
                    const int64_t at =
                        ((static_cast<int64_t>(b) * p.T + rr / p.G) * p.Hq + hk * p.G + rr % p.G) * D + c * 8;
                    v = *reinterpret_cast<const uint4*>(p.q + at);
                    v = make_uint4(v.x ^ flip, v.y ^ flip, v.z ^ flip, v.w ^ flip);
                }
                *reinterpret_cast<uint4*>(qs(r / kRows) + (c / 8) * Geo::kChunkBytes + sw128(r % kRows, c % 8)) = v;
            }
            fence_proxy_async_smem();  // visible to the tensor cores (async proxy)
            __syncwarp();
            if (lane == 0) mbar_arrive(q_full);
        }
        const int rr = r0 + (two_rows ? x * kRows : 0) + row;  // row of the (sequence, KV head)
        const bool live = rr < rows;
        const bool live_warp = __any_sync(0xffffffffu, live);
        const uint64_t tree_bits = tree >= 64 ? ~0ull : (1ull << tree) - 1;
        const uint64_t mask = live ? p.masks[static_cast<int64_t>(b) * p.T + rr / p.G] & tree_bits : 0;
        const uint32_t lane_base = static_cast<uint32_t>(wq * 32) << 16;
        const uint32_t tS = tmem + x * kKeys + lane_base, tO = tmem + Geo::kTmemO + x * D + lane_base;
        const float sl2 = p.scale_log2;
        float m_used = -INFINITY, l = 0.f;
        bool ok = true;
        int it = 0;
        uint32_t vs = two_rows ? 0u : static_cast<uint32_t>(x), vph = 0;  // V stage and phase of tile j
        for (int j = two_rows ? 0 : x; j < n; j += step, ++it) {
            // S_X complete also means the stream's previous P_X V complete: it was waited for before S_X was issued
            ok = __all_sync(0xffffffffu, wait(&s_full[x], it & 1, s_abort));
            if (!ok) break;
            tc_fence_after();
            const int k0 = (c0 + j) * kKeys;
            const bool masked = k0 + kKeys > hist;  // the tile reaches into the tree or past the context
            if (live_warp) {
                float s[kKeys];
                tmem_ld64(tS, reinterpret_cast<float(&)[64]>(s[0]));
                tmem_ld64(tS + 64, reinterpret_cast<float(&)[64]>(s[64]));
                if (masked) {
                    // per 64 keys: bit i of w = key i is seen; history keys all, tree keys by the row's mask
#pragma unroll
                    for (int hh = 0; hh < 2; ++hh) {
                        const int d = hist - (k0 + hh * 64);  // history keys from here on
                        const uint64_t old = d >= 64 ? ~0ull : d > 0 ? (1ull << d) - 1 : 0ull;
                        const uint64_t tr = d >= 64 ? 0ull : d >= 0 ? mask << d : d > -64 ? mask >> -d : 0ull;
                        const uint64_t w = old | tr;
                        const uint32_t w0 = static_cast<uint32_t>(w), w1 = static_cast<uint32_t>(w >> 32);
#pragma unroll
                        for (int c = 0; c < 64; ++c)
                            if (!(((c < 32 ? w0 : w1) >> (c & 31)) & 1u)) s[hh * 64 + c] = -INFINITY;
                    }
                }
                float e[4];
#pragma unroll
                for (int i = 0; i < 4; ++i) e[i] = max3f(s[i], s[4 + i], s[8 + i]);
#pragma unroll
                for (int c = 12; c + 8 <= kKeys; c += 8)
#pragma unroll
                    for (int i = 0; i < 4; ++i) e[i] = max3f(e[i], s[c + i], s[c + 4 + i]);
#pragma unroll
                for (int i = 0; i < 4; ++i) e[i] = fmaxf(e[i], s[kKeys - 4 + i]);
                const float ext = fmaxf(fmaxf(e[0], e[1]), fmaxf(e[2], e[3]));
                const float mx = ext * sl2;  // -inf: nothing seen
                float alpha = 1.f;
                if (mx > m_used + kRescaleLog2) {  // includes the first finite max (m_used = -inf)
                    alpha = m_used == -INFINITY ? 0.f : ex2(m_used - mx);
                    m_used = mx;
                }
                // O_X is idle here: the stream's previous product is complete, the next one not issued
                if (it > 0 && __any_sync(0xffffffffu, alpha != 1.f)) {
#pragma unroll 1
                    for (int c = 0; c < D; c += 16) {
                        float o[16];
                        tmem_ld16(tO + c, o);
#pragma unroll
                        for (int i = 0; i < 16; ++i) o[i] *= alpha;
                        tmem_st16f(tO + c, o);
                    }
                }
                const float neg_m = m_used == -INFINITY ? 0.f : -m_used;
                float ls[4] = {0.f, 0.f, 0.f, 0.f};
                const uint64_t sc2 = pack_f32x2(sl2, sl2), nm2 = pack_f32x2(neg_m, neg_m);
#pragma unroll
                for (int hh = 0; hh < 4; ++hh) {  // 32 keys at a time
                    uint32_t hv[16], lv[16];
#pragma unroll
                    for (int i = 0; i < 16; ++i) {
                        const int c = hh * 32 + 2 * i;
                        float x0, x1;
                        unpack_f32x2(fma_f32x2(pack_f32x2(s[c], s[c + 1]), sc2, nm2), x0, x1);
                        x0 = ex2(x0);
                        x1 = ex2(x1);
                        hv[i] = pack_half2(x0, x1);
                        if constexpr (kSplitP) {
                            const float2 f = unpack_half2(hv[i]);
                            lv[i] = pack_half2(x0 - f.x, x1 - f.y);
                            ls[i & 3] += x0 + x1;
                        } else {
                            ls[i & 3] = add_halves(hv[i], ls[i & 3]);
                        }
                    }
                    tmem_st16(tS + hh * 16, hv);
                    if constexpr (kSplitP) tmem_st16(tS + 64 + hh * 16, lv);
                }
                l = l * alpha + ((ls[0] + ls[1]) + (ls[2] + ls[3]));
            }
            if (masked && (!two_rows || x == 0)) {
                // V rows past the context are zeroed, so that whatever they hold cannot reach an output through a
                // zero weight; so are infinities and NaN among the tree's V rows, which not every row sees (the rows
                // that do get them back at the end).  With two row tiles stream A does it: its product is first.
                ok = __all_sync(0xffffffffu, wait(&v_full[vs], vph & 1, s_abort));
                if (!ok) break;
                uint8_t* vt = vst(vs);
                const int from = max(hist - k0, 0), end = ctx - k0;
                bool found = false;
                for (int e = wq * 32 + lane; e < (kKeys - from) * 8 * Geo::kChunks; e += 128) {
                    const int r = from + e / (8 * Geo::kChunks), rest = e % (8 * Geo::kChunks);
                    uint4* at = reinterpret_cast<uint4*>(vt + (rest / 8) * Geo::kChunkBytes + sw128(r, rest % 8));
                    if (r >= end) {
                        *at = make_uint4(0u, 0u, 0u, 0u);
                    } else {
                        uint4 v = *at;
                        bool bad = false;
                        v = make_uint4(finite_halves(v.x, bad), finite_halves(v.y, bad), finite_halves(v.z, bad),
                                       finite_halves(v.w, bad));
                        if (bad) {
                            *at = v;
                            found = true;
                        }
                    }
                }
                if (found) *s_bad_v = 1;
                fence_proxy_async_smem();  // visible to the tensor cores (async proxy)
            }
            tmem_wait_st();
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(&p_full[x]);
            if ((vs += step) >= VS) {
                vs -= VS;
                ++vph;
            }
        }
        if (ok && it > 0) ok = __all_sync(0xffffffffu, wait(&o_full[x], (it - 1) & 1, s_abort));
        tc_fence_after();
        row_warps_sync();  // both streams done: the rings are idle, the notes on bad blocks and values complete
        // the thread's state into the state area: slot x * 128 + row
        const bool drop = *s_bad_block != 0 || *s_abort != 0 || !ok || it == 0;
        float2* ml = reinterpret_cast<float2*>(smem + Geo::kMlOff);
        ml[x * kRows + row] = drop ? make_float2(-INFINITY, 0.f) : make_float2(m_used, l);
        if (live_warp && !drop) {
            float* mine = reinterpret_cast<float*>(smem + Geo::kStateOff) + (x * kRows + row) * Geo::kOStride;
#pragma unroll 1
            for (int c = 0; c < D; c += 32) {
                float o[32];
                tmem_ld32(tO + c, o);
#pragma unroll
                for (int i = 0; i < 32; i += 4)
                    *reinterpret_cast<float4*>(mine + c + i) = make_float4(o[i], o[i + 1], o[i + 2], o[i + 3]);
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
    if (*s_bad_block != 0) *s_bad_v = 0;  // the chunk is left out
    if (p.cluster > 1) {
        __syncwarp();
        cluster_sync_all();  // every CTA's states are in its shared memory
    } else {
        __syncthreads();
    }
    // ================= the cluster's states merged: each CTA takes a share of the rows =================
    {
        constexpr int kCols = D / 4;  // a thread per four columns of a row
        const int live_rows = min(two_rows ? 2 * kRows : kRows, rows - r0);
        const int share = (live_rows + p.cluster - 1) / p.cluster;
        const int ra = min(rank * share, live_rows), rb = min(ra + share, live_rows);
        const int ncta = min(p.cluster, (all_tiles - clus * per_clus + p.chunk - 1) / p.chunk);  // CTAs with tiles
        const uint32_t state0 = smem_u32(smem + Geo::kStateOff), ml0 = smem_u32(smem + Geo::kMlOff);
        const uint32_t flag0 = smem_u32(const_cast<int*>(s_bad_v));
        for (int e = threadIdx.x; e < (rb - ra) * kCols; e += kThreads) {
            const int r = ra + e / kCols, c = e % kCols * 4, rr = r0 + r;
            float m = -INFINITY, l = 0.f;
            float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
            unsigned bad_v = 0;
            for (int q = 0; q < ncta; ++q) {
                const uint32_t st = cluster_addr(state0, q), mls = cluster_addr(ml0, q);
                if (ld_cluster_u32(cluster_addr(flag0, q)) != 0) bad_v |= 1u << q;
                for (int slot = r; slot < 2 * kRows; slot += two_rows ? 2 * kRows : kRows) {
                    const float2 s = ld_cluster_f32x2(mls + slot * 8);
                    if (s.y == 0.f) continue;  // the state holds nothing (and its O may be unwritten)
                    const float4 a = ld_cluster_f32x4(st + (slot * Geo::kOStride + c) * 4);
                    const float mn = fmaxf(m, s.x);
                    const float f_old = m == mn ? 1.f : ex2(m - mn), f_new = s.x == mn ? 1.f : ex2(s.x - mn);
                    o = fma4(f_new, a, scale4(o, f_old));
                    l = l * f_old + s.y * f_new;
                    m = mn;
                }
            }
            const int64_t orow = (static_cast<int64_t>(b) * p.T + rr / p.G) * p.Hq + hk * p.G + rr % p.G;
            if (whole) o = scale4(o, l > 0.f || l != l ? 1.f / l : 0.f);
            if (bad_v != 0) {
                // infinities and NaN of the tree's V rows that this row sees, in the noted CTAs' keys
                const uint64_t mask = p.masks[static_cast<int64_t>(b) * p.T + rr / p.G];
                for (int t = 0; t < tree; ++t) {
                    const int pos = hist + t, q = pos / kKeys / p.chunk - clus * p.cluster;
                    if (!((mask >> t) & 1) || q < 0 || q >= ncta || !((bad_v >> q) & 1u)) continue;
                    const int64_t blk = table_row[pos / kBlockSize];
                    const __half* v = p.v_cache + ((blk * p.Hkv + hk) * kBlockSize + pos % kBlockSize) * D + c;
                    const float y[4] = {__half2float(v[0]), __half2float(v[1]), __half2float(v[2]), __half2float(v[3])};
                    if (!(fabsf(y[0]) < INFINITY)) o.x += y[0];
                    if (!(fabsf(y[1]) < INFINITY)) o.y += y[1];
                    if (!(fabsf(y[2]) < INFINITY)) o.z += y[2];
                    if (!(fabsf(y[3]) < INFINITY)) o.w += y[3];
                }
            }
            if (whole) {
                store_out4(p.out, p.out_f32, orow * D + c, o);
            } else {
                const int64_t prow = orow * p.nclus + clus;
                if (c == 0) *reinterpret_cast<float2*>(p.part_ml + prow * 2) = make_float2(m, l);
                *reinterpret_cast<float4*>(p.part_acc + prow * D + c) = o;
            }
        }
    }
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
    int tree, ctx;
    if (!lengths(p, b, tree, ctx) || t >= tree) return;
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

constexpr int kTreeSplitCluster = 4;  // CTAs per cluster where a context needs several clusters
constexpr int kTreeCtaCost = 8;       // in half key tiles
constexpr int kTreeCombineCost = 6;

template <int D, bool kSplitP>
static cudaError_t tree_setup() {
    static std::once_flag once;
    static cudaError_t err = cudaSuccess;
    std::call_once(once, [] {
        err = cudaFuncSetAttribute(tree::paged_decode_tree_kernel<D, kSplitP>,
                                   cudaFuncAttributeMaxDynamicSharedMemorySize, tree::Geom<D>::kSmemBytes);
    });
    return err;
}

// Clusters of cs CTAs (one per SM) that the device holds at a time; the SMs of a GPC that no whole cluster fills stay
// idle.  Asked once per device and size.
static int resident_clusters(int D, int cs, int sms) {
    static std::atomic<int> cache[128][2][tree::kMaxTreeCluster + 1];
    if (cs == 1) return sms;
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 128) return sms / cs;
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
    if (sms <= 0) return cudaErrorNoDevice;
    if (D != 64 && D != 128) return cudaErrorInvalidValue;
    const int G = Hq / Hkv;
    const int row_tiles = (T * G + tree::kRows - 1) / tree::kRows;
    plan->row_pairs = (row_tiles + 1) / 2;
    const int tiles = std::max(1, (max_ctx + tree::kKeys - 1) / tree::kKeys);
    const int64_t units = std::max<int64_t>(1, static_cast<int64_t>(B) * Hkv * plan->row_pairs);
    // The split of the context with the shortest run, counted in key tiles: waves of clusters times the tiles of a CTA
    // plus the start and end of a CTA; merging in a cluster costs little, partial states and the combine launch more.
    int64_t best_cost = INT64_MAX;
    for (int nc = 1; nc <= std::min(tiles, 128); ++nc) {
        const int chunk = (tiles + nc - 1) / nc;
        if ((tiles + chunk - 1) / chunk != nc) continue;
#ifdef KVC_TREE_NC
        if (nc != KVC_TREE_NC) continue;
#endif
        const int cs = std::min(nc, nc <= tree::kMaxTreeCluster ? tree::kMaxTreeCluster : kTreeSplitCluster);
        const int nclus = (nc + cs - 1) / cs;
        const int64_t resident = resident_clusters(D, cs, sms);
        const int64_t waves = (units * nclus + resident - 1) / resident;
        const int64_t cost = waves * (2 * chunk + kTreeCtaCost) + (nc > 1 ? 1 + cs / 2 : 0) + (nclus > 1 ? kTreeCombineCost + nclus / 4 : 0);
        if (cost < best_cost) {
            best_cost = cost;
            plan->chunk = chunk;
            plan->cluster = cs;
            plan->nclus = nclus;
        }
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
    p.max_blocks = a.max_blocks;
    p.num_blocks = a.num_blocks;
    p.max_ctx = a.max_context_len;
    p.out_f32 = a.out_f32;
    p.chunk = plan.chunk;
    p.cluster = plan.cluster;
    p.nclus = plan.nclus;
    p.row_pairs = plan.row_pairs;
    p.negate = a.scale < 0.f;
    p.scale_log2 = std::max(std::fabs(a.scale) * kLog2e, tree::kMinScaleLog2);
    const dim3 grid(static_cast<unsigned>(plan.row_pairs * plan.nclus * plan.cluster), a.Hkv, a.B);
    e = launch(tree::paged_decode_tree_kernel<D, kSplitP>, grid, dim3(tree::kThreads), Geo::kSmemBytes, stream, false,
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
