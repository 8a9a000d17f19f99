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
constexpr int kLoadWarp = kRowWarps + 1;
constexpr int kThreads = (kRowWarps + 2) * 32;
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
    static constexpr int kQOff = 0;
    static constexpr int kKOff = kQOff + 2 * kTileBytes;
    static constexpr int kVOff = kKOff + kKStages * kTileBytes;
    static constexpr int kBarOff = kVOff + kVStages * kTileBytes;
    static constexpr int kSmemBytes = kBarOff + 256 + 1024;  // barriers, TMEM address, flags; alignment
    static_assert(kSmemBytes <= 227 * 1024, "shared memory of one CTA");
    // the streams exchange half of their output columns in the K/V rings at the end
    static constexpr int kXStride = D / 2 + 4;  // floats per exchanged row (padded: rows on distinct banks)
    static_assert(2 * kRows * (kXStride + 2) * 4 <= kBarOff - kKOff, "exchange area");
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
    int chunk;       // key tiles per CTA
    int max_chunks;  // chunks of the longest context: stride of the partial states
    int row_pairs;   // pairs of row tiles of the widest tree
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
    constexpr int KS = Geo::kKStages, VS = Geo::kVStages;
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    uint64_t* bars = reinterpret_cast<uint64_t*>(smem + Geo::kBarOff);
    uint64_t* q_full = bars;                 // query rows in shared memory (one arrival per row warp)
    uint64_t* k_full = bars + 1;             // [KS] K tile landed
    uint64_t* k_empty = k_full + KS;         // [KS] S products of the stage's tile done
    uint64_t* v_full = k_empty + KS;         // [VS] V tile landed
    uint64_t* v_empty = v_full + VS;         // [VS] P V products of the stage's tile done
    uint64_t* s_full = v_empty + VS;         // [2] S_X of the stream's tile in TMEM
    uint64_t* p_full = s_full + 2;           // [2] P_X of the stream's tile in TMEM (4 arrivals)
    uint64_t* o_full = p_full + 2;           // [2] P_X V of the stream's tile done
    uint64_t* fin = o_full + 2;              // every MMA issued so far done
    uint32_t* s_tmem = reinterpret_cast<uint32_t*>(fin + 1);
    volatile int* s_abort = reinterpret_cast<volatile int*>(s_tmem + 1);
    volatile int* s_bad_block = s_abort + 1;  // a block id out of range: the chunk is left out
    volatile int* s_bad_v = s_abort + 2;      // an infinity or NaN among the tree's V values
    static_assert((1 + 2 * KS + 2 * VS + 7) * 8 + 16 <= 256, "barrier area");

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int pair = static_cast<int>(blockIdx.x) % p.row_pairs, chunk = static_cast<int>(blockIdx.x) / p.row_pairs;
    const int hk = blockIdx.y, b = blockIdx.z;
    int tree, ctx;
    if (!lengths(p, b, tree, ctx)) {
        if (chunk == 0 && pair == 0) {
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
    const int all_tiles = key_tiles(ctx), c0 = chunk * p.chunk;
    if (r0 >= rows || c0 >= all_tiles) return;
    const int n = min(p.chunk, all_tiles - c0);          // key tiles of this CTA
    const bool two_rows = rows - r0 > kRows;             // two row tiles: they are the streams
    const int step = two_rows ? 1 : 2;                   // key tiles between two of a stream's
    const int hist = ctx - tree;                         // keys before the tree
    const int pages = (ctx + kBlockSize - 1) / kBlockSize;
    const int nchunks = (all_tiles + p.chunk - 1) / p.chunk;

    auto qs = [&](int x) { return smem + Geo::kQOff + x * Geo::kTileBytes; };
    auto kst = [&](int st) { return smem + Geo::kKOff + st * Geo::kTileBytes; };
    auto vst = [&](int st) { return smem + Geo::kVOff + st * Geo::kTileBytes; };

    if (threadIdx.x == 0) {
        mbar_init(q_full, kRowWarps);
        for (int i = 0; i < KS; ++i) {
            mbar_init(&k_full[i], 1);
            mbar_init(&k_empty[i], 1);
        }
        for (int i = 0; i < VS; ++i) {
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
    if (warp == 0) {
        tmem_alloc(s_tmem, Geo::kTmemCols);
        tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *s_tmem;

    if (warp == kLoadWarp) {
        // ================= loads: lane i copies block i of every K and V tile =================
        if (lane == 0) {
            prefetch_tensormap(&tmK);
            prefetch_tensormap(&tmV);
        }
        // one pair of row tiles reads its K and V once; several pairs meet them in L2
        const uint64_t policy = p.row_pairs == 1 ? l2_policy_evict_first() : l2_policy_evict_normal();
        const int32_t* row = p.block_table + static_cast<int64_t>(b) * p.max_blocks;
        auto block_of = [&](int j) {
            const int page = (c0 + j) * kPages + lane;
            return lane < kPages && page < pages ? row[page] : -1;
        };
        auto load = [&](uint8_t* tile, const CUtensorMap* map, uint64_t* bar, int j, int phys) {
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
        int k_issued = 0, v_issued = 0, next = block_of(0);
        bool ok = true;
        for (int j = 0; ok && j < n; ++j) {
            int phys = next;
            if (j + 1 < n) next = block_of(j + 1);
            if (lane < min(kPages, pages - (c0 + j) * kPages) && (phys < 0 || phys >= p.num_blocks)) {
                atomicOr(p.err, KVC_DEVERR_BLOCK_ID);
                *s_bad_block = 1;  // seen by the row warps behind this tile's barriers
                phys = 0;          // a block of the pool, whose values are not used
            }
            __syncwarp();
            if (j >= KS) ok = __all_sync(0xffffffffu, wait(&k_empty[j % KS], ((j - KS) / KS) & 1, s_abort));
            if (!ok) break;
            load(kst(j % KS), &tmK, &k_full[j % KS], j, phys);
            k_issued = j + 1;
            if (j >= VS) ok = __all_sync(0xffffffffu, wait(&v_empty[j % VS], ((j - VS) / VS) & 1, s_abort));
            if (!ok) break;
            load(vst(j % VS), &tmV, &v_full[j % VS], j, phys);
            v_issued = j + 1;
        }
        // copies still in flight land before the shared memory is released (immediate unless aborted: the products
        // consumed every tile)
        if (lane == 0) {
            for (int t = max(0, k_issued - KS); t < k_issued; ++t)
                mbar_wait_bounded(&k_full[t % KS], (t / KS) & 1, kWaitNs / 8);
            for (int t = max(0, v_issued - VS); t < v_issued; ++t)
                mbar_wait_bounded(&v_full[t % VS], (t / VS) & 1, kWaitNs / 8);
        }
    } else if (warp == kMmaWarp) {
        // ================= tensor-core products (one thread) =================
        if (lane == 0) {
            constexpr uint32_t idS = umma_idesc_f16(kRows, kKeys, 0, 0);
            constexpr uint32_t idPV = umma_idesc_f16(kRows, D, 0, 1);
            const uint64_t dQ = umma_smem_desc(smem_u32(qs(0)), 16, 1024);
            const uint64_t dK = umma_smem_desc(smem_u32(kst(0)), 16, 1024);
            // V as the MN-major B operand: 8-key groups 1024 bytes apart, 64-dim atoms one chunk apart
            const uint64_t dV = umma_smem_desc(smem_u32(vst(0)), Geo::kChunkBytes, 1024);
            // S_X = Q_X K^T over D / 16 steps of 16 dims (with one row tile both streams use it)
            auto mma_s = [&](int x, int st) {
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
            auto mma_pv = [&](int x, int st, bool first) {
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
            bool ok = wait(q_full, 0, s_abort);
            // the first tile of each stream: tile 0 for both, or tiles 0 and 1
            for (int x = 0; ok && x < 2; ++x) {
                const int j = two_rows ? 0 : x;
                if (j >= n) break;
                if (!(ok = wait(&k_full[j], 0, s_abort))) break;
                tc_fence_after();
                mma_s(x, j);
                if (!two_rows || x == 1) umma_commit(&k_empty[j]);
            }
            for (int j = 0; ok && j < n; ++j) {
                if (!(ok = wait(&v_full[j % VS], (j / VS) & 1, s_abort))) break;
                const int jn = j + step;
                const uint32_t it = static_cast<uint32_t>(two_rows ? j : j >> 1);  // the streams' tile count
                // per stream of this tile: P_X V once P_X is in TMEM; then the stream's next S_X into the same
                // columns once that product has read P_X
                for (int x = two_rows ? 0 : (j & 1), left = two_rows ? 2 : 1; ok && left > 0; ++x, --left) {
                    if (!(ok = wait(&p_full[x], it & 1, s_abort))) break;
                    tc_fence_after();
                    mma_pv(x, j % VS, it == 0);
                    if (jn < n) {
                        if (!(ok = wait(&k_full[jn % KS], (jn / KS) & 1, s_abort))) break;
                        if (!(ok = wait(&o_full[x], it & 1, s_abort))) break;
                        tc_fence_after();
                        mma_s(x, jn % KS);
                    }
                }
                if (!ok) break;
                umma_commit(&v_empty[j % VS]);
                if (jn < n) umma_commit(&k_empty[jn % KS]);
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
                ok = __all_sync(0xffffffffu, wait(&v_full[j % VS], (j / VS) & 1, s_abort));
                if (!ok) break;
                uint8_t* vt = vst(j % VS);
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
        }
        if (ok && it > 0) ok = __all_sync(0xffffffffu, wait(&o_full[x], (it - 1) & 1, s_abort));
        tc_fence_after();
        row_warps_sync();  // both streams done; their notes on bad blocks and values are complete
        const bool drop = *s_bad_block != 0 || *s_abort != 0 || !ok;
        if (drop) {
            l = 0.f;
            m_used = -INFINITY;
        }
        float w_own = 1.f;   // weights of this stream's and the other's state in the merged one
        float w_other = 0.f;
        int col0 = 0, cols = D;
        float* xrow = nullptr;  // the other stream's half of this thread's row
        if (!two_rows) {
            // each stream keeps one half of the columns and hands the other half over, in the idle K/V rings
            float* area = reinterpret_cast<float*>(smem + Geo::kKOff);
            float2* ml = reinterpret_cast<float2*>(area + 2 * kRows * Geo::kXStride);
            float* mine = area + ((1 - x) * kRows + row) * Geo::kXStride;
            ml[x * kRows + row] = make_float2(m_used, l);
            if (it > 0 && live_warp && !drop) {
                const int give = (1 - x) * (D / 2);
#pragma unroll 1
                for (int c = 0; c < D / 2; c += 16) {
                    float o[16];
                    tmem_ld16(tO + give + c, o);
#pragma unroll
                    for (int i = 0; i < 16; i += 4)
                        *reinterpret_cast<float4*>(mine + c + i) = make_float4(o[i], o[i + 1], o[i + 2], o[i + 3]);
                }
            }
            row_warps_sync();
            const float2 theirs = ml[(1 - x) * kRows + row];
            const float M = fmaxf(m_used, theirs.x);
            // a stream that saw no key (or no tile at all) holds l = 0 and adds nothing
            w_own = l > 0.f ? (m_used == M ? 1.f : ex2(m_used - M)) : l != l ? 1.f : 0.f;
            w_other = theirs.y > 0.f ? (theirs.x == M ? 1.f : ex2(theirs.x - M)) : theirs.y != theirs.y ? 1.f : 0.f;
            l = (w_own != 0.f ? l * w_own : 0.f) + (w_other != 0.f ? theirs.y * w_other : 0.f);
            m_used = M;
            col0 = x * (D / 2);
            cols = D / 2;
            xrow = area + (x * kRows + row) * Geo::kXStride;
        }
        if (live_warp && !(*s_abort)) {
            const bool whole = nchunks == 1;
            const float inv = whole ? (l > 0.f || l != l ? 1.f / l : 0.f) : 1.f;
            const int64_t orow = (static_cast<int64_t>(b) * p.T + rr / p.G) * p.Hq + hk * p.G + rr % p.G;
            const int64_t prow = orow * p.max_chunks + chunk;
            if (live && !whole && col0 == 0)
                *reinterpret_cast<float2*>(p.part_ml + prow * 2) = make_float2(m_used, l);
            const bool bad_v = *s_bad_v != 0 && !drop;
            // a state that holds nothing is left out, not multiplied by 0 (1 / l may be NaN or infinite)
            const bool own = it > 0 && w_own != 0.f && l != 0.f, other = xrow != nullptr && w_other != 0.f;
            const float f_own = w_own * inv, f_other = w_other * inv;
#pragma unroll 1
            for (int c = col0; c < col0 + cols; c += 16) {
                float o[16];
                if (it > 0) {
                    tmem_ld16(tO + c, o);
                } else {
#pragma unroll
                    for (int i = 0; i < 16; ++i) o[i] = 0.f;
                }
                if (!live) continue;
#pragma unroll
                for (int i = 0; i < 16; ++i) o[i] = own ? o[i] * f_own : 0.f;
                if (other) {
#pragma unroll
                    for (int i = 0; i < 16; i += 4) {
                        const float4 y = *reinterpret_cast<const float4*>(xrow + c - col0 + i);
                        o[i] = fmaf(y.x, f_other, o[i]);
                        o[i + 1] = fmaf(y.y, f_other, o[i + 1]);
                        o[i + 2] = fmaf(y.z, f_other, o[i + 2]);
                        o[i + 3] = fmaf(y.w, f_other, o[i + 3]);
                    }
                }
                if (bad_v) {
                    // infinities and NaN of the tree's V rows that this row sees, in this chunk's keys
                    const int t0 = max(0, c0 * kKeys - hist), t1 = min(tree, (c0 + n) * kKeys - hist);
                    for (int t = t0; t < t1; ++t) {
                        if (!((mask >> t) & 1)) continue;
                        const int pos = hist + t;
                        const int64_t blk =
                            p.block_table[static_cast<int64_t>(b) * p.max_blocks + pos / kBlockSize];
                        const __half* v =
                            p.v_cache + ((blk * p.Hkv + hk) * kBlockSize + pos % kBlockSize) * D + c;
                        for (int i = 0; i < 16; ++i) {
                            const float y = __half2float(v[i]);
                            if (!(fabsf(y) < INFINITY)) o[i] += y;
                        }
                    }
                }
                if (!whole) {
                    float4* dst = reinterpret_cast<float4*>(p.part_acc + prow * D + c);
#pragma unroll
                    for (int i = 0; i < 4; ++i)
                        dst[i] = make_float4(o[4 * i], o[4 * i + 1], o[4 * i + 2], o[4 * i + 3]);
                } else if (p.out_f32) {
                    float4* dst = reinterpret_cast<float4*>(static_cast<float*>(p.out) + orow * D + c);
#pragma unroll
                    for (int i = 0; i < 4; ++i)
                        dst[i] = make_float4(o[4 * i], o[4 * i + 1], o[4 * i + 2], o[4 * i + 3]);
                } else {
                    uint4* dst = reinterpret_cast<uint4*>(static_cast<__half*>(p.out) + orow * D + c);
#pragma unroll
                    for (int i = 0; i < 2; ++i)
                        dst[i] = make_uint4(pack_half2(o[8 * i], o[8 * i + 1]), pack_half2(o[8 * i + 2], o[8 * i + 3]),
                                            pack_half2(o[8 * i + 4], o[8 * i + 5]),
                                            pack_half2(o[8 * i + 6], o[8 * i + 7]));
                }
            }
        }
    }
    // every TMEM access of the CTA is complete; the allocating warp frees it
    tc_fence_before();
    __syncthreads();
    if (warp == 0) {
        tc_fence_after();
        tmem_dealloc(tmem, Geo::kTmemCols);
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
    const int nchunks = (key_tiles(ctx) + p.chunk - 1) / p.chunk;
    if (nchunks <= 1) return;  // the attention kernel wrote the row
    float m = -INFINITY, l = 0.f;
    float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 4
    for (int s = 0; s < nchunks; ++s) {
        const int64_t at = row * p.max_chunks + s;
        const float2 ml = *reinterpret_cast<const float2*>(p.part_ml + at * 2);
        const float4 a = *reinterpret_cast<const float4*>(p.part_acc + at * D + c);
        if (ml.y == 0.f) continue;  // the row saw none of the chunk's keys
        const float mn = fmaxf(m, ml.x);
        const float f_old = m == mn ? 1.f : m == -INFINITY ? 0.f : ex2(m - mn), f_new = ml.x == mn ? 1.f : ex2(ml.x - mn);
        o = fma4(f_new, a, scale4(o, f_old));
        l = l * f_old + ml.y * f_new;
        m = mn;
    }
    store_out4(p.out, p.out_f32, row * D + c, scale4(o, l > 0.f || l != l ? 1.f / l : 0.f));
}

}  // namespace tree

cudaError_t tree_plan(int B, int Hq, int Hkv, int D, int max_ctx, int T, TreePlan* plan) {
    const int sms = sm_count();
    if (sms <= 0) return cudaErrorNoDevice;
    if (D != 64 && D != 128) return cudaErrorInvalidValue;
    const int G = Hq / Hkv;
    const int row_tiles = (T * G + tree::kRows - 1) / tree::kRows;
    plan->row_pairs = (row_tiles + 1) / 2;
    const int tiles = std::max(1, (max_ctx + tree::kKeys - 1) / tree::kKeys);
    const int64_t units = std::max<int64_t>(1, static_cast<int64_t>(B) * Hkv * plan->row_pairs);
    // The number of chunks with the shortest run, counted in key tiles: waves of CTAs (one per SM) times the tiles of
    // a chunk plus the start and end of a CTA (about four tiles' time); several chunks also pay for their states and
    // the combine launch (about three).
    int best = 1;
    int64_t best_cost = INT64_MAX;
    for (int nc = 1; nc <= std::min(tiles, 64); ++nc) {
        const int chunk = (tiles + nc - 1) / nc;
        const int used = (tiles + chunk - 1) / chunk;
        if (used != nc) continue;
        const int64_t waves = (units * nc + sms - 1) / sms;
        const int64_t cost = waves * (chunk + 4) + (nc > 1 ? 3 + nc / 8 : 0);
        if (cost < best_cost) {
            best_cost = cost;
            best = nc;
        }
    }
    plan->chunk = (tiles + best - 1) / best;
    plan->max_chunks = (tiles + plan->chunk - 1) / plan->chunk;
    plan->workspace_bytes =
        plan->max_chunks > 1 ? partials_bytes(static_cast<size_t>(B) * T * Hq * plan->max_chunks, D) : 0;
    return cudaSuccess;
}

template <int D, bool kSplitP>
static cudaError_t launch_tree_d(const TreeArgs& a, const TreePlan& plan, cudaStream_t stream) {
    using Geo = tree::Geom<D>;
    static std::once_flag attr_once;
    static cudaError_t attr_err = cudaSuccess;
    std::call_once(attr_once, [] {
        attr_err = cudaFuncSetAttribute(tree::paged_decode_tree_kernel<D, kSplitP>,
                                        cudaFuncAttributeMaxDynamicSharedMemorySize, Geo::kSmemBytes);
    });
    if (attr_err != cudaSuccess) return attr_err;
    const int64_t rows = static_cast<int64_t>(a.num_blocks) * a.Hkv * kBlockSize;
    CUtensorMap tmK, tmV;
    cudaError_t e = make_tile_map(&tmK, a.k_cache, D, rows);
    if (e == cudaSuccess) e = make_tile_map(&tmV, a.v_cache, D, rows);
    if (e != cudaSuccess) return e;
    const size_t nrow = static_cast<size_t>(a.B) * a.T * a.Hq * plan.max_chunks;
    tree::Params p;
    p.q = a.q;
    p.block_table = a.block_table;
    p.context_lens = a.context_lens;
    p.tree_lens = a.tree_lens;
    p.masks = a.masks;
    p.v_cache = a.v_cache;
    p.out = a.out;
    p.part_ml = static_cast<float*>(a.workspace);
    p.part_acc = plan.max_chunks > 1 ? partials_acc(p.part_ml, nrow) : nullptr;
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
    p.max_chunks = plan.max_chunks;
    p.row_pairs = plan.row_pairs;
    p.negate = a.scale < 0.f;
    p.scale_log2 = std::max(std::fabs(a.scale) * kLog2e, tree::kMinScaleLog2);
    const dim3 grid(static_cast<unsigned>(plan.row_pairs * plan.max_chunks), a.Hkv, a.B);
    e = launch(tree::paged_decode_tree_kernel<D, kSplitP>, grid, dim3(tree::kThreads), Geo::kSmemBytes, stream, false,
               1u, tmK, tmV, p);
    if (e != cudaSuccess || plan.max_chunks == 1) return e;
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
