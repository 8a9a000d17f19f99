// Varlen packed causal prefill with a sliding window and sinks, on the 5th-generation tensor cores of sm_103a.
//
// Row i of a segment sees the rows j <= i of the same segment with j > i - window or j < sinks:
//   out = softmax(q K^T * scale) V  over these, query head h reading KV head h / (Hq / Hkv),
// with the running-max / exp-sum rule of the FlashAttention article over key tiles.
//
// Layout.  An item is 256 query rows of a segment and a query head: two row tiles A and B of 128 rows (the M of the
// products; a TMEM lane and a softmax thread each), the two streams of the CTA.  Its key tiles of 128 are a list: the
// tile at the far end of A's window that B's no longer reaches (`lead`, 0 or 1 of them), the sinks' tiles, then from B's
// window to the diagonal; A takes the list without its end, B without its beginning, so that no tile is read that
// neither sees.  Streams work on them in units of 64 keys; of a last tile of sinks alone, on what holds some.
// Per stream X and unit:  S_X = Q_X K^T (both K-major in shared memory, 128-byte swizzle, as TMA writes them); the row
// warps take S_X from TMEM, mask it where the unit crosses an edge (bits of what a row sees, applied once), keep the
// running max lazily (it moves when it has grown by 2^4; O_X is then rescaled in TMEM) and write P_X over S_X in fp16;
// O_X += P_X V with P_X from TMEM and V MN-major.  Two buffers of S / P per stream let S of the next unit run under this
// one's softmax.
// Warps.  Eight row warps; one product warp per stream and product (S_A, S_B, PV_A, PV_B: one warp for all of them was
// the bound of the form with tiles of 128 keys and one buffer, prefill.cu's); a copy warp for Q and K, one for V.
// P.  One fp16 value, the row sums adding the rounded weights, or an fp16 high part plus residual (two products);
// weights are carried 2^11 times as large, so that fp16's 11 bits last down to 2^-25 of a row's largest one.
// Hidden values.  A masked key's weight is 0, and 0 times an infinity or NaN in its V row would be NaN: a row that comes
// out infinite or NaN is computed again from its visible keys alone.
// Items.  The grid has a CTA for every item that total_tokens and max_seqlen leave possible; a CTA that runs takes over
// those that have not started (cluster launch control).  One warp asks for them, finds the segment and row block that an
// index stands for (sums of the segments' row blocks, 32 segments at a time), and hands a description of the next item to
// the rest when the last one's copies are out (asked for earlier, few items pile up on some CTAs: five uneven prompts of
// 5841 tokens in all, window 512, 8 heads, D = 64, 35 us so and 24 otherwise; a CTA for every item 28).  Copies and
// products of the next item start under the end of this one (window 128 of 4 x 4096 tokens, 32 / 8 heads, D = 128: 165 us
// with a CTA per item, 125 so).
// Bound by a row warp's chain through a unit, some 1350 clocks at D = 64 for products of 370: 500 in the exponentials (256
// at their pipe's rate, shared with the other stream's), 230 in the load and the maximum, 140 in the wait for S, the rest
// in votes, branches and the handing over.  Now 4 x 4096 tokens, 32 / 8 heads, D = 128: 358 to 370 us with window 4096 (1490
// to 1536 TFLOP/s, 75 % of the measured rate), 232 with 1024, 106 to 117 with 128; 32,768 tokens, window 4096, 14 / 2 heads, D = 64: 512;
// the five uneven prompts 20.8.  Tried and slower: sixteen row warps, a set for each buffer that hands its maxima to the
// other (641 against 554: with twice the warps everything in them takes twice as long), a warp of its own for Q (window 128
// 117 -> 110, but 516 -> 520 at D = 64).
// Every wait is bounded; a timeout sets an error bit and drains the CTA.
#include <algorithm>
#include <cmath>
#include <cudaTypedefs.h>
#include <mutex>

#include "../../include/kvc.h"
#include "decode_common.cuh"
#include "f32x2.cuh"
#include "kvc_internal.h"
#include "prefill_window.cuh"
#include "ptx.cuh"
#include "tcgen05.cuh"

namespace kvc {
namespace pfw {

constexpr int kRows = 128;  // rows of a row tile
constexpr int kKeys = 128;  // keys of a key tile
constexpr int kHalf = 64;   // keys of a unit
constexpr int kRowWarps = 8;
constexpr int kSWarp = kRowWarps;       // S products of stream A, of stream B
constexpr int kPvWarp = kRowWarps + 2;  // P V products of stream A, of stream B
constexpr int kLoadKWarp = kRowWarps + 4;
constexpr int kLoadVWarp = kRowWarps + 5;
constexpr int kItemWarp = kRowWarps + 6;  // hands out the items to the other warps
constexpr int kThreads = (kRowWarps + 7) * 32;
constexpr int kSlots = 2;  // items described at a time
constexpr uint64_t kWaitNs = 1000000000ull;
// (as in the tree attention: weights carried 2^11 times as large; the max moves when a score is 2^15 above it; beyond
// kFar a step of a score's exponent is no longer small against fp16's range)
constexpr float kWeightLog2 = 11.f;
constexpr float kRescaleLog2 = 15.f;
constexpr float kFar = 0x1p22f;

template <int D>
struct Geom {
    static constexpr int kChunks = D / 64;  // 64-dim (128-byte) column chunks
    static constexpr int kKStages = D == 64 ? 5 : 3;
    static constexpr int kVStages = D == 64 ? 5 : 2;
    static constexpr int kChunkBytes = kRows * 128;  // 128 rows or keys x 64 dims
    static constexpr int kTileBytes = kChunks * kChunkBytes;
    static constexpr int kQOff = 0;  // Q_A, Q_B
    static constexpr int kVOff = kQOff + 2 * kTileBytes;
    static constexpr int kKOff = kVOff + kVStages * kTileBytes;
    // D = 64 (TMEM has the columns for it): row sums come from a product too, with a tile of 64 keys of ones
    static constexpr bool kSumProduct = D == 64;
    static constexpr int kOnesOff = kKOff + kKStages * kTileBytes;
    static constexpr int kOnesBytes = kSumProduct ? kHalf * 128 : 0;
    static constexpr int kBarOff = kOnesOff + kOnesBytes;
    static constexpr int kItemOff = kBarOff + 512;  // barriers, TMEM address, flag; then the items
    static constexpr int kSmemBytes = kItemOff + 384 + 1024;  // alignment
    static_assert(kSmemBytes <= 227 * 1024, "shared memory of one CTA");
    // TMEM columns: two buffers of S / P per stream, A [0, 128) and B [128, 256), then O_A and O_B, D columns each
    static constexpr int kTmemO = 4 * kHalf;
    static constexpr int kTmemL = kTmemO + 2 * D;  // row sums of A and B, 64 equal columns each
    static constexpr uint32_t kTmemCols = 512;
};

struct Params {
    const int32_t* cu_seqlens;
    const __half* q;
    const __half* k;
    const __half* v;
    void* out;
    unsigned* err;
    int nseq, total_tokens, tiles_per_seq, Hq, Hkv, G, out_f32, window, sinks;
    int negate;        // the scale is negative
    int out_wide;      // out is aligned to 32 bytes
    float scale_log2;  // |scale| * log2 e, at least kMinWindowScaleLog2
};

__device__ __forceinline__ uint32_t sw128(int row, int c) {
    return static_cast<uint32_t>(row * 128 + ((c ^ (row & 7)) << 4));
}
__device__ __forceinline__ void tma_load_3d(void* smem_dst, const CUtensorMap* map, uint64_t* bar, int x, int y, int z) {
    asm volatile(
        "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
        " [%0], [%1, {%3, %4, %5}], [%2];" ::"r"(smem_u32(smem_dst)),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(smem_u32(bar)), "r"(x), "r"(y), "r"(z)
        : "memory");
}
// 32 bytes of a row of the output, at once where they are aligned to it (a row per lane: an instruction takes as long for
// 16 bytes of each)
__device__ __forceinline__ void store_32(void* at, const uint32_t (&w)[8], bool wide) {
    if (wide) {
        asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(at), "r"(w[0]), "r"(w[1]), "r"(w[2]),
                     "r"(w[3]), "r"(w[4]), "r"(w[5]), "r"(w[6]), "r"(w[7])
                     : "memory");
    } else {
        static_cast<uint4*>(at)[0] = make_uint4(w[0], w[1], w[2], w[3]);
        static_cast<uint4*>(at)[1] = make_uint4(w[4], w[5], w[6], w[7]);
    }
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
// The same for a whole warp: one vote and one branch where the phase is over already, the rest out of the way.
__device__ __noinline__ bool wait_on(uint64_t* bar, uint32_t parity, volatile int* abort_flag) {
    return __all_sync(0xffffffffu, wait(bar, parity, abort_flag));
}
__device__ __forceinline__ bool wait_warp(uint64_t* bar, uint32_t parity, volatile int* abort_flag) {
    if (__builtin_expect(__all_sync(0xffffffffu, mbar_try_wait(bar, parity)), 1)) return true;
    return wait_on(bar, parity, abort_flag);
}
// The same for a whole warp whose waits sit between two products: without the hint of a long sleep.  (Polling took issue
// slots from the row warps: 266 against 257 us at 4 x 4096 tokens, window 1024, 32 / 8 heads, D = 128.)
__device__ __forceinline__ bool wait_all(uint64_t* bar, uint32_t parity, volatile int* abort_flag) {
    if (__all_sync(0xffffffffu, mbar_try_wait(bar, parity))) return true;
    const uint64_t t0 = global_timer_ns();
    for (uint32_t i = 1;; ++i) {
        if (__all_sync(0xffffffffu, mbar_try_wait(bar, parity))) return true;
        if ((i & 63u) == 0u) {
            if (__any_sync(0xffffffffu, *abort_flag != 0)) return false;
            if (__any_sync(0xffffffffu, global_timer_ns() - t0 > kWaitNs)) {
                *abort_flag = 1;
                return false;
            }
        }
    }
}

// One item: its rows and its list of key tiles.  Stream A works on entries [0, end[0]), B on [lead, end[1]).
struct Item {
    int beg, len, h, hk, r0;
    int lead, sink_tiles, far0, near0, end[2], entries;
    int narrow;  // the entry of which the first unit alone holds visible keys, or -1
    int any;     // 0: the last one was before this
    int2 part[2][3];  // the same list in keys, for either stream: from, to
    __device__ __forceinline__ int key_tile(int j) const {
        return j < lead ? far0 + j : j < lead + sink_tiles ? j - lead : near0 + j - lead - sink_tiles;
    }
    __device__ __forceinline__ int begin(int x) const { return x == 0 ? 0 : lead; }
    __device__ __forceinline__ int units(int j) const { return j == narrow ? 1 : 2; }
};
constexpr int kItemBytes = 128;
static_assert(sizeof(Item) <= kItemBytes, "items in shared memory");
// Row blocks of 256 rows that a segment has; its first row and its length.
__device__ __forceinline__ int row_blocks(const Params& p, int seg, int& beg, int& len, bool& bad) {
    beg = p.cu_seqlens[seg];
    const int end = p.cu_seqlens[seg + 1];
    len = end - beg;
    if (beg < 0 || end < beg || end > p.total_tokens) {
        bad = true;
        return 0;
    }
    const int n = len / (2 * kRows) + (len % (2 * kRows) != 0);
    if (n > p.tiles_per_seq) bad = true;  // (rows past max_seqlen are not computed)
    return min(n, p.tiles_per_seq);
}
// The segments that the item warp is at: lane i has segment `first` + i's, and the row blocks up to its end.
struct Segments {
    int first = -32, beg, len, blocks, before, upto;  // before, upto: row blocks in front of these 32, and with them
    int behind;                                       // row blocks up to this lane's segment, it included
    __device__ __forceinline__ Segments() : before(0), upto(0) {}
    __device__ __forceinline__ void next(const Params& p, int lane) {
        first += 32;
        before = upto;
        const int seg = first + lane;
        bool bad = false;
        beg = len = 0;
        blocks = seg < p.nseq ? row_blocks(p, seg, beg, len, bad) : 0;
        if (bad) atomicOr(p.err, KVC_DEVERR_SEQLENS);
        behind = blocks;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int t = __shfl_up_sync(0xffffffffu, behind, o);
            if (lane >= o) behind += t;
        }
        behind += before;
        upto = __shfl_sync(0xffffffffu, behind, 31);
    }
};
// Item `index` (rising from one to the next, as CTAs are handed out; else the search begins anew): the head changes
// first, then the row block, from a segment's last one down (its key list is the longest).  The whole warp; every lane
// gets it.
__device__ __forceinline__ Item make_item(const Params& p, Segments& s, unsigned index, int lane) {
    Item it;
    const int block = static_cast<int>(index / static_cast<unsigned>(p.Hq));
    it.h = static_cast<int>(index - static_cast<unsigned>(block) * p.Hq);
    it.hk = it.h / p.G;
    if (block < s.before) s = Segments();
    while (block >= s.upto && s.first + 32 < p.nseq) s.next(p, lane);
    it.any = block < s.upto;
    if (!it.any) return it;
    const int who = __ffs(__ballot_sync(0xffffffffu, block < s.behind)) - 1;
    it.beg = __shfl_sync(0xffffffffu, s.beg, who);
    it.len = __shfl_sync(0xffffffffu, s.len, who);
    it.r0 = (__shfl_sync(0xffffffffu, s.behind, who) - 1 - block) * 2 * kRows;
    const bool two = it.r0 + kRows < it.len;
    const int nt0 = (min(it.len, it.r0 + kRows) + kKeys - 1) / kKeys, nt1 = (min(it.len, it.r0 + 2 * kRows) + kKeys - 1) / kKeys;
    // (tile A's keys end at nt0, and no window begins behind it: far0 <= near0 <= nt0)
    it.sink_tiles = min((p.sinks + kKeys - 1) / kKeys, nt0);
    it.far0 = max(max(0, it.r0 - p.window + 1) / kKeys, it.sink_tiles);
    it.near0 = two ? max(max(0, it.r0 + kRows - p.window + 1) / kKeys, it.sink_tiles) : it.far0;
    it.lead = it.near0 - it.far0;
    it.end[0] = it.lead + it.sink_tiles + nt0 - it.near0;
    it.end[1] = two ? it.lead + it.sink_tiles + nt1 - it.near0 : 0;
    it.entries = max(it.end[0], it.end[1]);
    // the sinks' last tile: no row has its window begin in it, and its second half holds no sink
    const int k0 = (it.sink_tiles - 1) * kKeys;
    it.narrow = it.sink_tiles > 0 && k0 + kKeys - 1 <= it.r0 - p.window && p.sinks <= k0 + kHalf ? it.lead + it.sink_tiles - 1 : -1;
    const int2 sinks = make_int2(0, it.sink_tiles * kKeys - (it.narrow >= 0 ? kHalf : 0));
    it.part[0][0] = make_int2(it.far0 * kKeys, it.near0 * kKeys);
    it.part[0][1] = it.part[1][1] = sinks;
    it.part[0][2] = make_int2(it.near0 * kKeys, nt0 * kKeys);
    it.part[1][0] = make_int2(0, 0);
    it.part[1][2] = make_int2(it.near0 * kKeys, two ? nt1 * kKeys : it.near0 * kKeys);
    return it;
}

// Ask for a CTA of this grid that has not started (16 bytes to `answer`, counted on the barrier); whether there was one,
// and its index.
__device__ __forceinline__ void ask_for_cta(void* answer, uint64_t* bar) {
    asm volatile("clusterlaunchcontrol.try_cancel.async.shared::cta.mbarrier::complete_tx::bytes.b128 [%0], [%1];" ::"r"(
                     smem_u32(answer)),
                 "r"(smem_u32(bar))
                 : "memory");
}
__device__ __forceinline__ bool got_cta(const void* answer, unsigned& index) {
    uint32_t yes, x;
    asm volatile(
        "{\n\t.reg .b128 h;\n\t.reg .pred p;\n\t"
        "ld.shared.b128 h, [%2];\n\t"
        "clusterlaunchcontrol.query_cancel.is_canceled.pred.b128 p, h;\n\t"
        "selp.u32 %0, 1, 0, p;\n\tmov.u32 %1, 0;\n\t"
        "@p clusterlaunchcontrol.query_cancel.get_first_ctaid::x.b32.b128 %1, h;\n\t}"
        : "=r"(yes), "=r"(x)
        : "r"(smem_u32(answer))
        : "memory");
    index = x;
    return yes != 0;
}

template <int D, bool kSplitP>
__global__ void __launch_bounds__(kThreads, 1) prefill_window_kernel(const __grid_constant__ CUtensorMap tmQ,
                                                                     const __grid_constant__ CUtensorMap tmK,
                                                                     const __grid_constant__ CUtensorMap tmV,
                                                                     const Params p) {
    using Geo = Geom<D>;
    constexpr int KS = Geo::kKStages, VS = Geo::kVStages;
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    uint64_t* bars = reinterpret_cast<uint64_t*>(smem + Geo::kBarOff);
    uint64_t* q_full = bars;            // the item's query rows landed
    uint64_t* q_empty = bars + 1;       // its S products done (one arrival per stream)
    uint64_t* k_full = bars + 2;        // [KS] K tile landed
    uint64_t* k_empty = k_full + KS;    // [KS] S products of the stage's tile done (one arrival per stream)
    uint64_t* v_full = k_empty + KS;    // [VS] V tile landed (and mended)
    uint64_t* v_empty = v_full + VS;    // [VS] P V products of the stage's tile done (one arrival per stream)
    uint64_t* s_full = v_empty + VS;    // [2][2] S of stream x's buffer i in TMEM (index 2 x + i)
    uint64_t* p_full = s_full + 4;      // [2][2] P of the buffer in TMEM (4 arrivals)
    uint64_t* o_full = p_full + 4;      // [2][2] P V of the buffer done
    uint64_t* fin = o_full + 4;         // [4] every product that a product warp issued is done
    uint64_t* v_land = fin + 4;         // a V tile that reaches past its segment landed (then mended)
    uint64_t* item_full = v_land + 1;             // [kSlots] the slot's item is described
    uint64_t* item_empty = item_full + kSlots;    // [kSlots] the other warps are done with it
    uint64_t* cta_full = item_empty + kSlots;     // the answer is there
    uint64_t* wanted = cta_full + 1;              // the last item's copies are all out
    uint32_t* s_tmem = reinterpret_cast<uint32_t*>(wanted + 1);
    volatile int* s_abort = reinterpret_cast<volatile int*>(s_tmem + 1);
    static_assert((2 + 2 * KS + 2 * VS + 17 + 2 * kSlots + 2) * 8 + 8 <= 512, "barrier area");
    Item* const s_item = reinterpret_cast<Item*>(smem + Geo::kItemOff);            // [kSlots], kItemBytes each
    void* const s_answer = smem + Geo::kItemOff + kSlots * kItemBytes;
    auto slot_item = [&](uint32_t slot) -> const Item& {
        return *reinterpret_cast<const Item*>(reinterpret_cast<const uint8_t*>(s_item) + slot * kItemBytes);
    };

    const int warp = __shfl_sync(0xffffffffu, static_cast<int>(threadIdx.x >> 5), 0), lane = threadIdx.x & 31;
    auto qs = [&](int x) { return smem + Geo::kQOff + x * Geo::kTileBytes; };
    auto kst = [&](uint32_t st) { return smem + Geo::kKOff + st * Geo::kTileBytes; };
    auto vst = [&](uint32_t st) { return smem + Geo::kVOff + st * Geo::kTileBytes; };

    if (threadIdx.x == 0) {
        mbar_init(q_full, 1);
        mbar_init(q_empty, 2);
        for (int i = 0; i < KS; ++i) {
            mbar_init(&k_full[i], 1);
            mbar_init(&k_empty[i], 2);
        }
        for (int i = 0; i < VS; ++i) {
            mbar_init(&v_full[i], 1);
            mbar_init(&v_empty[i], 2);
        }
        for (int i = 0; i < 4; ++i) {
            mbar_init(&s_full[i], 1);
            mbar_init(&p_full[i], 4);
            mbar_init(&o_full[i], 1);
            mbar_init(&fin[i], 1);
        }
        mbar_init(v_land, 1);
        for (int i = 0; i < kSlots; ++i) {
            mbar_init(&item_full[i], 1);
            mbar_init(&item_empty[i], kItemWarp);
        }
        mbar_init(cta_full, 1);
        mbar_init(wanted, 1);
        *s_abort = 0;
        fence_barrier_init();
    }
    if (warp == 0) {
        tmem_alloc(s_tmem, Geo::kTmemCols);
        tmem_relinquish();
    }
    if constexpr (Geo::kSumProduct) {
        for (int e = threadIdx.x; e < Geo::kOnesBytes / 16; e += kThreads)
            reinterpret_cast<uint4*>(smem + Geo::kOnesOff)[e] = make_uint4(0x3c003c00u, 0x3c003c00u, 0x3c003c00u, 0x3c003c00u);
        fence_proxy_async_smem();  // visible to the tensor cores (async proxy)
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *s_tmem;
    grid_dependency_wait();  // nothing is read or written before the kernel in front is done

    bool ok = true;
    uint32_t turn = 0;  // items so far: the next one is in slot turn % kSlots
    auto next_item = [&]() { return __all_sync(0xffffffffu, wait(&item_full[turn % kSlots], turn / kSlots & 1, s_abort)); };
    auto item_done = [&]() {  // the warp has read what it needs of the item
        __syncwarp();
        if (lane == 0) mbar_arrive(&item_empty[turn % kSlots]);
        ++turn;
    };
    if (warp == kItemWarp) {
        // ================= items =================
        Segments segments;
        unsigned index = blockIdx.x;
        bool more = true;
        for (int answers = 0; ok; ++answers) {
            Item it;
            it.any = 0;
            if (more) it = make_item(p, segments, index, lane);
            if (it.any || !more) {
                if (turn >= kSlots) ok = __all_sync(0xffffffffu, wait(&item_empty[turn % kSlots], (turn / kSlots - 1) & 1, s_abort));
                if (!ok) break;
                if (lane == 0) {
                    *reinterpret_cast<Item*>(reinterpret_cast<uint8_t*>(s_item) + turn % kSlots * kItemBytes) = it;
                    mbar_arrive(&item_full[turn % kSlots]);
                }
                __syncwarp();
                // no item is taken over before the last one's copies are all out: others may have nothing left
                if (more) ok = __all_sync(0xffffffffu, wait(wanted, turn & 1, s_abort));
                ++turn;
            }
            if (!more || !ok) break;
            if (lane == 0) {
                mbar_arrive_expect_tx(cta_full, 16);
                ask_for_cta(s_answer, cta_full);
            }
            __syncwarp();
            const bool there = __all_sync(0xffffffffu, mbar_wait_bounded(cta_full, answers & 1, kWaitNs));
            more = there && got_cta(s_answer, index);
            if (!there) *s_abort = 1;
            fence_proxy_async_smem();  // the answer is read before the next one is written
            __syncwarp();
        }
        // the segments behind the last item are looked at too, for their errors, by one CTA
        if (blockIdx.x == 0)
            while (segments.first + 32 < p.nseq) segments.next(p, lane);
    } else if (warp >= kLoadKWarp) {
        // ================= copies: Q and K by one warp, V by the other, as far ahead as the rings allow =================
        const bool is_v = warp == kLoadVWarp;
        uint64_t* const full = is_v ? v_full : k_full;
        uint64_t* const empty = is_v ? v_empty : k_empty;
        const CUtensorMap* const map = is_v ? &tmV : &tmK;
        const uint32_t stages = is_v ? VS : KS;
        uint32_t st = 0, ph = 0;  // stage and use of the next tile
        int done = 0, mended = 0;
        if (lane == 0) {
            if (!is_v) prefetch_tensormap(&tmQ);
            prefetch_tensormap(map);
        }
        for (;; item_done()) {
            ok = ok && next_item();
            if (!ok) break;
            const Item it = slot_item(turn % kSlots);
            if (!it.any) break;
            if (!is_v) {
                if (done > 0) ok = __all_sync(0xffffffffu, wait(q_empty, (done - 1) & 1, s_abort));
                if (!ok) break;
                const int tiles = it.end[1] > 0 ? 2 : 1;
                if (lane == 0) {
                    mbar_arrive_expect_tx(q_full, tiles * Geo::kTileBytes);
                    for (int x = 0; x < tiles; ++x)
#pragma unroll
                        for (int c = 0; c < Geo::kChunks; ++c)
                            tma_load_3d(qs(x) + c * Geo::kChunkBytes, &tmQ, q_full, c * 64, it.h, it.beg + it.r0 + x * kRows);
                }
                __syncwarp();
            }
            ++done;
            for (int j = 0; j < it.entries; ++j) {
                if (ph > 0) ok = __all_sync(0xffffffffu, wait(&empty[st], (ph - 1) & 1, s_abort));
                if (!ok) break;
                const int k0 = it.key_tile(j) * kKeys;
                // V rows past the segment (the next one's) are zeroed, so that whatever they hold cannot reach an output
                // through a zero weight
                const bool mend = is_v && k0 + kKeys > it.len;
                uint8_t* const tile = is_v ? vst(st) : kst(st);
                if (lane == 0) {
                    uint64_t* const bar = mend ? v_land : &full[st];
                    mbar_arrive_expect_tx(bar, Geo::kTileBytes);
#pragma unroll
                    for (int c = 0; c < Geo::kChunks; ++c)
                        tma_load_3d(tile + c * Geo::kChunkBytes, map, bar, c * 64, it.hk, it.beg + k0);
                }
                __syncwarp();
                if (mend) {
                    ok = __all_sync(0xffffffffu, wait(v_land, mended & 1, s_abort));
                    if (!ok) break;
                    ++mended;
                    const int from = it.len - k0;
                    for (int e = lane; e < (kKeys - from) * 8 * Geo::kChunks; e += 32) {
                        const int r = from + e / (8 * Geo::kChunks), rest = e % (8 * Geo::kChunks);
                        *reinterpret_cast<uint4*>(tile + (rest / 8) * Geo::kChunkBytes + sw128(r, rest % 8)) =
                            make_uint4(0u, 0u, 0u, 0u);
                    }
                    fence_proxy_async_smem();  // visible to the tensor cores (async proxy)
                    __syncwarp();
                    if (lane == 0) mbar_arrive(&full[st]);
                }
                if (++st == stages) {
                    st = 0;
                    ++ph;
                }
            }
            if (!is_v && lane == 0) mbar_arrive(wanted);
        }
        // copies still in flight land before the shared memory is released (immediate unless aborted: the products
        // consumed every tile)
        if (lane == 0 && !ok) {
            if (!is_v && done > 0) mbar_wait_bounded(q_full, (done - 1) & 1, kWaitNs / 8);
            for (uint32_t s = 0; s < stages; ++s) {
                const uint32_t uses = ph + (s < st ? 1 : 0);  // of stage s
                if (uses > 0) mbar_wait_bounded(&full[s], (uses - 1) & 1, kWaitNs / 8);
            }
            if (is_v) mbar_wait_bounded(v_land, mended & 1, kWaitNs / 8);
        }
    } else if (warp >= kSWarp) {
        // ================= products: a warp per stream and product =================
        const int x = (warp - kSWarp) & 1;
        uint32_t st = 0, ph = 0;  // stage and use of the entry's tile
        int uc = 0, done = 0;     // units and items so far
        if (warp < kPvWarp) {
            constexpr uint32_t idS = umma_idesc_f16(kRows, kHalf, 0, 0);
            const uint64_t dQ = umma_smem_desc(smem_u32(qs(x)), 16, 1024);
            const uint64_t dK = umma_smem_desc(smem_u32(kst(0)), 16, 1024);
            for (;; item_done()) {
                ok = ok && next_item();
                if (!ok) break;
                const Item it = slot_item(turn % kSlots);
                if (!it.any) break;
                ok = wait_all(q_full, done & 1, s_abort);
                if (!ok) break;
                ++done;
                const int first = it.begin(x), end = it.end[x];
                for (int j = 0; j < it.entries; ++j) {
                    ok = wait_all(&k_full[st], ph & 1, s_abort);
                    if (!ok) break;
                    if (j >= first && j < end) {
                        const int units = it.units(j);
                        for (int half = 0; half < units; ++half, ++uc) {
                            const int buf = 2 * x + (uc & 1);
                            // the buffer's P of two units ago has been read
                            if (uc >= 2) ok = wait_all(&o_full[buf], ((uc - 2) >> 1) & 1, s_abort);
                            if (!ok) break;
                            tc_fence_after();
                            const uint64_t b0 = dK + static_cast<uint64_t>((st * Geo::kTileBytes + half * kHalf * 128) >> 4);
                            const uint32_t tS = tmem + buf * kHalf;
                            if (elect_one()) {
#pragma unroll
                                for (int i = 0; i < D / 16; ++i) {
                                    const int c = i >> 2, kk = i & 3;
                                    umma_f16_ss(tS, dQ + ((c * Geo::kChunkBytes + kk * 32) >> 4),
                                                b0 + ((c * Geo::kChunkBytes + kk * 32) >> 4), idS, i > 0);
                                }
                                umma_commit(&s_full[buf]);
                                if (half == units - 1) {
                                    umma_commit(&k_empty[st]);
                                    if (j == end - 1) umma_commit(q_empty);
                                }
                            }
                            __syncwarp();
                        }
                        if (!ok) break;
                    } else if (lane == 0) {
                        mbar_arrive(&k_empty[st]);  // not this stream's
                    }
                    if (++st == KS) {
                        st = 0;
                        ++ph;
                    }
                }
                if (ok && end == 0 && lane == 0) mbar_arrive(q_empty);  // a stream without rows
            }
        } else {
            // O_X += P V: 4 steps of 16 keys, P from TMEM (fp16, or its high part and residual); V as the MN-major B
            // operand: 8-key groups 1024 bytes apart, 64-dim atoms one chunk apart
            constexpr uint32_t idPV = umma_idesc_f16(kRows, D, 0, 1);
            const uint64_t dV = umma_smem_desc(smem_u32(vst(0)), Geo::kChunkBytes, 1024);
            const uint32_t tO = tmem + Geo::kTmemO + x * D, tL = tmem + Geo::kTmemL + x * 64;
            const uint64_t dOnes = umma_smem_desc(smem_u32(smem + Geo::kOnesOff), Geo::kChunkBytes, 1024);
            for (;; item_done()) {
                ok = ok && next_item();
                if (!ok) break;
                const Item it = slot_item(turn % kSlots);
                if (!it.any) break;
                const int first = it.begin(x), end = it.end[x];
                for (int j = 0; j < it.entries; ++j) {
                    ok = wait_all(&v_full[st], ph & 1, s_abort);
                    if (!ok) break;
                    if (j >= first && j < end) {
                        const int units = it.units(j);
                        for (int half = 0; half < units; ++half, ++uc) {
                            const int buf = 2 * x + (uc & 1);
                            ok = wait_all(&p_full[buf], (uc >> 1) & 1, s_abort);
                            if (!ok) break;
                            tc_fence_after();
                            const uint64_t v0 = dV + static_cast<uint64_t>((st * Geo::kTileBytes + half * kHalf * 128) >> 4);
                            const uint32_t tP = tmem + buf * kHalf;
                            const bool more = j > first || half > 0;  // O holds something of this item
                            if (elect_one()) {
#pragma unroll
                                for (int kk = 0; kk < kHalf / 16; ++kk) {
                                    const uint64_t bd = v0 + ((kk * 2048) >> 4);
                                    umma_f16_ts(tO, tP + kk * 8, bd, idPV, (more || kk > 0) ? 1u : 0u);
                                    if constexpr (kSplitP) umma_f16_ts(tO, tP + kHalf / 2 + kk * 8, bd, idPV, 1u);
                                }
                                if constexpr (Geo::kSumProduct) {
#pragma unroll
                                    for (int kk = 0; kk < kHalf / 16; ++kk) {
                                        const uint64_t bd = dOnes + ((kk * 2048) >> 4);
                                        umma_f16_ts(tL, tP + kk * 8, bd, idPV, (more || kk > 0) ? 1u : 0u);
                                        if constexpr (kSplitP) umma_f16_ts(tL, tP + kHalf / 2 + kk * 8, bd, idPV, 1u);
                                    }
                                }
                                umma_commit(&o_full[buf]);
                                if (half == units - 1) umma_commit(&v_empty[st]);
                            }
                            __syncwarp();
                        }
                        if (!ok) break;
                    } else if (lane == 0) {
                        mbar_arrive(&v_empty[st]);  // not this stream's
                    }
                    if (++st == VS) {
                        st = 0;
                        ++ph;
                    }
                }
            }
        }
        // every product issued is complete before the tensor memory is released
        __syncwarp();
        if (elect_one()) umma_commit(&fin[warp - kSWarp]);
        __syncwarp();
        mbar_wait_bounded(&fin[warp - kSWarp], 0, kWaitNs);
        if (!ok && lane == 0) atomicOr(p.err, KVC_DEVERR_TIMEOUT);
    } else {
        // ================= row warps: softmax and output; thread = query row = TMEM lane =================
        const int x = warp / 4, wq = warp & 3;
        const uint32_t lane_base = static_cast<uint32_t>(wq * 32) << 16;
        const uint32_t tO = tmem + Geo::kTmemO + x * D + lane_base, tL = tmem + Geo::kTmemL + x * 64 + lane_base;
        const float sl2 = p.scale_log2;
        const uint64_t sc2 = pack_f32x2(sl2, sl2);
        int uc = 0;  // units so far
        for (;; item_done()) {
            ok = ok && next_item();
            if (!ok) break;
            const Item& it = slot_item(turn % kSlots);
            if (!it.any) break;
            if (it.end[x] == 0) continue;
            const int rx = it.r0 + x * kRows;           // first row of the row tile
            const int qi = rx + wq * 32 + lane;         // row of the segment
            const int keys_end = min(qi + 1, it.len);  // of this row
            float m_used = -INFINITY, l = 0.f;
            bool far = false;  // some row of the warp has its m beyond kFar
            // The list's three stretches of keys, a unit at a time; what an item says is read where one ends, not for
            // every unit (a unit's loads from shared memory and what hung on them were 300 of its 1600 clocks)
            const int uc0 = uc;
            int part = x, k0 = 0, stop = 0;  // k0: the unit's first key
            auto next_part = [&]() {
                while (k0 == stop && part < 3) {
                    const int2 keys = it.part[x][part++];
                    k0 = keys.x;
                    stop = keys.y;
                }
                return k0 != stop;
            };
            for (bool left = next_part(); left; ++uc) {
                const int buf = 2 * x + (uc & 1);
                const uint32_t tS = tmem + buf * kHalf + lane_base;
                // units that every row of the tile sees need no mask
                const bool masked = k0 + kHalf - 1 > rx || (k0 <= rx + kRows - 1 - p.window && k0 + kHalf > p.sinks);
                uint32_t bits[2] = {~0u, ~0u};
                if (masked) {
                    bits[0] = window_bits(qi, k0, keys_end, p.window, p.sinks);
                    bits[1] = window_bits(qi, k0 + 32, keys_end, p.window, p.sinks);
                }
                ok = wait_warp(&s_full[buf], (uc >> 1) & 1, s_abort);
                if (!ok) break;
                tc_fence_after();
                if (masked && !__any_sync(0xffffffffu, (bits[0] | bits[1]) != 0)) {  // nothing for these 32 rows
                    float zero[32] = {};
                    tmem_st32(tS, zero);
                    if constexpr (kSplitP) tmem_st32(tS + 32, zero);
                } else {
                    float s[kHalf];
                    tmem_ld64(tS, s);
                    if (masked || p.negate) {
                        if (p.negate) {
#pragma unroll
                            for (int c = 0; c < kHalf; ++c) s[c] = -s[c];
                        }
                        mask_scores(s, bits, -INFINITY);
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
                    const bool moves = mx > m_used + kRescaleLog2;  // includes the first finite max (m_used = -inf)
                    if (__any_sync(0xffffffffu, moves)) {
                        const float m_new = moves ? __fsub_rd(mx, kWeightLog2) : m_used;
                        // (a row that had seen nothing has no weights in O and its sum)
                        const bool grows = moves && m_used != -INFINITY;
                        const float alpha = grows ? ex2(m_used - m_new) : 1.f;
                        m_used = m_new;
                        l *= alpha;
                        if constexpr (kSplitP) far = __any_sync(0xffffffffu, fabsf(m_used) >= kFar && m_used != -INFINITY);
                        // rescale O_X, which idles once the stream's previous product is complete (this unit's P is not
                        // there yet)
                        if (uc != uc0 && __any_sync(0xffffffffu, grows)) {
                            ok = __all_sync(0xffffffffu, wait(&o_full[buf ^ 1], ((uc - 1) >> 1) & 1, s_abort));
                            if (!ok) break;
                            tc_fence_after();
#pragma unroll 1
                            for (int c = 0; c < D; c += 32) {
                                float o[32];
                                tmem_ld32(tO + c, o);
#pragma unroll
                                for (int i = 0; i < 32; ++i) o[i] *= alpha;
                                tmem_st32(tO + c, o);
                            }
                            if constexpr (Geo::kSumProduct) {  // (the one column that is read)
                                float sum[4];
                                tmem_ld4(tL, sum);
#pragma unroll
                                for (int i = 0; i < 4; ++i) sum[i] *= alpha;
                                tmem_st4(tL, sum);
                            }
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
                                if (!Geo::kSumProduct) ls[i & 3] += x0 + x1;
                            } else if (!Geo::kSumProduct) {
                                ls[i & 3] = add_halves(hv[i], ls[i & 3]);
                            }
                        }
                        tmem_st16(tS + hh * 16, hv);
                        if constexpr (kSplitP) tmem_st16(tS + kHalf / 2 + hh * 16, lv);
                    }
                    if (!Geo::kSumProduct) l += (ls[0] + ls[1]) + (ls[2] + ls[3]);
                }
                tmem_wait_st();
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(&p_full[buf]);
                k0 += kHalf;
                left = k0 != stop || next_part();
            }
            if (ok) ok = __all_sync(0xffffffffu, wait(&o_full[2 * x + ((uc - 1) & 1)], ((uc - 1) >> 1) & 1, s_abort));
            if (!ok) break;
            tc_fence_after();
            if constexpr (Geo::kSumProduct) {
                float sum[4];
                tmem_ld4(tL, sum);
                l = sum[0];
            }
            const float inv = l > 0.f ? 1.f / l : 0.f;
            const int64_t row0 = (static_cast<int64_t>(it.beg + qi) * p.Hq + it.h) * D;
#pragma unroll 1
            for (int c = 0; c < D; c += 32) {
                float o[32];
                tmem_ld32(tO + c, o);
                if (qi < it.len) {
                    if (p.out_f32) {
                        float* dst = static_cast<float*>(p.out) + row0 + c;
#pragma unroll
                        for (int i = 0; i < 4; ++i) {
                            uint32_t w[8];
#pragma unroll
                            for (int k = 0; k < 8; ++k) w[k] = __float_as_uint(o[8 * i + k] * inv);
                            store_32(dst + 8 * i, w, p.out_wide);
                        }
                    } else {
                        __half* dst = static_cast<__half*>(p.out) + row0 + c;
#pragma unroll
                        for (int i = 0; i < 2; ++i) {
                            uint32_t w[8];
#pragma unroll
                            for (int k = 0; k < 8; ++k) w[k] = pack_half2(o[16 * i + 2 * k] * inv, o[16 * i + 2 * k + 1] * inv);
                            store_32(dst + 16 * i, w, p.out_wide);
                        }
                    }
                }
                float t = 0.f;
#pragma unroll
                for (int i = 0; i < 32; ++i) t = fmaf(o[i], 0.f, t);  // NaN if any is infinite or NaN
                unsigned again = __ballot_sync(0xffffffffu, qi < it.len && !(t == 0.f && l < INFINITY));
                for (; again != 0; again &= again - 1) {
                    const int i = rx + wq * 32 + __ffs(again) - 1;
                    const int64_t kv_stride = static_cast<int64_t>(p.Hkv) * D, kv0 = it.beg * kv_stride + it.hk * D;
                    const int64_t at = (static_cast<int64_t>(it.beg + i) * p.Hq + it.h) * D;
                    const float r = window_row_again<D>(p.q + at, p.k + kv0, p.v + kv0, kv_stride, i, p.window, p.sinks,
                                                        p.negate ? -sl2 : sl2, c);
                    __syncwarp();
                    if (p.out_f32)
                        static_cast<float*>(p.out)[at + c + lane] = r;
                    else
                        static_cast<__half*>(p.out)[at + c + lane] = __float2half_rn(r);
                }
            }
            tc_fence_before();  // O is read before the next item's products (behind this warp's next arrival) write it
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
}

// [T][H][D] fp16 viewed as (dim, head, token); boxes of 64 dims x 1 head x 128 tokens, 128-byte swizzle
static cudaError_t make_packed_map(CUtensorMap* map, const void* base, int D, int H, int T) {
    EncodeTiledFn fn = encode_fn();
    if (!fn) return cudaErrorNotSupported;
    cuuint64_t gdim[3] = {static_cast<cuuint64_t>(D), static_cast<cuuint64_t>(H), static_cast<cuuint64_t>(T)};
    cuuint64_t gstride[2] = {static_cast<cuuint64_t>(D) * 2, static_cast<cuuint64_t>(H) * D * 2};
    cuuint32_t box[3] = {64, 1, 128};
    cuuint32_t estr[3] = {1, 1, 1};
    CUresult r = fn(map, CU_TENSOR_MAP_DATA_TYPE_FLOAT16, 3, const_cast<void*>(base), gdim, gstride, box, estr,
                    CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                    CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    return r == CUDA_SUCCESS ? cudaSuccess : cudaErrorInvalidValue;
}

template <int D, bool kSplitP>
static cudaError_t launch_d(const PrefillArgs& a, cudaStream_t stream) {
    using Geo = Geom<D>;
    static std::once_flag attr_once;
    static cudaError_t attr_err = cudaSuccess;
    std::call_once(attr_once, [] {
        attr_err = cudaFuncSetAttribute(prefill_window_kernel<D, kSplitP>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                        Geo::kSmemBytes);
    });
    if (attr_err != cudaSuccess) return attr_err;
    CUtensorMap tq, tk, tv;
    cudaError_t e = make_packed_map(&tq, a.q, D, a.Hq, a.total_tokens);
    if (e == cudaSuccess) e = make_packed_map(&tk, a.k, D, a.Hkv, a.total_tokens);
    if (e == cudaSuccess) e = make_packed_map(&tv, a.v, D, a.Hkv, a.total_tokens);
    if (e != cudaSuccess) return e;
    Params p;
    p.cu_seqlens = a.cu_seqlens;
    p.q = a.q;
    p.k = a.k;
    p.v = a.v;
    p.out = a.out;
    p.err = a.err;
    p.nseq = a.nseq;
    p.total_tokens = a.total_tokens;
    p.tiles_per_seq = (a.max_seqlen + 2 * kRows - 1) / (2 * kRows);
    p.Hq = a.Hq;
    p.Hkv = a.Hkv;
    p.G = a.Hq / a.Hkv;
    p.out_f32 = a.out_f32;
    p.window = a.window;
    p.sinks = a.sinks;
    p.negate = a.scale < 0.f;
    p.out_wide = reinterpret_cast<uintptr_t>(a.out) % 32 == 0;
    p.scale_log2 = std::max(std::min(std::fabs(a.scale) * kLog2e, 3.4e38f), kMinWindowScaleLog2);
    // no more row blocks than max_seqlen allows, nor than the tokens fill, one of each segment in part
    const int64_t blocks = std::min<int64_t>(static_cast<int64_t>(p.tiles_per_seq) * a.nseq,
                                             a.total_tokens / (2 * kRows) + static_cast<int64_t>(a.nseq));
    const int64_t items = blocks * a.Hq;
    if (items > 2147483647LL) return cudaErrorInvalidConfiguration;
    return launch(prefill_window_kernel<D, kSplitP>, dim3(static_cast<unsigned>(items)), dim3(kThreads), Geo::kSmemBytes, stream, true, 1u, tq, tk,
                  tv, p);
}

}  // namespace pfw

cudaError_t launch_prefill_window(const PrefillArgs& a, cudaStream_t stream) {
    using namespace pfw;
    if (a.nseq <= 0 || a.total_tokens <= 0 || a.max_seqlen <= 0) return cudaSuccess;
    if (a.D == 64) return a.split_p ? launch_d<64, true>(a, stream) : launch_d<64, false>(a, stream);
    if (a.D == 128) return a.split_p ? launch_d<128, true>(a, stream) : launch_d<128, false>(a, stream);
    return cudaErrorInvalidValue;
}

}  // namespace kvc
