// Block tables, slots and positions of a step, built on the GPU from the request lengths.
//
// Sequence b goes from before_b to after_b tokens.  Its blocks j in [ceil(before / 16), ceil(after / 16)) are new; with
// a window they are used in turn: behind the first ns + R (ns blocks of sinks, R that a window is ever in) block j lies
// where block j - R lay, place(j) = ns + (j - ns) mod R, else place(j) = j.  So the sequence takes
//   need_b = min(ceil(after / 16), ns + R) - min(ceil(before / 16), ns + R)
// blocks from the list, those of sequence b behind those of the sequences before it, and block j is the list's entry
// for its place where the sequence did not hold that place before, else what the table has there.  Token t of the
// step, at position pos, gets slot table[pos / 16] * 16 + pos % 16, or -1 where a later block of the same step lies in
// its place (no later query sees it).
//
// Every CTA forms the prefix sums of tokens and blocks over all sequences by itself (a thread some consecutive ones,
// then a scan over the threads) and knows from the totals whether the step fits, so that one launch without any
// exchange is all or nothing; then it takes a share of the tokens, finds each one's sequence by bisection, and writes
// its slot and position, and the token that starts a block also the table's entry.  Bound by launch and dependent loads,
// not by bytes: 256 sequences' next tokens take 2.3 us, 128 prompts of up to 8192 tokens 5.4 (where their slots and
// entries alone would be 1.1): the sums, then for each token a bisection and two loads that follow one another (its
// sequence's lengths are kept with the sums: read again they were 0.35 us more).
#include "../../include/kvc.h"
#include "decode_common.cuh"
#include "kvc_internal.h"

namespace kvc {
namespace tables {

struct Params {
    const int32_t* before;  // null: zeros
    const int32_t* after;
    const int32_t* free_blocks;
    const int32_t* placed;
    int32_t* table;
    int32_t* new_placed;
    int32_t* cu_tokens;
    int64_t* slots;
    int32_t* positions;  // null: not asked for
    unsigned* err;
    int B, num_free, max_blocks, num_slots, per;  // per: sequences of a thread's sums
    int first, ring;  // blocks of sinks; blocks a window goes through (ring 0: no window)
};

struct Seq {
    int before, count;  // tokens
    int nb0, nb1;       // blocks before and after
    int had, need;      // distinct blocks before, and how many the step adds
};

__device__ __forceinline__ Seq make_seq(const Params& p, int before, int count) {
    const int after = before + count;
    Seq s;
    s.before = before;
    s.count = count;
    s.nb0 = (s.before + kBlockSize - 1) / kBlockSize;
    s.nb1 = (after + kBlockSize - 1) / kBlockSize;
    const int most = p.ring > 0 ? p.first + p.ring : p.max_blocks;
    s.had = min(s.nb0, most);
    s.need = min(s.nb1, most) - s.had;
    return s;
}
__device__ __forceinline__ Seq load_seq(const Params& p, int b, bool* bad) {
    int before = p.before != nullptr ? p.before[b] : 0, after = p.after[b];
    if (before < 0 || after < before || after > p.max_blocks * kBlockSize) {  // (max_blocks * 16 is below 2^31)
        *bad = true;
        before = after = 0;
    }
    return make_seq(p, before, after - before);
}

// The sums of many sequences want many threads, for few a CTA of fewer starts sooner: with 128 / 512 threads, in us, 256
// sequences' next tokens 2.3 / 2.7, 128 prompts of up to 8192 tokens 5.4 / 6.2, the next tokens of 1024 sequences 3.5 /
// 3.3, of 4096 17.9 / 6.7.
template <int kThreads>
__global__ void __launch_bounds__(kThreads) kv_block_tables_kernel(const Params p) {
    constexpr int kWarps = kThreads / 32;
    __shared__ int s_tok[kThreads], s_need[kThreads];  // sums before each thread's sequences
    __shared__ int64_t s_warp[2][kWarps];
    __shared__ int2 s_lens[kThreads];  // lengths of each thread's first sequence, before and new
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    grid_dependency_wait();  // nothing is read or written before the kernel in front is done
    const int placed = *p.placed;
    const int b0 = min(p.B, tid * p.per), b1 = min(p.B, b0 + p.per);
    int64_t tok = 0, need = 0;
    bool bad = false;
    for (int b = b0; b < b1; ++b) {
        const Seq s = load_seq(p, b, &bad);
        tok += s.count;
        need += s.need;
        if (b == b0) s_lens[tid] = make_int2(s.before, s.count);
    }
    int64_t tok_in = tok, need_in = need;  // inclusive sums
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int64_t t = __shfl_up_sync(0xffffffffu, tok_in, o), n = __shfl_up_sync(0xffffffffu, need_in, o);
        if (lane >= o) {
            tok_in += t;
            need_in += n;
        }
    }
    if (lane == 31) {
        s_warp[0][warp] = tok_in;
        s_warp[1][warp] = need_in;
    }
    __syncthreads();
    int64_t all_tok = 0, all_need = 0;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) {
        if (w == warp) {
            tok_in += all_tok;
            need_in += all_need;
        }
        all_tok += s_warp[0][w];
        all_need += s_warp[1][w];
    }
    const bool fits = placed >= 0 && placed <= p.num_free && all_need <= p.num_free - placed && all_tok <= p.num_slots;
    const int total = fits ? static_cast<int>(all_tok) : 0;
    s_tok[tid] = fits ? static_cast<int>(tok_in - tok) : 0;
    s_need[tid] = fits ? static_cast<int>(need_in - need) : 0;
    if (blockIdx.x == 0) {
        if (bad) atomicOr(p.err, KVC_DEVERR_CONTEXT);
        if (tid == 0) {
            if (!fits) atomicOr(p.err, KVC_DEVERR_BLOCKS);
            *p.new_placed = fits ? placed + static_cast<int>(all_need) : placed;
            p.cu_tokens[0] = 0;
        }
        int64_t at = tok_in - tok;
        for (int b = b0; b < b1; ++b) {
            at += load_seq(p, b, &bad).count;
            p.cu_tokens[b + 1] = fits ? static_cast<int>(at) : 0;
        }
    }
    __syncthreads();
    for (int64_t t64 = static_cast<int64_t>(blockIdx.x) * kThreads + tid; t64 < p.num_slots;
         t64 += static_cast<int64_t>(gridDim.x) * kThreads) {
        const int t = static_cast<int>(t64);
        int64_t slot = -1;
        int pos = 0;
        if (t < total) {
            // the last thread whose sequences begin at or before token t (one without tokens never is)
            int lo = 0;
#pragma unroll
            for (int step = kThreads / 2; step > 0; step >>= 1)
                if (s_tok[lo + step] <= t) lo += step;
            int b = lo * p.per, from = s_tok[lo], taken = s_need[lo];
            Seq s = make_seq(p, s_lens[lo].x, s_lens[lo].y);
            while (from + s.count <= t) {
                from += s.count;
                taken += s.need;
                s = load_seq(p, ++b, &bad);
            }
            pos = s.before + t - from;
            const int j = pos / kBlockSize;
            int32_t* const row = p.table + static_cast<int64_t>(b) * p.max_blocks;
            const bool kept = p.ring == 0 || j < p.first || j >= s.nb1 - p.ring;
            if (kept || pos % kBlockSize == 0) {
                int block;
                if (j < s.nb0) {
                    block = row[j];  // the block that the sequence's last token before lies in
                } else {
                    const int place = p.ring > 0 && j >= p.first + p.ring ? p.first + (j - p.first) % p.ring : j;
                    block = place < s.had ? row[place] : p.free_blocks[placed + taken + place - s.had];
                    if (pos % kBlockSize == 0) row[j] = block;
                }
                if (kept && block >= 0) slot = static_cast<int64_t>(block) * kBlockSize + pos % kBlockSize;
            }
        }
        p.slots[t] = slot;
        if (p.positions != nullptr) p.positions[t] = pos;
    }
}

// (1024 threads on an SM: with 512 a token's dependent loads show, with 1536 the sums that every CTA forms do)
template <int kThreads>
static cudaError_t launch_threads(Params& p, cudaStream_t stream) {
    p.per = std::max(1, (p.B + kThreads - 1) / kThreads);
    const int64_t want = (static_cast<int64_t>(p.num_slots) + kThreads - 1) / kThreads;
    const int grid = static_cast<int>(std::max<int64_t>(1, std::min<int64_t>(want, 1024 / kThreads * sm_count())));
    return launch(kv_block_tables_kernel<kThreads>, dim3(grid), dim3(kThreads), 0, stream, true, 1u, p);
}

}  // namespace tables

cudaError_t launch_block_tables(const BlockTableArgs& a, cudaStream_t stream) {
    if (sm_count() <= 0) return cudaErrorNoDevice;
    tables::Params p;
    p.before = a.lens_before;
    p.after = a.lens_after;
    p.free_blocks = a.free_blocks;
    p.placed = a.placed;
    p.table = a.block_table;
    p.new_placed = a.new_placed;
    p.cu_tokens = a.cu_tokens;
    p.slots = a.slots;
    p.positions = a.positions;
    p.err = a.err;
    p.B = a.B;
    p.num_free = a.num_free;
    p.max_blocks = a.max_blocks;
    p.num_slots = a.num_slots;
    p.first = a.window > 0 ? (a.sinks + kBlockSize - 1) / kBlockSize : 0;
    p.ring = a.window > 0 ? (a.window + 2 * kBlockSize - 2) / kBlockSize : 0;
    return a.B <= 512 ? tables::launch_threads<128>(p, stream) : tables::launch_threads<512>(p, stream);
}

}  // namespace kvc
