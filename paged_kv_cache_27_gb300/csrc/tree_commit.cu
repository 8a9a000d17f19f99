// The kept path of a drafted tree, moved to the end of its sequence's context.
//
// A tree's nodes sit in the cache at positions base .. base + tree_len - 1 (base = context length - tree length) in
// node order; the nodes of the kept path 0 = n_0 < n_1 < ... belong at base, base + 1, ...  For every layer, K and V
// and KV head: row[base + i] = row[base + n_i], bit for bit, and the new context length is base + path length.
//
// In place: n_i >= i, and row base + i is written after every source with a smaller index was read and is no source of
// a later one (n_j >= j > i), so rows moved in path order in batches (all loads of a batch before its stores) never
// read an overwritten row.  A warp takes one layer's K or V of one sequence and some of its KV heads; rows are 16-byte
// chunks over the lanes.  The work is a few KB per sequence and layer: the kernel is bound by the latency of its
// dependent loads (lengths and path, block table, rows) and the number of warps it is spread over.
#include "../../include/kvc.h"
#include "decode_common.cuh"
#include "kvc_internal.h"

namespace kvc {
namespace commit {

constexpr int kWarps = 4;

struct Params {
    uint4* k_pool;       // [L][NB][Hkv][16][D]
    uint4* v_pool;
    int64_t layer_u4;    // 16-byte chunks per layer
    const int32_t* block_table;
    const int32_t* context_lens;
    const int32_t* tree_lens;
    const int32_t* path;
    const int32_t* path_len;
    int32_t* new_context_lens;
    unsigned* err;
    int num_blocks, max_blocks, P, L, Hkv, chunks, heads_per_warp, head_parts;  // chunks: 16-byte chunks of a row
};

__global__ void __launch_bounds__(kWarps * 32) kv_tree_commit_kernel(const Params p) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, b = blockIdx.y;
    const int w = blockIdx.x * kWarps + warp;  // (layer, K or V, part of the heads)
    __shared__ int2 s_move[kWarps][kMaxTreeNodes];  // (from, to): block * 16 + offset of the rows that move
    grid_dependency_wait();  // nothing is read or written before the kernel in front is done
    if (w >= p.L * 2 * p.head_parts) return;  // whole warps
    const int part = w % p.head_parts, kv = (w / p.head_parts) & 1, layer = w / p.head_parts / 2;
    const bool first = w == 0;
    const int ctx = p.context_lens[b], tree = p.tree_lens != nullptr ? p.tree_lens[b] : p.P, len = p.path_len[b];
    const int base = ctx - tree;
    const int32_t* row = p.block_table + static_cast<int64_t>(b) * p.max_blocks;
    bool ok = tree >= 0 && base >= 0 && ctx <= static_cast<int64_t>(p.max_blocks) * kBlockSize && len >= 0 &&
              len <= p.P && len <= tree && tree <= kMaxTreeNodes;
    int moves = 0;
    if (ok) {
        bool good = true;
        bool bad_block = false;
        for (int i0 = 0; i0 < len; i0 += 32) {
            const int i = i0 + lane;
            int node = i, prev = i - 1;
            if (i < len) {
                node = p.path[static_cast<int64_t>(b) * p.P + i];
                if (i > 0) prev = p.path[static_cast<int64_t>(b) * p.P + i - 1];
                good = good && (i > 0 ? node > prev : node == 0) && node >= i && node < tree;
            }
            const bool mv = i < len && good && node != i;
            int2 m = make_int2(0, 0);
            if (mv) {
                const int from = base + node, to = base + i;
                const int fb = row[from / kBlockSize], tb = row[to / kBlockSize];
                if (fb < 0 || fb >= p.num_blocks || tb < 0 || tb >= p.num_blocks) bad_block = true;
                m = make_int2(fb * kBlockSize + from % kBlockSize, tb * kBlockSize + to % kBlockSize);
            }
            const unsigned who = __ballot_sync(0xffffffffu, mv);
            if (mv) s_move[warp][moves + __popc(who & ((1u << lane) - 1u))] = m;
            moves += __popc(who);
        }
        bad_block = __any_sync(0xffffffffu, bad_block);
        ok = __all_sync(0xffffffffu, good) && !bad_block;
        if (bad_block && first && lane == 0) atomicOr(p.err, KVC_DEVERR_BLOCK_ID);
        if (!ok && !bad_block && first && lane == 0) atomicOr(p.err, KVC_DEVERR_TREE);
    } else if (first && lane == 0) {
        atomicOr(p.err, KVC_DEVERR_CONTEXT);
    }
    if (first && lane == 0) p.new_context_lens[b] = ok ? base + len : ctx;
    if (!ok) return;  // the sequence is left as it was
    __syncwarp();
    uint4* pool = (kv ? p.v_pool : p.k_pool) + layer * p.layer_u4;
    const int h0 = part * p.heads_per_warp, nh = min(p.heads_per_warp, p.Hkv - h0);
    const int per_row = nh * p.chunks, total = moves * per_row;
    constexpr int U = 4;
    const int shift = p.chunks == 16 ? 4 : 3;  // chunks of a row: 8 or 16
    for (int e0 = 0; e0 < total; e0 += 32 * U) {
        uint4 x[U];
        int to[U];  // row of the layer's pool; every lane's chunk of a row is the same one throughout
        const int c = lane & (p.chunks - 1);
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int e = e0 + u * 32 + lane;
            to[u] = -1;
            if (e < total) {
                const int hr = e >> shift, i = hr / nh, h = h0 + hr - i * nh;
                const int2 m = s_move[warp][i];
                const int from = ((m.x / kBlockSize) * p.Hkv + h) * kBlockSize + m.x % kBlockSize;
                to[u] = ((m.y / kBlockSize) * p.Hkv + h) * kBlockSize + m.y % kBlockSize;
                x[u] = pool[(static_cast<int64_t>(from) << shift) + c];
            }
        }
        __syncwarp();
#pragma unroll
        for (int u = 0; u < U; ++u)
            if (to[u] >= 0) pool[(static_cast<int64_t>(to[u]) << shift) + c] = x[u];
        __syncwarp();
    }
}

}  // namespace commit

cudaError_t launch_tree_commit(const CommitArgs& a, cudaStream_t stream) {
    if (a.B <= 0) return cudaSuccess;
    const int sms = sm_count();
    if (sms <= 0) return cudaErrorNoDevice;
    commit::Params p;
    p.k_pool = reinterpret_cast<uint4*>(a.k_pool);
    p.v_pool = reinterpret_cast<uint4*>(a.v_pool);
    p.chunks = a.D / 8;
    p.layer_u4 = static_cast<int64_t>(a.num_blocks) * a.Hkv * kBlockSize * p.chunks;
    p.block_table = a.block_table;
    p.context_lens = a.context_lens;
    p.tree_lens = a.tree_lens;
    p.path = a.path;
    p.path_len = a.path_len;
    p.new_context_lens = a.new_context_lens;
    p.err = a.err;
    p.num_blocks = a.num_blocks;
    p.max_blocks = a.max_blocks;
    p.P = a.P;
    p.L = a.L;
    p.Hkv = a.Hkv;
    // A warp per layer and pool, split over the KV heads up to 128 warps per SM (twice what it holds): 24 layers x 64
    // sequences x 8 heads, D = 128, up to 7 rows each: 13.8 us with 32 a SM, 12.0 with 64, 11.5 with 128, 13.6 with 256.
    const int64_t units = static_cast<int64_t>(a.L) * 2 * a.B, slots = static_cast<int64_t>(sms) * 128;
    const int parts = static_cast<int>(std::min<int64_t>(a.Hkv, std::max<int64_t>(1, slots / units)));
    p.heads_per_warp = (a.Hkv + parts - 1) / parts;
    p.head_parts = (a.Hkv + p.heads_per_warp - 1) / p.heads_per_warp;
    const int64_t warps = static_cast<int64_t>(a.L) * 2 * p.head_parts;
    const dim3 grid(static_cast<unsigned>((warps + commit::kWarps - 1) / commit::kWarps), a.B);
    return launch(commit::kv_tree_commit_kernel, grid, dim3(commit::kWarps * 32), 0, stream, true, 1u, p);
}

}  // namespace kvc
