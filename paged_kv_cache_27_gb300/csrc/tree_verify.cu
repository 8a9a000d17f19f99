// Verification of a tree of drafted tokens against the target's probabilities, and the step's next token.
//
// The rule (speculative decoding paragraph of "Tornar a inferência barata", neuralialabs.com: a drafted token x is
// kept with probability min(1, p(x) / q(x)), else the next token comes from the residual max(0, p - q), rescaled),
// for several drafted children per node.  At node c, with the target's row p and the draft's row q, the children
// x_1, x_2, ... are tried in order against p_0 = p, q_0 = q:
//   keep x_k if  u_k q_k(x_k) < p_k(x_k);   else  p_{k+1} = max(0, p_k - q_k) / its sum,
//   q_{k+1} = q_k, or, for children drawn without replacement, q_k without x_k, rescaled.
// The walk goes on from a kept child; where no child is kept the next token is drawn from the last p_k.
//
// What makes it one row pass per refused token: every p_k is max(0, p - a_k q) / S_k.  With q_k = q / R_k on the
// tokens not yet refused (R_k their mass; 1 with replacement), max(0, (p - a q)^+ / S - q / R) is
// (p - (a + S / R) q)^+ / S, so
//   a_{k+1} = a_k + S_k / R_k,   S_{k+1} = sum (p - a_{k+1} q)^+,   a_0 = 0, S_0 = R_0 = 1,
// and a refused token stays at zero: it was refused where p_k(x) <= q_k(x), and a only grows.
//
// Sums.  Which token a draw hits is a comparison of running sums, so they are kept in 64-bit integers, in units of
// 2^-52: p is read to 2^-53, a q is formed as a product of two floats' sum with q (48 bits of a) with its rounding
// error carried along.  Integer sums do not depend on their order, so results repeat bit for bit for every grid.
//
// Layout.  One thread-block cluster per sequence; its CTAs share the vocabulary in slices (a warp a part of a slice)
// and exchange their sums through distributed shared memory, and all of them follow the same decisions on the same
// numbers (the tree's, read by rank 0 once; the sums).  The kernel is bound by the two rows it reads per pass.
#include <atomic>

#include "../../include/kvc.h"
#include "decode_common.cuh"
#include "kvc_internal.h"
#include "ptx.cuh"

namespace kvc {
namespace verify {

constexpr int kThreads = 512;
constexpr int kWarps = kThreads / 32;
constexpr int kMaxClusterV = 8;
constexpr float kUnit = 0x1p52f;  // probabilities are counted in 2^-52; a row's sum has room up to 4096
constexpr double kUnitInv = 0x1p-52;

struct Params {
    const void* p;
    const void* q;
    int64_t p_stride, q_stride;  // elements between the rows of two nodes
    const int32_t* tokens;
    const int32_t* parents;
    const int32_t* tree_lens;
    const float* uniforms;
    int32_t* path;
    int32_t* path_len;
    int32_t* next_token;
    unsigned* err;
    int T, V, distinct, slice;  // slice: vocabulary entries per CTA
};

struct Tree {  // rank 0's copy is read by the other CTAs
    int32_t token[kMaxTreeNodes];
    int32_t parent[kMaxTreeNodes];
    float u[kMaxTreeNodes];
    float p[kMaxTreeNodes];  // target and draft probability of the node's token at its parent
    float q[kMaxTreeNodes];
};

__device__ __forceinline__ void st_cluster_u64(uint32_t addr, uint64_t v) {
    asm volatile("st.shared::cluster.u64 [%0], %1;" ::"r"(addr), "l"(v) : "memory");
}

// a probability: NaN and negative values count as 0, values above 1 as 1
__device__ __forceinline__ float prob(float x) { return __saturatef(x); }
__device__ __forceinline__ float load_prob(const float* row, int i) { return prob(__ldg(row + i)); }
__device__ __forceinline__ float load_prob(const __half* row, int i) { return prob(__half2float(__ldg(row + i))); }

// (p - a q)^+ in units of 2^-52, a = ah + al
__device__ __forceinline__ uint64_t weight(float p, float q, float ah, float al) {
    const float h = ah * q;
    if (!(h < 2.f)) return 0;  // p <= 1
    const float e = fmaf(al, q, fmaf(ah, q, -h));  // a q = h + e
    const int64_t w = __float2ll_rn(p * kUnit) - __float2ll_rn(h * kUnit) - __float2ll_rn(e * kUnit);
    return w > 0 ? static_cast<uint64_t>(w) : 0;
}

__device__ __forceinline__ uint64_t warp_sum(uint64_t v) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    return v;
}

// this lane's share of the weights of entries [b, e): entries b + lane, b + lane + 32, ...
template <typename T>
__device__ __forceinline__ uint64_t lane_weights(const T* __restrict__ p, const T* __restrict__ q, int b, int e, float ah,
                                                 float al) {
    constexpr int U = 8;
    const int lane = threadIdx.x & 31;
    uint64_t sum = 0;
    const bool use_q = ah != 0.f;
    for (int i0 = b; i0 < e; i0 += 32 * U) {
        float pv[U], qv[U];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int i = i0 + u * 32 + lane;
            pv[u] = i < e ? load_prob(p, i) : 0.f;
            qv[u] = i < e && use_q ? load_prob(q, i) : 0.f;
        }
#pragma unroll
        for (int u = 0; u < U; ++u) sum += weight(pv[u], qv[u], ah, al);
    }
    return sum;
}

template <typename T>
__global__ void __launch_bounds__(kThreads) draft_tree_verify_kernel(const Params p) {
    __shared__ Tree s_tree;
    __shared__ uint64_t s_tot[2][kMaxClusterV];  // the CTAs' sums of a pass, by pass parity
    __shared__ uint64_t s_warp[kWarps], s_part[kWarps];
    __shared__ float s_a[2];
    __shared__ int s_cmd, s_node;  // warp 0's decision: 1 = pass over node s_node's rows with a, 0 = draw
    __shared__ int s_path[kMaxTreeNodes];
    const int b = blockIdx.y, tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int rank = static_cast<int>(blockIdx.x), cs = static_cast<int>(gridDim.x);  // one cluster spans x
    int n_nodes = p.tree_lens != nullptr ? p.tree_lens[b] : p.T;
    if (n_nodes < 0 || n_nodes > p.T) {
        if (rank == 0 && tid == 0) atomicOr(p.err, KVC_DEVERR_TREE);
        n_nodes = 0;
    }
    const T* const prow = static_cast<const T*>(p.p) + static_cast<int64_t>(b) * p.T * p.p_stride;
    const T* const qrow = static_cast<const T*>(p.q) + static_cast<int64_t>(b) * p.T * p.q_stride;
    if (rank == 0 && tid < kMaxTreeNodes) {
        const int64_t at = static_cast<int64_t>(b) * p.T + tid;
        int par = -2, tok = 0;  // a node that no walk reaches
        float u = 0.f, pc = 0.f, qc = 0.f;
        if (tid < n_nodes) {
            u = p.uniforms[at];
            if (tid > 0) {
                par = p.parents[at];
                tok = p.tokens[at];
                if (par < 0 || par >= tid || tok < 0 || tok >= p.V) {
                    atomicOr(p.err, KVC_DEVERR_TREE);
                    par = -2;
                } else {
                    pc = load_prob(prow + par * p.p_stride, tok);
                    qc = load_prob(qrow + par * p.q_stride, tok);
                }
            }
        }
        s_tree.token[tid] = tok;
        s_tree.parent[tid] = par;
        s_tree.u[tid] = u;
        s_tree.p[tid] = pc;
        s_tree.q[tid] = qc;
    }
    cluster_sync_all();
    if (rank != 0 && n_nodes > 0) {  // (rank 0 stays until the first pass's barrier; without nodes it leaves at once)
        const uint32_t src = map_to_rank(&s_tree, 0);
        for (int i = tid; i < static_cast<int>(sizeof(Tree) / 4); i += kThreads)
            reinterpret_cast<uint32_t*>(&s_tree)[i] = ld_cluster_u32(src + 4 * i);
    }
    if (tid == 0) s_path[0] = 0;
    __syncthreads();

    const int v0 = min(rank * p.slice, p.V), v1 = min(v0 + p.slice, p.V);
    const int wsz = ((v1 - v0 + kWarps - 1) / kWarps + 31) / 32 * 32;  // entries per warp
    const int w0 = min(v0 + warp * wsz, v1), w1 = min(w0 + wsz, v1);

    // the walk's state, kept by warp 0
    int cur = 0, len = n_nodes > 0 ? 1 : 0, last = 0;
    double a = 0.0, S = 1.0, R = 1.0;
    bool summed = false;  // s_tot holds the sums of (cur, a)
    int parity = 0;
    uint64_t total = 0;
    const bool empty = n_nodes == 0;
    while (!empty) {
        if (warp == 0) {
            int cmd = -1;
            while (cmd < 0) {
                // the next child of cur behind `last`
                const unsigned lo = __ballot_sync(0xffffffffu, lane > last && s_tree.parent[lane] == cur);
                const unsigned hi = __ballot_sync(0xffffffffu, lane + 32 > last && s_tree.parent[lane + 32] == cur);
                if ((lo | hi) == 0) {
                    cmd = summed ? 0 : 1;  // draw, from the sums there are or after a pass
                    break;
                }
                const int c = lo ? __ffs(lo) - 1 : 31 + __ffs(hi);
                last = c;
                const double pc = s_tree.p[c], qc = s_tree.q[c];
                const double left = fmax(pc - a * qc, 0.0);
                if (R > 0.0 && static_cast<double>(s_tree.u[c]) * qc * S < left * R) {
                    if (lane == 0) s_path[len] = c;
                    ++len;
                    cur = c;
                    a = 0.0;
                    S = R = 1.0;
                    summed = false;
                } else {
                    if (R > 0.0) {
                        const double a_new = a + S / R;
                        if (a_new != a) {
                            a = a_new;
                            cmd = 1;
                        }
                    }
                    if (p.distinct) R -= qc;
                }
            }
            if (lane == 0) {
                s_cmd = cmd;
                s_node = cur;
                s_a[0] = static_cast<float>(a);
                s_a[1] = static_cast<float>(a - static_cast<double>(static_cast<float>(a)));
            }
        }
        __syncthreads();
        const int cmd = s_cmd, node = s_node;
        const float ah = s_a[0], al = s_a[1];
        const T* const pr = prow + node * p.p_stride;
        const T* const qr = qrow + node * p.q_stride;
        if (cmd == 1) {
            const uint64_t ws = warp_sum(lane_weights(pr, qr, w0, w1, ah, al));
            if (lane == 0) s_warp[warp] = ws;
            __syncthreads();
            if (warp == 0) {
                const uint64_t cta = warp_sum(lane < kWarps ? s_warp[lane] : 0);
                if (lane < cs) st_cluster_u64(map_to_rank(&s_tot[parity][rank], lane), cta);
            }
            cluster_sync_all();
            total = 0;
            for (int r = 0; r < cs; ++r) total += s_tot[parity][r];
            S = static_cast<double>(total) * kUnitInv;
            summed = true;
            parity ^= 1;
            continue;
        }
        // draw: the first entry whose running weight exceeds u * total
        const uint64_t* tot = s_tot[parity ^ 1];
        if (total == 0) {
            if (ah != 0.f) {  // nothing of the residual is left: the target's own row
                a = 0.0;
                S = 1.0;
                summed = false;
                last = kMaxTreeNodes;  // no further child is tried
                __syncthreads();
                continue;
            }
            if (rank == 0 && tid == 0) {
                atomicOr(p.err, KVC_DEVERR_TREE);
                p.next_token[b] = -1;
            }
            break;
        }
        const double x = fmin(fmax(static_cast<double>(s_tree.u[0]), 0.0), 1.0) * static_cast<double>(total);
        uint64_t th = static_cast<uint64_t>(x);
        if (th >= total) th = total - 1;
        int owner = 0;
        while (owner < cs - 1 && th >= tot[owner]) th -= tot[owner++];
        if (owner != rank) break;
        // the CTA's warp whose part holds it (s_warp: this pass's sums), then that part again in kWarps pieces
        int sw = 0;
        while (sw < kWarps - 1 && th >= s_warp[sw]) th -= s_warp[sw++];
        const int sb = min(v0 + sw * wsz, v1), se = min(sb + wsz, v1);
        const int psz = ((se - sb + kWarps - 1) / kWarps + 31) / 32 * 32;
        const int pb = min(sb + warp * psz, se), pe = min(pb + psz, se);
        const uint64_t ps = warp_sum(lane_weights(pr, qr, pb, pe, ah, al));
        if (lane == 0) s_part[warp] = ps;
        __syncthreads();
        int pw = 0;
        while (pw < kWarps - 1 && th >= s_part[pw]) th -= s_part[pw++];
        if (warp != pw) break;
        int found = -1;
        for (int i0 = pb; i0 < pe && found < 0; i0 += 32) {
            const int i = i0 + lane;
            uint64_t incl = i < pe ? weight(load_prob(pr, i), ah != 0.f ? load_prob(qr, i) : 0.f, ah, al) : 0;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const uint64_t below = __shfl_up_sync(0xffffffffu, incl, o);
                if (lane >= o) incl += below;
            }
            const unsigned hit = __ballot_sync(0xffffffffu, incl > th);
            if (hit != 0)
                found = i0 + __ffs(hit) - 1;
            else
                th -= __shfl_sync(0xffffffffu, incl, 31);
        }
        if (lane == 0) p.next_token[b] = found;
        break;
    }
    if (rank == 0 && warp == 0) {
        __syncwarp();
        for (int i = lane; i < p.T; i += 32) p.path[static_cast<int64_t>(b) * p.T + i] = i < len ? s_path[i] : -1;
        if (lane == 0) {
            p.path_len[b] = len;
            if (empty) p.next_token[b] = -1;
        }
    }
}

}  // namespace verify

template <typename T>
static cudaError_t launch_verify_t(const verify::Params& p, int B, int cs, cudaStream_t stream) {
    return launch(verify::draft_tree_verify_kernel<T>, dim3(cs, B), dim3(verify::kThreads), 0, stream, false,
                  static_cast<unsigned>(cs), p);
}

cudaError_t launch_tree_verify(const VerifyArgs& a, cudaStream_t stream) {
    if (a.B <= 0) return cudaSuccess;
    verify::Params p;
    p.p = a.p;
    p.q = a.q;
    p.p_stride = a.p_stride;
    p.q_stride = a.q_stride;
    p.tokens = a.tokens;
    p.parents = a.parents;
    p.tree_lens = a.tree_lens;
    p.uniforms = a.uniforms;
    p.path = a.path;
    p.path_len = a.path_len;
    p.next_token = a.next_token;
    p.err = a.err;
    p.T = a.T;
    p.V = a.V;
    p.distinct = a.distinct;
    // CTAs per sequence: a warp should have a few loads in flight per lane before it is worth another CTA's share
    int cs = 1;
    while (cs < verify::kMaxClusterV && a.V > cs * verify::kThreads * 2) cs *= 2;
    p.slice = (a.V + cs - 1) / cs;
    return a.probs_f32 ? launch_verify_t<float>(p, a.B, cs, stream) : launch_verify_t<__half>(p, a.B, cs, stream);
}

}  // namespace kvc
