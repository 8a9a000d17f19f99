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
// and a refused token stays at zero: it was refused where p_k(x) <= q_k(x), and a only grows.  (An a above 2^100 counts
// as 2^100: a q stays finite, and what it leaves of p is a difference only where q is below 2^-100.)
//
// Sums.  Which token a draw hits is a comparison of running sums, so they are kept in 64-bit integers, in units of
// 2^-45.  A weight p - a q is formed in fp32 with every rounding error carried along (a as the sum of two floats, the
// product's error by fma, the difference's by the two-term difference), and split exactly into a multiple of 2^-23 and
// a remainder that is rounded to 2^-45, both by adding a constant whose last bit has that value: the sums are integer
// additions of the results' bits.  (Conversions of floats to 64-bit integers run at the FP64 unit's rate: a pass over
// 64 x 128,257 entries took 30 us with them.)  Integer sums do not depend on their order, so results repeat bit for bit
// for every grid.  Weights that are not positive are multiplied away by 0 inside the sums' fma instructions: 20
// instructions for two entries of two rows, four of them the clamps to [0, 1].
//
// Layout.  One thread-block cluster per sequence; its CTAs share the vocabulary in slices (a warp a part of a slice),
// every warp sends its sum of a pass to all CTAs of the cluster, and all of them follow the same decisions on the same
// numbers (the tree's, gathered by rank 0 for all; the sums).
//
// What bounds it.  A sequence's passes follow one another: each needs the sum of the one before.  64 sequences of
// 128,257 fp32 entries (16 nodes, three distinct children a node): 2.1 passes on average, 6 at most.  The first passes
// read 66 MB from memory; of a pass of a cluster alone on its SMs (4.8 us), about 2.5 us are arithmetic and loads from
// L2, 1.0 the exchange of the sums (the barrier of a cluster takes 0.7), 0.65 the decision.  29 to 45 us by the walks
// that are drawn (16 draws, median 36.4; with fp16 rows 31 to 47, median 37.2: half the bytes, and conversions in
// front of the same arithmetic), where one reading of the two rows of every sequence takes 9.7; one sequence of 32,000
// entries (8 nodes, a chain) 6.6 us.
#include <algorithm>
#include <atomic>

#include "../../include/kvc.h"
#include "decode_common.cuh"
#include "f32x2.cuh"
#include "kvc_internal.h"
#include "ptx.cuh"

namespace kvc {
namespace verify {

constexpr int kMaxClusterV = 8;
constexpr int kUnitBits = 45;  // weights are counted in 2^-45; a row's sum has room up to 2^19

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

__device__ __forceinline__ void st_cluster_u64(uint32_t addr, uint64_t v) {
    asm volatile("st.shared::cluster.u64 [%0], %1;" ::"r"(addr), "l"(v) : "memory");
}

// a probability: NaN and negative values count as 0, values above 1 as 1
__device__ __forceinline__ float prob(float x) { return __saturatef(x); }
// (Ordinary loads: the rows may be written by the kernel in front, under whose end this one is launched, so they are not
// constant for its whole life, which loads through the read-only path ask for.)
__device__ __forceinline__ float load_prob(const float* row, int i) { return prob(row[i]); }
__device__ __forceinline__ float load_prob(const __half* row, int i) { return prob(__half2float(row[i])); }

// (p - a q)^+ <= 1, a = ah + al >= 0, as a multiple of 2^-23 (in the bits of the first, above those of 1) and a
// remainder, at most about 2^-24, in units of 2^-45 (in the bits of the second, above those of kFine)
constexpr float kCoarse = 1.f;            // one ulp is 2^-23 up to 2
constexpr float kFine = 1.5f * 0x1p-22f;  // one ulp is 2^-45 within 2^-23 on both sides
struct Split {
    float coarse, fine;
};
__device__ __forceinline__ Split split_weight(float p, float q, float ah, float al) {
    const float h = __fmul_rn(ah, q);
    const float e = __fmaf_rn(al, q, __fmaf_rn(ah, q, -h));  // a q = h + e
    // p - h = r + d exactly where r > e: there p >= h, or r itself is exact
    const float r = __fsub_rn(p, h), d = __fsub_rn(__fsub_rn(p, r), h);
    const float m = r > e ? 1.f : 0.f;
    Split s;
    s.coarse = __fmaf_rn(r, m, kCoarse);
    s.fine = __fadd_rn(__fmaf_rn(__fsub_rn(d, e), m, __fmaf_rn(r, m, __fsub_rn(kCoarse, s.coarse))), kFine);
    return s;
}
__device__ __forceinline__ int coarse_units(const Split& s) {
    return __float_as_int(s.coarse) - __float_as_int(kCoarse);
}
__device__ __forceinline__ int fine_units(const Split& s) { return __float_as_int(s.fine) - __float_as_int(kFine); }
__device__ __forceinline__ uint64_t units(int64_t coarse, int64_t fine) {
    return static_cast<uint64_t>(coarse * (int64_t(1) << (kUnitBits - 23)) + fine);
}

__device__ __forceinline__ uint64_t warp_sum(uint64_t v) {
    const uint32_t m = (1u << 24) - 1;  // 24 bits at a time: their sum over a warp fits 32
    const uint64_t a = __reduce_add_sync(0xffffffffu, static_cast<uint32_t>(v) & m);
    const uint64_t b = __reduce_add_sync(0xffffffffu, static_cast<uint32_t>(v >> 24) & m);
    const uint64_t c = __reduce_add_sync(0xffffffffu, static_cast<uint32_t>(v >> 48));
    return a + (b << 24) + (c << 48);
}

__device__ __forceinline__ uint64_t sub_f32x2(uint64_t a, uint64_t b) {
    return fma_f32x2(b, pack_f32x2(-1.f, -1.f), a);  // one rounding of a - b
}
// What the entries of a pass are weighed with: nothing (a = 0, the target's row itself), a = 1 (after a node's first
// refusal, always), any a.  The same numbers come out of each, for less work: of a pair 8, 16 and 20 instructions.
enum { kPlain = 0, kOne = 1, kAny = 2 };
struct Factor {
    uint64_t ah, al, neg_ah;  // a = ah + al, twice each
    float h, l;
    int mode;
};
// sums of weights in the two parts' units, brought together every few weights
template <int kMode>
struct LaneSum {
    uint64_t sum = 0;
    uint32_t coarse = 0, fine = 0;  // bits, modulo 2^32, of at most 32 weights (whose parts' sums stay below 2^29)
    uint32_t pairs = 0;
    // the weights of two entries, as split_weight gives them one by one
    __device__ __forceinline__ void add(uint64_t p, uint64_t q, const Factor& f) {
        const uint64_t one = pack_f32x2(kCoarse, kCoarse);
        uint64_t co, rest;
        if constexpr (kMode == kPlain) {
            co = add_f32x2(p, one);
            rest = add_f32x2(p, sub_f32x2(one, co));
        } else {
            uint64_t r, c;
            float e0 = 0.f, e1 = 0.f, r0, r1;
            if constexpr (kMode == kOne) {
                r = sub_f32x2(p, q);
                c = sub_f32x2(sub_f32x2(p, r), q);
            } else {
                const uint64_t nh = mul_f32x2(f.neg_ah, q);
                const uint64_t e = fma_f32x2(f.al, q, fma_f32x2(f.ah, q, nh));
                r = add_f32x2(p, nh);
                c = sub_f32x2(add_f32x2(sub_f32x2(p, r), nh), e);
                unpack_f32x2(e, e0, e1);
            }
            unpack_f32x2(r, r0, r1);
            const uint64_t m = pack_f32x2(r0 > e0 ? 1.f : 0.f, r1 > e1 ? 1.f : 0.f);
            co = fma_f32x2(r, m, one);
            rest = fma_f32x2(c, m, fma_f32x2(r, m, sub_f32x2(one, co)));
        }
        const uint64_t fi = add_f32x2(rest, pack_f32x2(kFine, kFine));
        coarse += static_cast<uint32_t>(co) + static_cast<uint32_t>(co >> 32);
        fine += static_cast<uint32_t>(fi) + static_cast<uint32_t>(fi >> 32);
        ++pairs;
    }
    __device__ __forceinline__ void flush() {
        sum += units(static_cast<int>(coarse - 2 * pairs * __float_as_uint(kCoarse)),
                     static_cast<int>(fine - 2 * pairs * __float_as_uint(kFine)));
        coarse = fine = pairs = 0;
    }
};
// this lane's share of the weights of entries [b, e), one at a time: entries b + lane, b + lane + 32, ...
template <int kMode, typename T>
__device__ __forceinline__ void add_entries(LaneSum<kMode>& acc, const T* p, const T* q, int b, int e,
                                            const Factor& f) {
    constexpr int U = 8;
    for (int i0 = b + (threadIdx.x & 31); i0 < e; i0 += 32 * U) {
        float pv[U], qv[U];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int i = i0 + u * 32;
            pv[u] = i < e ? load_prob(p, i) : 0.f;
            qv[u] = kMode != kPlain && i < e ? load_prob(q, i) : 0.f;
        }
#pragma unroll
        for (int u = 0; u < U; u += 2) acc.add(pack_f32x2(pv[u], pv[u + 1]), pack_f32x2(qv[u], qv[u + 1]), f);
        acc.flush();
    }
}
template <typename T>
__device__ __forceinline__ void unpack16(const uint4& v, uint64_t (&x)[8 / sizeof(T)]) {
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
    if constexpr (sizeof(T) == 4) {
        x[0] = pack_f32x2(prob(__uint_as_float(w[0])), prob(__uint_as_float(w[1])));
        x[1] = pack_f32x2(prob(__uint_as_float(w[2])), prob(__uint_as_float(w[3])));
    } else {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const float2 f = unpack_half2(w[i]);
            x[i] = pack_f32x2(prob(f.x), prob(f.y));
        }
    }
}
// this lane's share of the weights of entries [b, e).  Rows of one alignment (a vocabulary of any size, but one stride
// and 16-byte aligned tensors) are read 16 bytes at a time between their first and last few entries (64 sequences x
// 128,257 entries: 78 -> 59 us), the next vectors ahead of the current ones' arithmetic (50 -> 48 us), the few entries
// asked for before them (48 -> 47 us).  A ring of asynchronous copies to shared memory in place of the registers is
// slower, alone on an SM (3.5 -> 4.0 us a pass) and not (43 -> 45 us).
template <int kMode, typename T>
__device__ __forceinline__ uint64_t lane_weights(const T* p, const T* q, int b, int e, const Factor& f) {
    LaneSum<kMode> acc;
    if (kMode != kPlain && (reinterpret_cast<uintptr_t>(p) ^ reinterpret_cast<uintptr_t>(q)) & 15u) {
        add_entries(acc, p, q, b, e, f);
        return acc.sum;
    }
    constexpr int V = 16 / sizeof(T), U = 2;
    const int skip = static_cast<int>((0 - reinterpret_cast<uintptr_t>(p + b)) & 15u) / static_cast<int>(sizeof(T));
    const int a = min(e, b + skip);
    const int nv = (e - a) / V, lane = threadIdx.x & 31;
    const uint4* pv = reinterpret_cast<const uint4*>(p + a);
    const uint4* qv = reinterpret_cast<const uint4*>(q + a);
    // the entries in front of the first vector and behind the last, fewer than V each: one per lane, asked for first
    const int at = lane < V ? b + lane : a + nv * V + lane - V;
    const int edge = (lane < V ? at < a : lane < 2 * V && at < e) ? at : -1;
    const float pe = edge >= 0 ? load_prob(p, edge) : 0.f;
    const float qe = kMode != kPlain && edge >= 0 ? load_prob(q, edge) : 0.f;
    uint4 x[U], y[U], nx[U], ny[U];  // the vectors at work, and the next ones on their way
    auto fetch = [&](int i0) {
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int i = i0 + u * 32;
            nx[u] = ny[u] = make_uint4(0u, 0u, 0u, 0u);
            if (i < nv) {
                nx[u] = pv[i];
                if constexpr (kMode != kPlain) ny[u] = qv[i];
            }
        }
    };
    fetch(lane);
    for (int i0 = lane; i0 < nv; i0 += 32 * U) {
#pragma unroll
        for (int u = 0; u < U; ++u) {
            x[u] = nx[u];
            y[u] = ny[u];
        }
        fetch(i0 + 32 * U);
#pragma unroll
        for (int u = 0; u < U; ++u) {
            uint64_t fx[V / 2], fy[V / 2];
            unpack16<T>(x[u], fx);
            unpack16<T>(y[u], fy);
#pragma unroll
            for (int k = 0; k < V / 2; ++k) acc.add(fx[k], fy[k], f);
        }
        acc.flush();
    }
    acc.add(pack_f32x2(pe, 0.f), pack_f32x2(qe, 0.f), f);
    acc.flush();
    return acc.sum;
}
template <typename T>
__device__ __forceinline__ uint64_t lane_weights(const T* p, const T* q, int b, int e, const Factor& f) {
    return f.mode == kPlain ? lane_weights<kPlain, T>(p, q, b, e, f)
           : f.mode == kOne ? lane_weights<kOne, T>(p, q, b, e, f)
                            : lane_weights<kAny, T>(p, q, b, e, f);
}

// Sums of two floats, ~48 bits: the walk's scalars (the FP64 unit is slow: a trial took 0.6 us on it).  The error-free
// sum is Knuth's, the error-free product one rounded product and its error by fma.
struct Two {
    float h, l;
};
__device__ __forceinline__ Two two_sum(float a, float b) {
    const float s = __fadd_rn(a, b), t = __fsub_rn(s, a);
    return {s, __fadd_rn(__fsub_rn(a, __fsub_rn(s, t)), __fsub_rn(b, t))};
}
__device__ __forceinline__ Two two_prod(float a, float b) {
    const float s = __fmul_rn(a, b);
    return {s, __fmaf_rn(a, b, -s)};
}
__device__ __forceinline__ Two operator+(Two a, Two b) {
    Two s = two_sum(a.h, b.h);
    const Two t = two_sum(a.l, b.l);
    s = two_sum(s.h, __fadd_rn(s.l, t.h));
    return two_sum(s.h, __fadd_rn(s.l, t.l));
}
__device__ __forceinline__ Two operator-(Two a) { return {-a.h, -a.l}; }
__device__ __forceinline__ Two operator*(Two a, Two b) {
    const Two p = two_prod(a.h, b.h);
    return two_sum(p.h, __fadd_rn(p.l, __fmaf_rn(a.h, b.l, __fmul_rn(a.l, b.h))));
}
__device__ __forceinline__ Two operator/(Two a, Two b) {
    const float q0 = __fdiv_rn(a.h, b.h);
    const Two r = a + -(b * Two{q0, 0.f});
    return two_sum(q0, __fdiv_rn(__fadd_rn(r.h, r.l), b.h));
}
__device__ __forceinline__ bool positive(Two a) { return a.h > 0.f || (a.h == 0.f && a.l > 0.f); }
// a sum of weights as a number (exact below 2^48 units)
__device__ __forceinline__ Two from_units(uint64_t n) {
    return two_sum(__fmul_rn(static_cast<float>(static_cast<uint32_t>(min(n >> 24, uint64_t(0xFFFFFFFFu)))), 0x1p-21f),
                   __fmul_rn(static_cast<float>(static_cast<uint32_t>(n) & 0xFFFFFFu), 0x1p-45f));
}
// floor(u n) for 0 <= u <= 1
__device__ __forceinline__ uint64_t scaled(float u, uint64_t n) {
    u = __saturatef(u);
    if (u >= 1.f) return n;
    const uint32_t bits = __float_as_uint(u);
    const uint64_t m = bits & 0x7FFFFFu;
    const int e = static_cast<int>(bits >> 23) - 86;  // u = (2^23 + m) 2^(e - 64)
    if (e + 86 == 0) return 0;                        // below 2^-126
    const uint64_t frac = e >= 0 ? (m | 0x800000u) << e : e > -24 ? (m | 0x800000u) >> -e : 0;
    return __umul64hi(frac, n);
}

template <typename T, int kThreads>
__global__ void __launch_bounds__(kThreads, 768 / kThreads) draft_tree_verify_kernel(const Params p) {
    constexpr int kWarps = kThreads / 32;
    __shared__ float4 s_tree[kMaxTreeNodes];        // a node's (key, u, p, q): p and q of its token at its parent
    __shared__ uint64_t s_tot[2][kMaxClusterV * kWarps];  // the warps' sums of a pass, by pass parity
    __shared__ uint64_t s_part[kWarps];
    __shared__ float s_a[2];
    __shared__ int s_pass, s_node;  // warp 0's decision: a pass over node s_node's rows with a, or the draw
    __shared__ int s_path[kMaxTreeNodes];
    const int b = blockIdx.y, tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int rank = static_cast<int>(blockIdx.x), cs = static_cast<int>(gridDim.x);  // one cluster spans x
    asm volatile("barrier.cluster.arrive.relaxed.aligned;" ::: "memory");  // this CTA runs
    grid_dependency_wait();  // nothing is read or written before the kernel in front is done
    int n_nodes = p.tree_lens != nullptr ? p.tree_lens[b] : p.T;
    const T* const prow = static_cast<const T*>(p.p) + static_cast<int64_t>(b) * p.T * p.p_stride;
    const T* const qrow = static_cast<const T*>(p.q) + static_cast<int64_t>(b) * p.T * p.q_stride;
    // rank 0 gathers the tree for the whole cluster (decisions must not differ between its CTAs), a thread a node and
    // one or more CTAs to tell
    // key: parent << 24 | token, which is below 2^24; negative: a node that no walk reaches
    float4 mine = make_float4(__int_as_float(-1), 0.f, 0.f, 0.f);
    if (rank == 0) {
        const int t = tid & (kMaxTreeNodes - 1);
        const bool in = t < p.T;
        const int64_t at = static_cast<int64_t>(b) * p.T + t;
        const int par = in && t > 0 ? p.parents[at] : -1, tok = in && t > 0 ? p.tokens[at] : 0;
        const float u = in ? p.uniforms[at] : 0.f;
        if (t < n_nodes) {
            mine.y = u;
            if (t > 0) {
                if (par < 0 || par >= t || tok < 0 || tok >= p.V) {
                    if (tid == t) atomicOr(p.err, KVC_DEVERR_TREE);
                } else {
                    mine.x = __int_as_float(par << 24 | tok);
                    mine.z = load_prob(prow + par * p.p_stride, tok);
                    mine.w = load_prob(qrow + par * p.q_stride, tok);
                }
            }
        }
    }
    if (n_nodes < 0 || n_nodes > p.T) {
        if (rank == 0 && tid == 0) atomicOr(p.err, KVC_DEVERR_TREE);
        n_nodes = 0;
    }
    asm volatile("barrier.cluster.wait.aligned;" ::: "memory");  // every CTA of the cluster runs
    if (rank == 0) {
        const uint32_t dst = smem_u32(&s_tree[tid & (kMaxTreeNodes - 1)]);
        for (int r = tid / kMaxTreeNodes; r < cs; r += kThreads / kMaxTreeNodes) {
            uint32_t remote;
            asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(remote) : "r"(dst), "r"(r));
            st_cluster_f32x4(remote, mine);
        }
    }
    cluster_sync_all();
    const auto key_of = [&](int t) { return __float_as_int(s_tree[t].x); };

    const int v0 = min(rank * p.slice, p.V), v1 = min(v0 + p.slice, p.V);
    const int wsz = ((v1 - v0 + kWarps - 1) / kWarps + 31) / 32 * 32;  // entries per warp
    const int w0 = min(v0 + warp * wsz, v1), w1 = min(w0 + wsz, v1);

    // the walk: warp 0 of each CTA takes it, the others have its word
    int cur = 0, len = n_nodes > 0 ? 1 : 0, last = 0;
    const Two zero{0.f, 0.f}, one{1.f, 0.f};
    Two a = zero, S = one, R = one;
    bool summed = false;  // s_tot and total hold the sums of (cur, a)
    int parity = 0;
    uint64_t total = 0;
    const bool empty = n_nodes == 0;
    while (!empty) {
        if (warp == 0) {
            bool pass;
            for (;;) {
                // the next child of cur behind `last`
                const int key0 = key_of(lane), key1 = key_of(lane + 32);
                const unsigned lo = __ballot_sync(0xffffffffu, lane > last && key0 >> 24 == cur);
                const unsigned hi = __ballot_sync(0xffffffffu, lane + 32 > last && key1 >> 24 == cur);
                if ((lo | hi) == 0) {
                    pass = !summed;  // draw, from the sums there are or after a pass
                    break;
                }
                const int c = lo ? __ffs(lo) - 1 : 31 + __ffs(hi);
                last = c;
                const float4 child = s_tree[c];
                const Two uq = two_prod(child.y, child.w);
                // u q S < (p - a q)^+ R; at a node's first child u q < p; where the residual's sum is 0, nothing of it is
                // left, whatever a single difference's sign (its rounding's, mostly) may be
                const Two left = Two{child.z, 0.f} + -(a * Two{child.w, 0.f});
                if (positive(R) && positive(S) && positive(left) && positive(left * R + -(uq * S))) {
                    if (lane == 0) s_path[len] = c;
                    ++len;
                    cur = c;
                    a = zero;
                    S = R = one;
                    summed = false;
                    continue;
                }
                const Two mass = R;
                if (p.distinct) {
                    // its mass leaves the draft's row, unless an earlier child had its token
                    const int key = __float_as_int(child.x);
                    if (!__any_sync(0xffffffffu, (lane < c && key0 == key) || (lane + 32 < c && key1 == key)))
                        R = R + Two{-child.w, 0.f};
                }
                if (positive(mass)) {
                    Two next = a + (p.distinct ? S / mass : S);
                    if (!(next.h < 0x1p100f)) next = Two{0x1p100f, 0.f};  // keeps every product finite
                    if (next.h != a.h || next.l != a.l) {
                        a = next;
                        pass = true;
                        break;
                    }
                }
            }
            if (lane == 0) {
                s_pass = pass;
                s_node = cur;
                s_a[0] = a.h;
                s_a[1] = a.l;
            }
        }
        __syncthreads();
        const bool pass = s_pass;
        const int node = s_node;
        Factor f;
        f.h = s_a[0];
        f.l = s_a[1];
        f.ah = pack_f32x2(f.h, f.h);
        f.al = pack_f32x2(f.l, f.l);
        f.neg_ah = pack_f32x2(-f.h, -f.h);
        f.mode = f.h == 0.f ? kPlain : f.h == 1.f && f.l == 0.f ? kOne : kAny;
        const T* const pr = prow + node * p.p_stride;
        const T* const qr = qrow + node * p.q_stride;
        if (pass) {
            const uint64_t ws = warp_sum(lane_weights(pr, qr, w0, w1, f));
            if (lane < cs) st_cluster_u64(map_to_rank(&s_tot[parity][rank * kWarps + warp], lane), ws);
            cluster_sync_all();
            uint64_t part = 0;
#pragma unroll
            for (int i = lane; i < kMaxClusterV * kWarps; i += 32)
                if (i < cs * kWarps) part += s_tot[parity][i];
            total = warp_sum(part);
            S = from_units(total);
            summed = true;
            parity ^= 1;
            continue;
        }
        // draw: the first entry whose running weight exceeds u * total
        if (total == 0) {
            if (f.mode != kPlain) {  // nothing of the residual is left: the target's own row
                a = zero;
                S = one;
                summed = false;
                last = kMaxTreeNodes;  // no further child is tried
                __syncthreads();       // every warp has read the word that is now replaced
                continue;
            }
            if (rank == 0 && tid == 0) {
                atomicOr(p.err, KVC_DEVERR_TREE);
                p.next_token[b] = -1;
            }
            break;
        }
        uint64_t th = scaled(s_tree[0].y, total);
        if (th >= total) th = total - 1;
        const uint64_t* const sums = s_tot[parity ^ 1];
        uint64_t tot = 0;  // of the CTA of this lane's number
        if (lane < cs) {
#pragma unroll
            for (int w = 0; w < kWarps; ++w) tot += sums[lane * kWarps + (w + lane) % kWarps];
        }
        uint64_t incl = tot;
#pragma unroll
        for (int o = 1; o < kMaxClusterV; o <<= 1) {
            const uint64_t below = __shfl_up_sync(0xffffffffu, incl, o);
            if (lane >= o) incl += below;
        }
        const int owner = __ffs(__ballot_sync(0xffffffffu, incl > th)) - 1;
        if (owner != rank) break;
        th -= __shfl_sync(0xffffffffu, incl - tot, owner);
        // the CTA's warp whose part holds it, then that part again in kWarps pieces
        const uint64_t* const warps = sums + rank * kWarps;
        int sw = 0;
        while (sw < kWarps - 1 && th >= warps[sw]) th -= warps[sw++];
        const int sb = min(v0 + sw * wsz, v1), se = min(sb + wsz, v1);
        const int psz = ((se - sb + kWarps - 1) / kWarps + 31) / 32 * 32;
        const int pb = min(sb + warp * psz, se), pe = min(pb + psz, se);
        const uint64_t ps = warp_sum(lane_weights(pr, qr, pb, pe, f));
        if (lane == 0) s_part[warp] = ps;
        __syncthreads();
        int pw = 0;
        while (pw < kWarps - 1 && th >= s_part[pw]) th -= s_part[pw++];
        if (warp != pw) break;
        constexpr int kRun = 8;  // up to 8 consecutive entries per lane: one prefix sum over the lanes for 256 entries
        const int run = min((pe - pb + 31) / 32, kRun);
        int found = -1;
        for (int i0 = pb; i0 < pe && found < 0; i0 += 32 * run) {
            const int i = i0 + lane * run;
            uint64_t w[kRun], sum = 0;
#pragma unroll
            for (int k = 0; k < kRun; ++k) {
                w[k] = 0;
                if (k < run && i + k < pe) {
                    const float q = f.mode != kPlain ? load_prob(qr, i + k) : 0.f;
                    const Split s = split_weight(load_prob(pr, i + k), q, f.h, f.l);
                    w[k] = units(coarse_units(s), fine_units(s));
                }
                sum += w[k];
            }
            uint64_t upto = sum;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const uint64_t below = __shfl_up_sync(0xffffffffu, upto, o);
                if (lane >= o) upto += below;
            }
            const unsigned hit = __ballot_sync(0xffffffffu, upto > th);
            if (hit != 0) {
                const int at = __ffs(hit) - 1;
                uint64_t left = th - (upto - sum);  // in lane `at`
                int k = 0;
#pragma unroll
                for (int j = 0; j < kRun - 1; ++j) {
                    if (k == j && j < run - 1 && left >= w[j]) {
                        left -= w[j];
                        ++k;
                    }
                }
                found = __shfl_sync(0xffffffffu, i + k, at);
            } else {
                th -= __shfl_sync(0xffffffffu, upto, 31);
            }
        }
        if (lane == 0) p.next_token[b] = found;
        break;
    }
    if (rank == 0 && warp == 0) {
        __syncwarp();
        for (int i = lane; i < p.T; i += 32)
            p.path[static_cast<int64_t>(b) * p.T + i] = i >= len ? -1 : i == 0 ? 0 : s_path[i];
        if (lane == 0) {
            p.path_len[b] = len;
            if (empty) p.next_token[b] = -1;
        }
    }
}

}  // namespace verify

template <typename T>
static cudaError_t launch_verify_t(const verify::Params& p, int B, int cs, bool wide, cudaStream_t stream) {
    const dim3 grid(cs, B);
    return wide ? launch(verify::draft_tree_verify_kernel<T, 512>, grid, dim3(512), 0, stream, true,
                         static_cast<unsigned>(cs), p)
                : launch(verify::draft_tree_verify_kernel<T, 256>, grid, dim3(256), 0, stream, true,
                         static_cast<unsigned>(cs), p);
}

// Clusters of cs CTAs that the device holds at a time (a GPC's SMs that no whole cluster fills stay idle).  Asked once
// per device, type and size.
static int resident_clusters(bool f32, bool wide, int cs, int sms) {
    const int per_sm = wide ? 1 : 768 / 256;
    if (cs == 1) return sms * per_sm;
    static std::atomic<int> cache[128][2][2][verify::kMaxClusterV + 1];
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 128) return std::max(1, sms * per_sm / cs);
    std::atomic<int>& slot = cache[dev][f32][wide][cs];
    int n = slot.load(std::memory_order_relaxed);
    if (n > 0) return n;
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute attr;
    attr.id = cudaLaunchAttributeClusterDimension;
    attr.val.clusterDim.x = cs;
    attr.val.clusterDim.y = attr.val.clusterDim.z = 1;
    cfg.gridDim = dim3(cs);
    cfg.blockDim = dim3(wide ? 512 : 256);
    cfg.attrs = &attr;
    cfg.numAttrs = 1;
    const auto ask = [&](auto kernel) { return cudaOccupancyMaxActiveClusters(&n, kernel, &cfg); };
    const cudaError_t e = f32 ? (wide ? ask(verify::draft_tree_verify_kernel<float, 512>)
                                      : ask(verify::draft_tree_verify_kernel<float, 256>))
                              : (wide ? ask(verify::draft_tree_verify_kernel<__half, 512>)
                                      : ask(verify::draft_tree_verify_kernel<__half, 256>));
    if (e != cudaSuccess || n < 1) {
        cudaGetLastError();
        n = std::max(1, sms * per_sm / cs);
    }
    slot.store(n, std::memory_order_relaxed);
    return n;
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
    // CTAs per sequence and threads per CTA: the choice with the shortest run of two passes, in us.  A pass takes an
    // exchange of the sums (1.1, in a cluster 1.55) and a CTA's arithmetic (87 ns per 1000 entries with 512 threads,
    // one CTA per SM; 197 with 256, three), or the memory's time for all rows that are read at once: the second pass
    // reads them from L2 where they fit.  A start takes 2; clusters that are not resident wait for others.  (Clusters
    // of eight for every larger V, 512 threads while every CTA had an SM: 512 sequences x 8000 entries 47.6 us, here
    // 11.3; 19 x 128,257 12.0, here 8.2; 64 x 128,257 with four refusals each 44.7, here 37.7.)
    const int sms = sm_count();
    if (sms <= 0) return cudaErrorNoDevice;
    constexpr double kMemory = 6.8e6, kL2 = 13.6e6, kL2Bytes = 100e6;  // bytes per us; bytes that stay
    double best = 1e300;
    int cs = 1;
    bool wide = false;
    for (int w = 1; w >= 0; --w) {
        for (const int c : {8, 6, 4, 3, 2, 1}) {
            const int resident = resident_clusters(a.probs_f32, w != 0, c, sms);
            const double work = static_cast<double>(a.V) / c * (w ? 87e-6 : 197e-6);
            const double bytes = static_cast<double>(std::min(a.B, resident)) * a.V * (a.probs_f32 ? 8 : 4);
            const double passes = 2 * (c > 1 ? 1.55 : 1.1) + 0.2 * work + std::max(work, bytes / kMemory) +
                                  std::max(work, bytes / (bytes <= kL2Bytes ? kL2 : kMemory));
            const double waves = a.B <= resident ? 1. : static_cast<double>(a.B) / resident + 0.2;
            if (waves * (2. + passes) < best) {
                best = waves * (2. + passes);
                cs = c;
                wide = w != 0;
            }
        }
    }
    p.slice = (a.V + cs - 1) / cs;
    return a.probs_f32 ? launch_verify_t<float>(p, a.B, cs, wide, stream)
                       : launch_verify_t<__half>(p, a.B, cs, wide, stream);
}

}  // namespace kvc
