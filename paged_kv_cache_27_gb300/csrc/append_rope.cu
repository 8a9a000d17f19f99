// Query / key norm, position rotation and append in one pass over a step's projected rows.
//
// For every token t and head row x of D values (query rows, and the key rows of the KV heads):
//   y_i = x_i * rsqrt(mean_i(x_i^2) + eps) * w_i            (left out without weights)
//   (y_a, y_b) <- (y_a cos g - y_b sin g, y_b cos g + y_a sin g)   for the rot_dim / 2 pairs (a, b) of the row,
//                 g = position[t] * frequency of the pair
// Pairs are (i, i + rot_dim / 2), or (2 i, 2 i + 1) when interleaved.  The query rows go to q_out, the key rows and
// the untouched value rows into their slot of the paged cache (and to k_out / v_out where a caller wants them packed,
// as the prefill does).  Arithmetic is fp32, each value is rounded to fp16 once, at its store.
//
// Angles.  fp32 has no room for position * frequency (a position of 100,000 leaves 2^-7 of a radian), so a frequency
// is held as the fraction of a full turn it advances per position, a 64-bit integer in units of 2^-64 turns
// (kv_rope_turns).  The product with the position then wraps modulo one turn by itself, exactly; it is rounded to 2^-32
// turn (off by 2^-33), and to fp32 as a multiple of pi for sincospif (by 2^-26 turn at most, half a step below half a
// turn).
//
// Layout.  A row is D / 16 lanes of two 16-byte chunks each, chosen so that both values of every pair sit in one
// lane (chunks l and l + rot_dim / 16, or 2 l and 2 l + 1): no exchange between lanes but the sum of squares.  A warp
// takes kRows = 512 / D rows at a time and keeps one token's cosines and sines in registers for all its heads; they
// are computed once per warp (rot_dim / 2 angles over 32 lanes) and handed out through shared memory.
//
// What bounds it.  Long prompts: memory, rows read and written once (16,384 tokens, 32 / 8 heads, D = 128: 66.2 us, 90
// % of a copy's rate).  Many tokens of few heads (60,000, 14 / 2, D = 64: 82 us, twice what its bytes take): each kind of
// rows is a loop of its own whose loads follow the last one's stores, and 18 rows fill 18 of a warp's 4 x 8 places.  Fewer
// rows: the launch, two dependent loads (position and slot, then rows), the angles and the store (512 tokens of the
// first 5.1 us, 1923 tokens, 14 / 2 heads, D = 64 4.1 us, one token 2.5 us).
#include <type_traits>

#include "../../include/kvc.h"
#include "decode_common.cuh"
#include "kvc_internal.h"
#include "f32x2.cuh"
#include "ptx.cuh"

namespace kvc {
namespace rope {

constexpr int kWarps = 8;
// Passes whose loads are in flight together, and CTAs per SM the registers are shared out for: 16,384 tokens, 32 / 8
// heads, D = 128: 2 / 3 71.9 us, 2 / 2 83.2, 4 / 2 77.1, 3 / 3 (spills) 71.4, 2 / 4 (spills) 82.2.
constexpr int U = 2;
constexpr int kCtasPerSm = 3;

struct Params {
    const __half* q;
    const __half* k;
    const __half* v;
    int64_t q_stride, k_stride, v_stride;  // elements between tokens
    const __half* qw;
    const __half* kw;
    const int32_t* positions;
    const uint64_t* turns;
    __half* q_out;
    __half* k_out;
    __half* v_out;
    __half* k_cache;
    __half* v_cache;
    const int64_t* slots;
    unsigned* err;
    int64_t n;
    int Hq, Hkv, num_blocks, rot, interleaved, split, passes_per_warp;
    float eps;
};

// eight fp16 values as four packed pairs of fp32, and back (one rounding each)
__device__ __forceinline__ void unpack8(const uint4& u, uint64_t (&f)[4]) {
    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float2 t = unpack_half2(w[i]);
        f[i] = pack_f32x2(t.x, t.y);
    }
}
__device__ __forceinline__ uint32_t pack2(uint64_t v) {
    float a, b;
    unpack_f32x2(v, a, b);
    return pack_half2(a, b);
}
__device__ __forceinline__ uint4 pack8(const uint64_t (&f)[4]) {
    return make_uint4(pack2(f[0]), pack2(f[1]), pack2(f[2]), pack2(f[3]));
}
__device__ __forceinline__ uint64_t neg_f32x2(uint64_t v) { return v ^ 0x8000000080000000ull; }
// (a, b) turned by the angle whose cosine and sine are half `hi` of c and s
__device__ __forceinline__ uint64_t rotate_pair(uint64_t v, uint64_t c, uint64_t s, int hi) {
    float a, b, c0, c1, s0, s1;
    unpack_f32x2(v, a, b);
    unpack_f32x2(c, c0, c1);
    unpack_f32x2(s, s0, s1);
    const float cc = hi ? c1 : c0, ss = hi ? s1 : s0;
    return pack_f32x2(fmaf(a, cc, -(b * ss)), fmaf(b, cc, a * ss));
}

template <bool kStream>
__device__ __forceinline__ uint4 load16(const __half* p) {
    return kStream ? __ldcs(reinterpret_cast<const uint4*>(p)) : *reinterpret_cast<const uint4*>(p);
}
template <bool kStream>
__device__ __forceinline__ void store16(__half* p, uint4 v) {
    if constexpr (kStream)
        __stcs(reinterpret_cast<uint4*>(p), v);
    else
        *reinterpret_cast<uint4*>(p) = v;
}

// kAll: the whole row is rotated.  Otherwise a lane behind rot_dim computes along and keeps its values by a select (a
// rotation by nothing would add 0 times the other value, NaN where that is not finite).  16,384 tokens, 32 / 8 heads,
// D = 128: 66.2 us with kAll, 67.4 without; a branch in place of the selects takes longer (1923 tokens, 14 / 2 heads,
// D = 64, half rotated: 4.3 us against 4.0).
template <int D, bool kStream, bool kAll>
__global__ void __launch_bounds__(kWarps * 32, kCtasPerSm) kv_append_rope_kernel(const Params p) {
    constexpr int kLanes = D / 16;        // lanes of a row
    constexpr int kRows = 32 / kLanes;    // rows a warp handles at a time
    __shared__ float2 s_cs[kWarps][D / 2];  // (cos, sin) of the warp's token
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int64_t w = static_cast<int64_t>(blockIdx.x) * kWarps + warp;
    // (a 64-bit division takes longer than a row; tokens are split only where they are few)
    const uint32_t part = p.split == 1 ? 0u : static_cast<uint32_t>(w) % static_cast<uint32_t>(p.split);
    const int64_t t = p.split == 1 ? w : static_cast<uint32_t>(w) / static_cast<uint32_t>(p.split);
    grid_dependency_wait();  // nothing is read or written before the kernel in front is done
    if (t >= p.n) return;  // whole warps
    const int l = lane % kLanes, rsub = lane / kLanes;

    const int64_t pos = p.rot > 0 ? p.positions[t] : 0;
    for (int i = lane; i < p.rot / 2; i += 32) {
        const int32_t a = static_cast<int32_t>((static_cast<uint64_t>(pos) * p.turns[i] + 0x80000000u) >> 32);
        float s, c;
        sincospif(static_cast<float>(a) * 0x1p-31f, &s, &c);
        s_cs[warp][i] = make_float2(c, s);
    }
    __syncwarp();

    // this lane's two chunks, and whether they are rotated (both or neither: rot_dim is a multiple of 16)
    const int hc = p.rot / 16;  // chunks of the first half of the rotated dims
    const bool on = kAll || l < hc;
    const bool apart = on && !p.interleaved;
    const int c0 = apart ? l : 2 * l, c1 = apart ? l + hc : 2 * l + 1;  // (behind the pairs: 2 hc + 2 (l - hc))
    // cosines and sines of the lane's 8 pairs
    uint64_t cs[4], sn[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int a = p.interleaved ? (i < 2 ? c0 * 4 + 2 * i : c1 * 4 + 2 * i - 4) : c0 * 8 + 2 * i;
        const float2 x = on ? s_cs[warp][a] : make_float2(1.f, 0.f), y = on ? s_cs[warp][a + 1] : make_float2(1.f, 0.f);
        cs[i] = pack_f32x2(x.x, y.x);
        sn[i] = pack_f32x2(x.y, y.y);
    }

    // the token's cache slot
    int64_t dst = -1;  // first element of (KV head 0, the token's offset) in its block
    if (p.slots != nullptr) {
        const int64_t slot = p.slots[t];
        if (slot >= static_cast<int64_t>(p.num_blocks) * kBlockSize) {
            if (lane == 0) atomicOr(p.err, KVC_DEVERR_SLOT);
        } else if (slot >= 0) {
            dst = ((slot / kBlockSize) * p.Hkv * kBlockSize + slot % kBlockSize) * D;
        }
    }

    // The warp's share of the passes: query rows, key rows, value rows, kRows heads at a time.
    const int pass0 = static_cast<int>(part) * p.passes_per_warp, pass1 = pass0 + p.passes_per_warp;
    const int pq = (p.Hq + kRows - 1) / kRows, pk = (p.Hkv + kRows - 1) / kRows;
    const auto rows = [&](auto kind, int first, int last) {  // passes [first, last) of one kind of rows
        constexpr int kKind = decltype(kind)::value;  // 0 query, 1 key, 2 value
        if (first >= last) return;
        const int H = kKind == 0 ? p.Hq : p.Hkv;
        const __half* src = (kKind == 0 ? p.q + t * p.q_stride : kKind == 1 ? p.k + t * p.k_stride : p.v + t * p.v_stride);
        __half* const packed = kKind == 0 ? p.q_out : kKind == 1 ? p.k_out : p.v_out;
        __half* const cache = kKind == 1 ? p.k_cache : p.v_cache;
        const __half* const wt = kKind == 0 ? p.qw : p.kw;
        uint4 w0 = make_uint4(0u, 0u, 0u, 0u), w1 = w0;
        if (kKind < 2 && wt != nullptr) {
            w0 = *reinterpret_cast<const uint4*>(wt + c0 * 8);
            w1 = *reinterpret_cast<const uint4*>(wt + c1 * 8);
        }
        for (int pass = first; pass < last; pass += U) {
            uint4 raw[U][2];
#pragma unroll
            for (int u = 0; u < U; ++u) {
                const int h = (pass + u) * kRows + rsub;
                raw[u][0] = raw[u][1] = make_uint4(0u, 0u, 0u, 0u);
                if (pass + u < last && h < H) {
                    raw[u][0] = load16<kStream>(src + h * D + c0 * 8);
                    raw[u][1] = load16<kStream>(src + h * D + c1 * 8);
                }
            }
#pragma unroll
            for (int u = 0; u < U; ++u) {
                if (pass + u >= last) break;
                const int h = (pass + u) * kRows + rsub;
                uint4 o0 = raw[u][0], o1 = raw[u][1];
                if constexpr (kKind < 2) {
                    uint64_t x[4], y[4];  // pairs of neighbouring values
                    unpack8(o0, x);
                    unpack8(o1, y);
                    if (wt != nullptr) {
                        uint64_t s2 = 0;
#pragma unroll
                        for (int i = 0; i < 4; ++i) s2 = fma_f32x2(x[i], x[i], fma_f32x2(y[i], y[i], s2));
                        float sa, sb;
                        unpack_f32x2(s2, sa, sb);
                        float ss = sa + sb;
#pragma unroll
                        for (int off = kLanes / 2; off > 0; off >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, off);
                        const float inv = rsqrtf(ss * (1.f / D) + p.eps);
                        const uint64_t inv2 = pack_f32x2(inv, inv);
                        uint64_t wx[4], wy[4];
                        unpack8(w0, wx);
                        unpack8(w1, wy);
#pragma unroll
                        for (int i = 0; i < 4; ++i) {
                            x[i] = mul_f32x2(mul_f32x2(x[i], inv2), wx[i]);
                            y[i] = mul_f32x2(mul_f32x2(y[i], inv2), wy[i]);
                        }
                    }
                    if (p.interleaved) {
#pragma unroll
                        for (int i = 0; i < 4; ++i) {
                            const uint64_t ra = rotate_pair(x[i], cs[i / 2], sn[i / 2], i & 1);
                            const uint64_t rb = rotate_pair(y[i], cs[2 + i / 2], sn[2 + i / 2], i & 1);
                            x[i] = on ? ra : x[i];
                            y[i] = on ? rb : y[i];
                        }
                    } else {
#pragma unroll
                        for (int i = 0; i < 4; ++i) {
                            const uint64_t a = x[i], b = y[i];
                            const uint64_t ra = fma_f32x2(a, cs[i], neg_f32x2(mul_f32x2(b, sn[i])));
                            const uint64_t rb = fma_f32x2(b, cs[i], mul_f32x2(a, sn[i]));
                            x[i] = on ? ra : a;
                            y[i] = on ? rb : b;
                        }
                    }
                    // without a norm, dims that are not rotated keep their bits
                    if (wt != nullptr || on) {
                        o0 = pack8(x);
                        o1 = pack8(y);
                    }
                }
                if (h >= H) continue;
                auto put = [&](__half* row) {
                    store16<kStream>(row + c0 * 8, o0);
                    store16<kStream>(row + c1 * 8, o1);
                };
                if (kKind == 0 || packed != nullptr) put(packed + (t * H + h) * D);
                if (kKind > 0 && dst >= 0) put(cache + dst + static_cast<int64_t>(h) * kBlockSize * D);
            }
        }
    };
    rows(std::integral_constant<int, 0>(), pass0, min(pass1, pq));
    rows(std::integral_constant<int, 1>(), max(pass0 - pq, 0), min(pass1 - pq, pk));
    rows(std::integral_constant<int, 2>(), max(pass0 - pq - pk, 0), min(pass1 - pq - pk, pk));
}

}  // namespace rope

cudaError_t launch_append_rope(const RopeArgs& a, cudaStream_t stream) {
    if (a.n <= 0) return cudaSuccess;
    const int sms = sm_count();
    if (sms <= 0) return cudaErrorNoDevice;
    rope::Params p;
    p.q = a.q;
    p.k = a.k;
    p.v = a.v;
    p.q_stride = a.q_stride;
    p.k_stride = a.k_stride;
    p.v_stride = a.v_stride;
    p.qw = a.q_weight;
    p.kw = a.k_weight;
    p.positions = a.positions;
    p.turns = a.turns;
    p.q_out = a.q_out;
    p.k_out = a.k_out;
    p.v_out = a.v_out;
    p.k_cache = a.k_cache;
    p.v_cache = a.v_cache;
    p.slots = a.slots;
    p.err = a.err;
    p.n = a.n;
    p.Hq = a.Hq;
    p.Hkv = a.Hkv;
    p.num_blocks = a.num_blocks;
    p.rot = a.rot_dim;
    p.interleaved = a.interleaved;
    p.eps = a.eps;
    // Warps per token: few tokens spread their heads over the GPU's SMs (one pass of rows per warp at least), many
    // keep a token in one warp, which computes its cosines and sines once.
    const int per_pass = 512 / a.D;
    const int passes = (a.Hq + per_pass - 1) / per_pass + 2 * ((a.Hkv + per_pass - 1) / per_pass);
    const int64_t want = static_cast<int64_t>(sms) * rope::kWarps;
    int split = static_cast<int>(std::min<int64_t>(passes, std::max<int64_t>(1, want / a.n)));
    p.passes_per_warp = (passes + split - 1) / split;
    split = (passes + p.passes_per_warp - 1) / p.passes_per_warp;
    p.split = split;
    const int64_t blocks = (a.n * split + rope::kWarps - 1) / rope::kWarps;
    if (blocks > 2147483647LL) return cudaErrorInvalidConfiguration;
    // Rows beyond what L2 holds (129 MB, read and written) stream past it: 16,384 tokens, 32 / 8 heads, D = 128: 72.0 ->
    // 67.9 us.  Smaller calls (512 tokens: 5.7 us either way) leave their rows there for the attention that follows.
    const bool stream_by = a.n * (a.Hq + 2 * a.Hkv) * a.D * 4 > (int64_t(128) << 20);
    const dim3 grid(static_cast<unsigned>(blocks)), block(rope::kWarps * 32);
    const auto go = [&](auto kernel) { return launch(kernel, grid, block, 0, stream, true, 1u, p); };
    switch (a.D + (stream_by ? 2 : 0) + (a.rot_dim == a.D ? 1 : 0)) {
        case 64: return go(rope::kv_append_rope_kernel<64, false, false>);
        case 65: return go(rope::kv_append_rope_kernel<64, false, true>);
        case 66: return go(rope::kv_append_rope_kernel<64, true, false>);
        case 67: return go(rope::kv_append_rope_kernel<64, true, true>);
        case 128: return go(rope::kv_append_rope_kernel<128, false, false>);
        case 129: return go(rope::kv_append_rope_kernel<128, false, true>);
        case 130: return go(rope::kv_append_rope_kernel<128, true, false>);
        case 131: return go(rope::kv_append_rope_kernel<128, true, true>);
        default: return cudaErrorInvalidValue;
    }
}

}  // namespace kvc
