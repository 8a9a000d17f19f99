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
// (kv_rope_turns).  The product with the position then wraps modulo one turn by itself, exactly; its top 32 bits are
// the angle in units of 2^-32 turns, and sincospif takes them as a multiple of pi (error 2^-24 turns / 2).
//
// Layout.  A row is D / 16 lanes of two 16-byte chunks each, chosen so that both values of every pair sit in one
// lane (chunks l and l + rot_dim / 16, or 2 l and 2 l + 1): no exchange between lanes but the sum of squares.  A warp
// takes kRows = 512 / D rows at a time and keeps one token's cosines and sines in registers for all its heads; they
// are computed once per warp (rot_dim / 2 angles over 32 lanes) and handed out through shared memory.
#include <atomic>

#include "../../include/kvc.h"
#include "decode_common.cuh"
#include "kvc_internal.h"
#include "ptx.cuh"

namespace kvc {
namespace rope {

#ifndef KVC_ROPE_U
#define KVC_ROPE_U 2
#endif
#ifndef KVC_ROPE_CTAS
#define KVC_ROPE_CTAS 2
#endif
constexpr int kWarps = 8;

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
    int Hq, Hkv, num_blocks, rot, interleaved, split, rows_per_warp;
    float eps;
};

__device__ __forceinline__ void unpack8(const uint4& u, float (&f)[8]) {
    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float2 t = unpack_half2(w[i]);
        f[2 * i] = t.x;
        f[2 * i + 1] = t.y;
    }
}
__device__ __forceinline__ uint4 pack8(const float (&f)[8]) {
    return make_uint4(pack_half2(f[0], f[1]), pack_half2(f[2], f[3]), pack_half2(f[4], f[5]), pack_half2(f[6], f[7]));
}

template <int D>
__global__ void __launch_bounds__(kWarps * 32, KVC_ROPE_CTAS) kv_append_rope_kernel(const Params p) {
    constexpr int kLanes = D / 16;        // lanes of a row
    constexpr int kRows = 32 / kLanes;    // rows a warp handles at a time
    __shared__ float2 s_cs[kWarps][D / 2];  // (cos, sin) of the warp's token
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int64_t w = static_cast<int64_t>(blockIdx.x) * kWarps + warp;
    const int64_t t = w / p.split;
    if (t >= p.n) return;  // whole warps
    const int l = lane % kLanes, rsub = lane / kLanes;

    const int64_t pos = p.rot > 0 ? p.positions[t] : 0;
    for (int i = lane; i < p.rot / 2; i += 32) {
        const int32_t a = static_cast<int32_t>((static_cast<uint64_t>(pos) * p.turns[i]) >> 32);
        float s, c;
        sincospif(static_cast<float>(a) * 0x1p-31f, &s, &c);
        s_cs[warp][i] = make_float2(c, s);
    }
    __syncwarp();

    // this lane's two chunks and, per chunk, whether it is rotated
    const int hc = p.rot / 16;  // chunks of the first half of the rotated dims
    int c0, c1;
    bool r0, r1;
    if (p.interleaved) {
        c0 = 2 * l;
        c1 = c0 + 1;
        r0 = c0 * 8 < p.rot;
        r1 = c1 * 8 < p.rot;
    } else {
        r0 = r1 = l < hc;
        c0 = r0 ? l : 2 * l;  // behind the pairs: 2 hc + 2 (l - hc)
        c1 = r0 ? l + hc : 2 * l + 1;
    }
    // cosines and sines of the lane's 8 pairs
    float cs[8], sn[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const int a = p.interleaved ? (i < 4 ? c0 * 4 + i : c1 * 4 + i - 4) : c0 * 8 + i;
        const bool on = p.interleaved ? (i < 4 ? r0 : r1) : r0;
        const float2 x = on ? s_cs[warp][a] : make_float2(1.f, 0.f);
        cs[i] = x.x;
        sn[i] = x.y;
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

    const int total = p.Hq + 2 * p.Hkv;
    const int row_end = min(total, (static_cast<int>(w % p.split) + 1) * p.rows_per_warp);
    constexpr int U = KVC_ROPE_U;  // iterations whose loads are in flight together
    for (int rb = static_cast<int>(w % p.split) * p.rows_per_warp; rb < row_end; rb += U * kRows) {
        uint4 raw[U][2];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int r = rb + u * kRows + rsub;
            raw[u][0] = raw[u][1] = make_uint4(0u, 0u, 0u, 0u);
            if (r < row_end) {
                const __half* src = r < p.Hq ? p.q + t * p.q_stride + r * D
                                    : r < p.Hq + p.Hkv ? p.k + t * p.k_stride + (r - p.Hq) * D
                                                       : p.v + t * p.v_stride + (r - p.Hq - p.Hkv) * D;
                raw[u][0] = *reinterpret_cast<const uint4*>(src + c0 * 8);
                raw[u][1] = *reinterpret_cast<const uint4*>(src + c1 * 8);
            }
        }
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int r = rb + u * kRows + rsub;
            const bool is_v = r >= p.Hq + p.Hkv, is_q = r < p.Hq;
            uint4 o0 = raw[u][0], o1 = raw[u][1];
            float x[8], y[8];
            unpack8(o0, x);
            unpack8(o1, y);
            const __half* wt = is_q ? p.qw : p.kw;
            float ss = 0.f;
#pragma unroll
            for (int i = 0; i < 8; ++i) ss = fmaf(x[i], x[i], fmaf(y[i], y[i], ss));
#pragma unroll
            for (int off = kLanes / 2; off > 0; off >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, off);
            if (!is_v) {
                if (wt != nullptr) {
                    const float inv = rsqrtf(ss * (1.f / D) + p.eps);
                    float wx[8], wy[8];
                    unpack8(__ldg(reinterpret_cast<const uint4*>(wt + c0 * 8)), wx);
                    unpack8(__ldg(reinterpret_cast<const uint4*>(wt + c1 * 8)), wy);
#pragma unroll
                    for (int i = 0; i < 8; ++i) {
                        x[i] *= inv * wx[i];
                        y[i] *= inv * wy[i];
                    }
                }
                if (p.interleaved) {
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const float a = x[2 * i], b = x[2 * i + 1], e = y[2 * i], f = y[2 * i + 1];
                        x[2 * i] = a * cs[i] - b * sn[i];
                        x[2 * i + 1] = b * cs[i] + a * sn[i];
                        y[2 * i] = e * cs[4 + i] - f * sn[4 + i];
                        y[2 * i + 1] = f * cs[4 + i] + e * sn[4 + i];
                    }
                } else {
#pragma unroll
                    for (int i = 0; i < 8; ++i) {
                        const float a = x[i], b = y[i];
                        x[i] = a * cs[i] - b * sn[i];
                        y[i] = b * cs[i] + a * sn[i];
                    }
                }
                // without a norm, dims that are not rotated keep their bits
                if (wt != nullptr || r0) o0 = pack8(x);
                if (wt != nullptr || r1) o1 = pack8(y);
            }
            if (r >= row_end) continue;
            auto put = [&](__half* row) {
                *reinterpret_cast<uint4*>(row + c0 * 8) = o0;
                *reinterpret_cast<uint4*>(row + c1 * 8) = o1;
            };
            if (is_q) {
                put(p.q_out + (t * p.Hq + r) * D);
            } else {
                const int h = is_v ? r - p.Hq - p.Hkv : r - p.Hq;
                __half* packed = is_v ? p.v_out : p.k_out;
                if (packed != nullptr) put(packed + (t * p.Hkv + h) * D);
                if (dst >= 0) put((is_v ? p.v_cache : p.k_cache) + dst + static_cast<int64_t>(h) * kBlockSize * D);
            }
        }
    }
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
    const int rows = a.Hq + 2 * a.Hkv, per_pass = 512 / a.D;
    // Warps per token: few tokens spread their heads over the GPU's SMs (one pass of rows per warp at least), many
    // keep a token in one warp, which computes its cosines and sines once.
    const int64_t want = static_cast<int64_t>(sms) * rope::kWarps;
    const int passes = (rows + per_pass - 1) / per_pass;
    int split = static_cast<int>(std::min<int64_t>(passes, std::max<int64_t>(1, want / a.n)));
    const int passes_each = (passes + split - 1) / split;
    split = (passes + passes_each - 1) / passes_each;
    p.split = split;
    p.rows_per_warp = passes_each * per_pass;
    const int64_t blocks = (a.n * split + rope::kWarps - 1) / rope::kWarps;
    if (blocks > 2147483647LL) return cudaErrorInvalidConfiguration;
    const dim3 grid(static_cast<unsigned>(blocks)), block(rope::kWarps * 32);
    if (a.D == 64)
        rope::kv_append_rope_kernel<64><<<grid, block, 0, stream>>>(p);
    else if (a.D == 128)
        rope::kv_append_rope_kernel<128><<<grid, block, 0, stream>>>(p);
    else
        return cudaErrorInvalidValue;
    return cudaGetLastError();
}

}  // namespace kvc
