// What a row sees through a sliding window and sinks, and rows computed again from that alone (prefill_window.cu).
#pragma once
#include <cuda_fp16.h>
#include <stdint.h>

#include "ptx.cuh"

namespace kvc {

// The n lowest of 32 bits.
__device__ __forceinline__ uint32_t low_bits(int n) { return n >= 32 ? ~0u : n <= 0 ? 0u : (1u << n) - 1u; }

// Bit i: key k0 + i is visible to row qi, whose keys end at `end` (behind its own, or at its segment's end).
__device__ __forceinline__ uint32_t window_bits(int qi, int k0, int end, int window, int sinks) {
    return (low_bits(end - k0) & ~low_bits(qi - window + 1 - k0)) | low_bits(min(sinks, end) - k0);
}

// Scores of keys that are not visible become `fill`, whose weight is 0 whatever the scale is (which is not 0, see
// kMinWindowScaleLog2): after that a tile needs no mask.  (Comparing positions key by key, in the maximum and again in
// the weights, a masked tile took three times the time of another one.)
template <int N>
__device__ __forceinline__ void mask_scores(float (&s)[N], const uint32_t* bits, float fill) {
#pragma unroll
    for (int c = 0; c < N; ++c) s[c] = (bits[c >> 5] >> (c & 31)) & 1u ? s[c] : fill;
}
// a scale of 0 is taken as this: scores of fp16 rows (below 2^41) still vanish next to 1, and a masked one stays infinite
constexpr float kMinWindowScaleLog2 = 0x1p-100f;

// 32 columns (lane: column col0 + lane) of row qi's output from its visible keys alone, two passes over them: for rows
// that came out infinite or NaN.  The products give 0 * inf = NaN where a key that the row does not see holds an
// infinity or NaN (its weight is 0); here such a key is not touched, so that only what the row sees can make it so.
// One warp per row, D / 32 dims of the score's product per lane.
template <int D>
__device__ __noinline__ float window_row_again(const __half* q_row, const __half* k, const __half* v, int64_t kv_stride,
                                               int qi, int window, int sinks, float scale_log2, int col0) {
    constexpr int E = D / 32;
    const int lane = threadIdx.x & 31;
    float qv[E];
#pragma unroll
    for (int i = 0; i < E; ++i) qv[i] = __half2float(q_row[lane * E + i]);
    const int start = max(0, qi - window + 1), first = min(sinks, start);
    auto score = [&](int kj) {
        float s = 0.f;
#pragma unroll
        for (int i = 0; i < E; ++i) s = fmaf(qv[i], __half2float(k[kj * kv_stride + lane * E + i]), s);
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
        return s * scale_log2;
    };
    const int from = first > 0 ? 0 : start;
    auto next = [&](int kj) { return kj + 1 == first ? start : kj + 1; };
    float m = -INFINITY;
    for (int kj = from; kj <= qi; kj = next(kj)) m = fmaxf(m, score(kj));
    float l = 0.f, acc = 0.f;
    bool nan = false;
    for (int kj = from; kj <= qi; kj = next(kj)) {
        const float x = score(kj);
        nan |= x != x;
        if (m == -INFINITY) continue;
        const float w = ex2(x - m);
        l += w;
        acc = fmaf(w, __half2float(v[kj * kv_stride + col0 + lane]), acc);
    }
    return nan ? __int_as_float(0x7fffffff) : l != 0.f ? acc / l : 0.f;
}

}  // namespace kvc
