// Append to a cache of e4m3 codes with one power-of-two scale for each (block, KV head) of K and of V.
//
//   scale = 2^e, e the least exponent for which no value of the block's rows exceeds 448 * 2^e (-32 for zeros);
//   code = e4m3(x * 2^-e), rounded to nearest even.
// A power of two costs a floating-point code no precision, and makes both the product and, where a later row has the
// block's scale grow, the recoding of its earlier rows exact but for codes that become subnormal.  An infinity becomes
// +-448 and a NaN the code of NaN; neither counts for the scale.
//
// The rows of one block are a run of the call's tokens (consecutive tokens, consecutive slots).  A warp takes K or V
// of one KV head of a run: it holds the up to 16 rows in registers, reduces the largest magnitude, compares it with the
// old scale where the block held rows before (slots are filled in order: the run's first offset says how many), recodes
// those if the scale grows, and writes codes and scale.  One pass over everything, 3 bytes per value: memory bounds the
// long appends (16,384 tokens, 8 heads, D = 128: 17.5 us where nothing is in L2, 86 % of the measured copy rate, 14.4
// where rows are; 65,536 tokens, 2 heads, D = 64: 11.5 and 8.0), launch and three dependent loads the short ones (32
// tokens, 2 heads, D = 64: 2.0).
#include "../../include/kvc.h"
#include "decode_common.cuh"
#include "kvc_internal.h"

namespace kvc {
namespace append8 {

constexpr int kWarps = 4;

struct Params {
    const __half* k;
    const __half* v;
    int64_t k_stride, v_stride;
    const int64_t* slots;
    uint8_t* codes;
    float* scales;
    unsigned* err;
    int64_t n, num_slots;  // tokens; slots of the cache
    int Hkv, tile;         // tokens per warp (1 .. 16)
};

// 2^e for the least e with top <= 448 * 2^e (top: the bits of a finite, not negative fp16 value)
__device__ __forceinline__ float scale_for(uint32_t top) {
    const uint32_t f = __float_as_uint(__half2float(__ushort_as_half(static_cast<unsigned short>(top))));
    if (f == 0) return 0x1p-32f;
    // 448 = 1.75 * 2^8
    return __uint_as_float(((f >> 23) - 8 + ((f & 0x7fffffu) > 0x600000u ? 1 : 0)) << 23);
}

__device__ __forceinline__ uint32_t largest(uint4 x, uint32_t top) {
    const __half2* h = reinterpret_cast<const __half2*>(&x);
    // (a NaN loses every comparison)
    const __half2 m = __hmax2(__hmax2(__habs2(h[0]), __habs2(h[1])), __hmax2(__habs2(h[2]), __habs2(h[3])));
    const __half2 t = __hmax2(m, __half2half2(__ushort_as_half(static_cast<unsigned short>(top))));
    return __half_as_ushort(__hmax(__low2half(t), __high2half(t)));
}
// the same without infinities
__device__ uint32_t largest_finite(uint4 x, uint32_t top) {
    const uint32_t w[4] = {x.x, x.y, x.z, x.w};
    for (int i = 0; i < 8; ++i) {
        const uint32_t a = (w[i >> 1] >> (16 * (i & 1))) & 0x7fffu;
        if (a < 0x7c00u) top = max(top, a);
    }
    return top;
}

__device__ __forceinline__ uint2 codes_of(uint4 x, float inv) {
    uint32_t r[2];
    const uint32_t w[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const float2 a = unpack_half2(w[2 * i]), b = unpack_half2(w[2 * i + 1]);
        r[i] = float2_to_e4m3x2(a.x * inv, a.y * inv) |
               static_cast<uint32_t>(float2_to_e4m3x2(b.x * inv, b.y * inv)) << 16;
    }
    return make_uint2(r[0], r[1]);
}
__device__ __forceinline__ uint32_t recode(uint32_t four, float ratio) {
    const float2 a = unpack_half2(e4m3x2_to_half2(four)), b = unpack_half2(e4m3x2_to_half2(four >> 16));
    return float2_to_e4m3x2(a.x * ratio, a.y * ratio) |
           static_cast<uint32_t>(float2_to_e4m3x2(b.x * ratio, b.y * ratio)) << 16;
}

// Registers for 32 warps on an SM (40 at D = 64), CTAs of four: the loads of a warp follow one another, so what is in
// flight is warps times rows (16,384 tokens of 8 heads, D = 128, 24 warps in CTAs of eight 19.5 us, 32 of eight 18.0, 32 of
// four 17.5, 40 of four 18.3; 65,536 of 2 heads, D = 64, 12.5, 12.4 with 32 and 11.5 with 40).  Tried and slower: rows asked
// for along with the slots (19.2).
template <int D>
__global__ void __launch_bounds__(kWarps * 32, D == 64 ? 10 : 8) kv_append_fp8_block_kernel(const Params p) {
    constexpr int kLanes = D / 8;         // lanes of a row, 8 values each
    constexpr int kRows = 32 / kLanes;    // rows of a pass
    constexpr int kPasses = kBlockSize / kRows;
    const int lane = threadIdx.x & 31;
    const int64_t item = static_cast<int64_t>(blockIdx.x) * kWarps + (threadIdx.x >> 5);
    const int per_tile = 2 * p.Hkv;
    const int64_t t0 = item / per_tile * p.tile;
    const int hk = static_cast<int>(item % per_tile), h = hk >> 1, kv = hk & 1;
    grid_dependency_wait();  // nothing is read or written before the kernel in front is done
    if (t0 >= p.n) return;
    // the tokens that begin a run among this warp's
    const int64_t mine = t0 + lane;
    int64_t slot = -1, prev = -1;
    if (lane < p.tile && mine < p.n) {
        slot = p.slots[mine];
        if (mine > 0) prev = p.slots[mine - 1];
    }
    if (slot >= p.num_slots) {
        if (hk == 0) atomicOr(p.err, KVC_DEVERR_SLOT);
        slot = -1;
    }
    unsigned heads = __ballot_sync(0xffffffffu, slot >= 0 && (slot % kBlockSize == 0 || prev + 1 != slot));
    const __half* const rows = kv ? p.v : p.k;
    const int64_t stride = kv ? p.v_stride : p.k_stride;
    while (heads != 0) {
        const int who = __ffs(heads) - 1;
        heads &= heads - 1;
        const int64_t t = t0 + who, s = __shfl_sync(0xffffffffu, slot, who);
        const int first = static_cast<int>(s % kBlockSize);
        const bool in_run = lane < kBlockSize - first && t + lane < p.n && p.slots[t + lane] == s + lane;
        const int run = __ffs(~__ballot_sync(0xffffffffu, in_run)) - 1;  // 1 .. 16 - first
        const int64_t at = (s / kBlockSize * p.Hkv + h) * 2 + kv;
        uint8_t* const tile = p.codes + at * (kBlockSize * D);
        const float old = first > 0 ? p.scales[at] : 0.f;
        uint4 x[kPasses];
        uint32_t top = 0;
#pragma unroll
        for (int i = 0; i < kPasses; ++i) {
            const int r = i * kRows + lane / kLanes;
            x[i] = make_uint4(0u, 0u, 0u, 0u);
            if (r < run) x[i] = *reinterpret_cast<const uint4*>(rows + (t + r) * stride + h * D + lane % kLanes * 8);
        }
#pragma unroll
        for (int i = 0; i < kPasses; ++i) top = largest(x[i], top);
        top = __reduce_max_sync(0xffffffffu, top);
        if (top >= 0x7c00u) {  // infinities
            top = 0;
#pragma unroll
            for (int i = 0; i < kPasses; ++i) top = largest_finite(x[i], top);
            top = __reduce_max_sync(0xffffffffu, top);
        }
        float scale = scale_for(top);
        if (first > 0) {
            if (old >= scale) {
                scale = old;
            } else {
                const float ratio = old / scale;
                uint4* const held = reinterpret_cast<uint4*>(tile);
                for (int e = lane; e < first * (D / 16); e += 32) {
                    uint4 c = held[e];
                    held[e] = make_uint4(recode(c.x, ratio), recode(c.y, ratio), recode(c.z, ratio), recode(c.w, ratio));
                }
            }
        }
        const float inv = 1.f / scale;
#pragma unroll
        for (int i = 0; i < kPasses; ++i) {
            const int r = i * kRows + lane / kLanes;
            if (r < run) *reinterpret_cast<uint2*>(tile + (first + r) * D + lane % kLanes * 8) = codes_of(x[i], inv);
        }
        if (lane == 0 && !(first > 0 && old == scale)) p.scales[at] = scale;
    }
}

}  // namespace append8

cudaError_t launch_append_fp8_block(const AppendFp8BlockArgs& a, cudaStream_t stream) {
    if (a.n <= 0) return cudaSuccess;
    append8::Params p;
    p.k = a.k;
    p.v = a.v;
    p.k_stride = a.k_stride;
    p.v_stride = a.v_stride;
    p.slots = a.slots;
    p.codes = a.codes;
    p.scales = a.scales;
    p.err = a.err;
    p.n = a.n;
    p.num_slots = static_cast<int64_t>(a.num_blocks) * kBlockSize;
    p.Hkv = a.Hkv;
    // Tokens of a warp: one where there are few, so that the runs of a decode step (a token each) are all worked on at
    // once; 16 where there are many, so that the warps of a prompt's runs are not one in many; 4 between.  8 heads,
    // D = 128, in us with 1 / 4 / 16: 16,384 tokens of prompts 55 / 22 / 14.4, 1024 of a prompt 4.6 / 3.1 / 3.0; steps of
    // 256 sequences 3.1 / 4.6 / 13.6, of 1024 8.5 / 8.0 / 14.4, of 2048 15.5 / 13.9 / 17.9.
    const int64_t units = a.n * 2 * a.Hkv;
    p.tile = units <= 4096 ? 1 : units <= 65536 ? 4 : 16;
    const int64_t items = (p.n + p.tile - 1) / p.tile * 2 * p.Hkv, grid = (items + append8::kWarps - 1) / append8::kWarps;
    if (grid > 2147483647LL) return cudaErrorInvalidConfiguration;
    const dim3 g(static_cast<unsigned>(grid)), block(append8::kWarps * 32);
    return a.D == 64 ? launch(append8::kv_append_fp8_block_kernel<64>, g, block, 0, stream, true, 1u, p)
                     : launch(append8::kv_append_fp8_block_kernel<128>, g, block, 0, stream, true, 1u, p);
}

}  // namespace kvc
