// C-ABI layer: argument validation, checked mode, the cache handle and the
// host-side block management; device work is forwarded to the launchers.
#include <cuda_runtime.h>

#include <algorithm>
#include <atomic>
#include <cmath>
#include <cstdarg>
#include <cstdio>
#include <cstring>
#include <initializer_list>
#include <new>
#include <string>
#include <tuple>
#include <type_traits>
#include <unordered_map>
#include <utility>
#include <vector>

#include "../../include/kvc.h"
#include "block_pool.h"
#include "kvc_internal.h"
#include "stage_copy.h"

struct kvc_cache {
    kvc_config cfg;
    void* k_pool;
    void* v_pool;
    kvc::BlockPool pool;
    kvc_cache(const kvc_config& c, void* k, void* v) : cfg(c), k_pool(k), v_pool(v), pool(c.num_blocks) {}
};

namespace {

thread_local std::string g_last_error;
std::atomic<int> g_checked{0};

kvc_status fail(kvc_status s, const char* fmt, ...) {
    char buf[512];
    va_list ap;
    va_start(ap, fmt);
    vsnprintf(buf, sizeof(buf), fmt, ap);
    va_end(ap);
    g_last_error = buf;
    return s;
}

kvc_status cuda_fail(cudaError_t e, const char* where) {
    return fail(KVC_ERR_CUDA, "%s: %s", where, cudaGetErrorString(e));
}

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

cudaStream_t as_stream(void* s) { return static_cast<cudaStream_t>(s); }

kvc_status check_config(const kvc_config* c) {
    if (!c) return fail(KVC_ERR_INVALID, "null config");
    if (c->num_layers < 1 || c->num_blocks < 1 || c->num_kv_heads < 1 || c->head_dim < 1)
        return fail(KVC_ERR_INVALID, "config sizes must be positive");
    if (c->block_size != kvc::kBlockSize)
        return fail(KVC_ERR_UNSUPPORTED, "block_size %d not supported (16 only)", c->block_size);
    if (c->head_dim != 64 && c->head_dim != 128)
        return fail(KVC_ERR_UNSUPPORTED, "head_dim %d not supported (64, 128)", c->head_dim);
    if (c->dtype != KVC_F16) return fail(KVC_ERR_UNSUPPORTED, "cache dtype must be KVC_F16");
    if (static_cast<int64_t>(c->num_blocks) * c->num_kv_heads * c->block_size >= (int64_t(1) << 31))
        return fail(KVC_ERR_UNSUPPORTED, "num_blocks * num_kv_heads * block_size must be < 2^31");
    return KVC_OK;
}

template <typename T>
kvc_status copy_to_host(std::vector<T>& dst, const T* src, size_t n, cudaStream_t s) {
    dst.resize(n);
    if (n == 0) return KVC_OK;
    cudaError_t e = cudaMemcpyAsync(dst.data(), src, n * sizeof(T), cudaMemcpyDeviceToHost, s);
    if (e == cudaSuccess) e = cudaStreamSynchronize(s);
    if (e != cudaSuccess) return cuda_fail(e, "checked mode copy");
    return KVC_OK;
}

// Checked mode reads device arrays into vectors; running out of host memory there is an error code like any other.
template <typename F>
kvc_status checked(F&& check) {
    if (!g_checked.load()) return KVC_OK;
    try {
        return check();
    } catch (...) {
        return KVC_ERR_OOM;
    }
}

// Arguments from 64-bit words (kvc_call): integers and pointers as they are, a float from a double.
template <typename T>
bool from_word(const unsigned char* at, T* out) {
    if constexpr (std::is_same_v<T, float>) {
        double d;
        std::memcpy(&d, at, 8);
        *out = static_cast<float>(d);
    } else if constexpr (sizeof(T) == 8) {
        std::memcpy(out, at, 8);
    } else {
        int64_t i;
        std::memcpy(&i, at, 8);
        *out = static_cast<T>(i);
        if (static_cast<int64_t>(*out) != i) return false;
    }
    return true;
}
template <typename... A, size_t... I>
kvc_status call_with_words(kvc_status (*fn)(A...), const void* words, int count, void* stream, std::index_sequence<I...>) {
    constexpr int kCount = sizeof...(I);
    if (count != kCount) return fail(KVC_ERR_INVALID, "the call has %d arguments, not %d", kCount, count);
    std::tuple<A...> args;
    const unsigned char* const w = static_cast<const unsigned char*>(words);
    if (!(from_word(w + 8 * I, &std::get<I>(args)) && ...)) return fail(KVC_ERR_INVALID, "an argument beyond its type");
    std::get<kCount>(args) = stream;
    return std::apply(fn, args);
}
template <typename... A>
kvc_status call_with_words(kvc_status (*fn)(A...), const void* words, int count, void* stream) {
    return call_with_words(fn, words, count, stream, std::make_index_sequence<sizeof...(A) - 1>());
}

}  // namespace

int kvc::set_last_error(int status, const char* msg) {
    g_last_error = msg;
    return status;
}

extern "C" {

const char* kvc_last_error_string(void) { return g_last_error.c_str(); }

int kvc_version(void) { return 100; }

kvc_status kvc_set_checked_mode(int on) {
    g_checked.store(on ? 1 : 0);
    return KVC_OK;
}

kvc_status kvc_device_error_flags(uint32_t* flags, int clear) {
    if (!flags) return fail(KVC_ERR_INVALID, "null flags");
    unsigned* w = nullptr;
    cudaError_t e = kvc::device_error_word(&w);
    if (e != cudaSuccess) return cuda_fail(e, "device error word");
    unsigned v = 0;
    e = cudaMemcpy(&v, w, sizeof(v), cudaMemcpyDeviceToHost);
    if (e != cudaSuccess) return cuda_fail(e, "read device error word");
    if (clear) {
        e = cudaMemset(w, 0, sizeof(unsigned));
        if (e == cudaSuccess) e = cudaDeviceSynchronize();
        if (e != cudaSuccess) return cuda_fail(e, "clear device error word");
    }
    *flags = v;
    return KVC_OK;
}

kvc_status kv_cache_pool_bytes(const kvc_config* cfg, size_t* bytes) {
    kvc_status s = check_config(cfg);
    if (s != KVC_OK) return s;
    if (!bytes) return fail(KVC_ERR_INVALID, "null output");
    *bytes = static_cast<size_t>(cfg->num_layers) * cfg->num_blocks * cfg->num_kv_heads * cfg->block_size *
             cfg->head_dim * 2;
    return KVC_OK;
}

kvc_status kv_cache_create(const kvc_config* cfg, void* k_pool, void* v_pool, kvc_handle* out) {
    kvc_status s = check_config(cfg);
    if (s != KVC_OK) return s;
    if (!out) return fail(KVC_ERR_INVALID, "null handle output");
    if ((k_pool == nullptr) != (v_pool == nullptr)) return fail(KVC_ERR_INVALID, "k_pool and v_pool: both or neither");
    if (k_pool && (!aligned16(k_pool) || !aligned16(v_pool))) return fail(KVC_ERR_INVALID, "pools must be 16-byte aligned");
    kvc_cache* h = new (std::nothrow) kvc_cache(*cfg, k_pool, v_pool);
    if (!h) return fail(KVC_ERR_OOM, "host allocation failed");
    *out = h;
    return KVC_OK;
}

kvc_status kv_cache_destroy(kvc_handle h) {
    delete h;
    return KVC_OK;
}

kvc_status kv_cache_layer(kvc_handle h, int layer, void** k_layer, void** v_layer) {
    if (!h || !k_layer || !v_layer) return fail(KVC_ERR_INVALID, "null argument");
    if (!h->k_pool) return fail(KVC_ERR_INVALID, "host-only cache has no device pools");
    if (layer < 0 || layer >= h->cfg.num_layers) return fail(KVC_ERR_INVALID, "layer %d out of range", layer);
    const size_t per = static_cast<size_t>(h->cfg.num_blocks) * h->cfg.num_kv_heads * h->cfg.block_size *
                       h->cfg.head_dim * 2;
    *k_layer = static_cast<char*>(h->k_pool) + per * layer;
    *v_layer = static_cast<char*>(h->v_pool) + per * layer;
    return KVC_OK;
}

kvc_status kv_block_alloc(kvc_handle h, int32_t* block) {
    if (!h || !block) return fail(KVC_ERR_INVALID, "null argument");
    auto lk = h->pool.lock();
    const int32_t b = h->pool.alloc();
    if (b < 0) return fail(KVC_ERR_OOM, "OOM -- no free blocks");
    *block = b;
    return KVC_OK;
}

kvc_status kv_block_share(kvc_handle h, int32_t block) {
    if (!h) return fail(KVC_ERR_INVALID, "null handle");
    auto lk = h->pool.lock();
    if (!h->pool.live(block)) return fail(KVC_ERR_INVALID, "block %d is not live", block);
    h->pool.share(block);
    return KVC_OK;
}

kvc_status kv_block_release(kvc_handle h, int32_t block) {
    if (!h) return fail(KVC_ERR_INVALID, "null handle");
    auto lk = h->pool.lock();
    if (!h->pool.live(block)) return fail(KVC_ERR_INVALID, "block %d is not live", block);
    h->pool.release(block);
    return KVC_OK;
}

kvc_status kv_block_refcount(kvc_handle h, int32_t block, int32_t* refcount) {
    if (!h || !refcount) return fail(KVC_ERR_INVALID, "null argument");
    if (block < 0 || block >= h->cfg.num_blocks) return fail(KVC_ERR_INVALID, "block %d out of range", block);
    auto lk = h->pool.lock();
    *refcount = h->pool.refcount(block);
    return KVC_OK;
}

kvc_status kv_block_num_free(kvc_handle h, int32_t* num_free) {
    if (!h || !num_free) return fail(KVC_ERR_INVALID, "null argument");
    auto lk = h->pool.lock();
    *num_free = h->pool.num_free();
    return KVC_OK;
}

kvc_status kv_cache_utilisation(kvc_handle h, double* percent) {
    if (!h || !percent) return fail(KVC_ERR_INVALID, "null argument");
    auto lk = h->pool.lock();
    *percent = static_cast<double>(h->pool.total() - h->pool.num_free()) / h->pool.total() * 100.0;
    return KVC_OK;
}

static kvc_status copy_blocks_device(kvc_handle h, const int32_t* src, const int32_t* dst, int n, void* stream) {
    const int64_t block_elems = static_cast<int64_t>(h->cfg.num_kv_heads) * h->cfg.block_size * h->cfg.head_dim;
    cudaError_t e = kvc::launch_copy_blocks(src, dst, n, static_cast<__half*>(h->k_pool), static_cast<__half*>(h->v_pool),
                                            h->cfg.num_layers, h->cfg.num_blocks, block_elems, as_stream(stream));
    if (e != cudaSuccess) return cuda_fail(e, "copy_blocks launch");
    return KVC_OK;
}

kvc_status kv_copy_blocks(kvc_handle h, const int32_t* src, const int32_t* dst, int n, void* stream) {
    if (!h) return fail(KVC_ERR_INVALID, "null handle");
    if (n < 0 || (n > 0 && (!src || !dst))) return fail(KVC_ERR_INVALID, "bad copy list");
    if (n == 0) return KVC_OK;
    if (!h->k_pool) return fail(KVC_ERR_INVALID, "host-only cache has no device pools");
    for (int i = 0; i < n; ++i)
        if (src[i] < 0 || src[i] >= h->cfg.num_blocks || dst[i] < 0 || dst[i] >= h->cfg.num_blocks)
            return fail(KVC_ERR_INVALID, "copy pair %d (%d -> %d) out of range", i, src[i], dst[i]);
    return copy_blocks_device(h, src, dst, n, stream);
}

kvc_status kv_block_cow(kvc_handle h, int32_t block, int32_t* new_block, void* stream) {
    if (!h || !new_block) return fail(KVC_ERR_INVALID, "null argument");
    int32_t nb;
    {
        auto lk = h->pool.lock();
        if (!h->pool.live(block)) return fail(KVC_ERR_INVALID, "block %d is not live", block);
        if (h->pool.refcount(block) <= 1) {
            *new_block = block;
            return KVC_OK;
        }
        if (!h->k_pool) return fail(KVC_ERR_INVALID, "host-only cache has no device pools");
        nb = h->pool.alloc();
        if (nb < 0) return fail(KVC_ERR_OOM, "OOM -- no free blocks for copy-on-write");
        h->pool.release(block);
    }
    kvc_status s = copy_blocks_device(h, &block, &nb, 1, stream);
    if (s != KVC_OK) return s;
    *new_block = nb;
    return KVC_OK;
}

kvc_status kv_slot_mapping(const int32_t* block_table, int max_blocks, int B, const int32_t* first_pos,
                           const int32_t* count, int block_size, int64_t* slots) {
    if (B < 0 || max_blocks < 1 || block_size < 1) return fail(KVC_ERR_INVALID, "bad sizes");
    if (B > 0 && (!block_table || !first_pos || !count || !slots)) return fail(KVC_ERR_INVALID, "null argument");
    int64_t o = 0;
    for (int b = 0; b < B; ++b) {
        if (first_pos[b] < 0 || count[b] < 0) return fail(KVC_ERR_INVALID, "sequence %d: negative position/count", b);
        for (int32_t k = 0; k < count[b]; ++k) {
            const int64_t pos = static_cast<int64_t>(first_pos[b]) + k;
            const int64_t j = pos / block_size;
            if (j >= max_blocks) return fail(KVC_ERR_CAPACITY, "sequence %d: position %lld beyond its block table", b, (long long)pos);
            const int32_t blk = block_table[static_cast<int64_t>(b) * max_blocks + j];
            if (blk < 0) return fail(KVC_ERR_CAPACITY, "sequence %d: no block for position %lld", b, (long long)pos);
            slots[o++] = static_cast<int64_t>(blk) * block_size + pos % block_size;
        }
    }
    return KVC_OK;
}

kvc_status kv_step_prepare(kvc_handle h, int32_t* block_table, int max_blocks, int32_t* num_blocks,
                           const int32_t* positions, int B, int64_t* slot_mapping, int32_t* copy_src,
                           int32_t* copy_dst, int* n_copies) {
    if (!h || B < 0 || max_blocks < 1) return fail(KVC_ERR_INVALID, "bad arguments");
    if (!n_copies || (B > 0 && (!block_table || !num_blocks || !positions || !slot_mapping || !copy_src || !copy_dst)))
        return fail(KVC_ERR_INVALID, "null argument");
    const int bs = h->cfg.block_size;
    auto lk = h->pool.lock();
    // dry run: validate and count the blocks this step needs
    std::unordered_map<int32_t, int32_t> taken;  // references dropped by earlier copies in this step
    int32_t need = 0;
    for (int b = 0; b < B; ++b) {
        const int32_t pos = positions[b], nb = num_blocks[b];
        if (pos < 0 || nb < 0 || nb > max_blocks) return fail(KVC_ERR_INVALID, "sequence %d: bad position/num_blocks", b);
        const int32_t j = pos / bs;
        if (j == nb) {
            if (nb == max_blocks) return fail(KVC_ERR_CAPACITY, "sequence %d: block table full", b);
            ++need;
        } else if (j < nb) {
            const int32_t blk = block_table[static_cast<int64_t>(b) * max_blocks + j];
            if (!h->pool.live(blk)) return fail(KVC_ERR_INVALID, "sequence %d: block %d is not live", b, blk);
            const int32_t rc = h->pool.refcount(blk) - taken[blk];
            if (rc > 1) {
                ++need;
                ++taken[blk];
            }
        } else {
            return fail(KVC_ERR_CAPACITY, "sequence %d: position %d skips past its last block", b, pos);
        }
    }
    if (need > h->pool.num_free()) return fail(KVC_ERR_OOM, "OOM -- step needs %d blocks, %d free", need, h->pool.num_free());
    int nc = 0;
    for (int b = 0; b < B; ++b) {
        const int32_t pos = positions[b];
        const int32_t j = pos / bs;
        int32_t* row = block_table + static_cast<int64_t>(b) * max_blocks;
        if (j == num_blocks[b]) {
            row[j] = h->pool.alloc();
            ++num_blocks[b];
        } else {
            const int32_t blk = row[j];
            if (h->pool.refcount(blk) > 1) {
                const int32_t nb = h->pool.alloc();
                h->pool.release(blk);
                copy_src[nc] = blk;
                copy_dst[nc] = nb;
                ++nc;
                row[j] = nb;
            }
        }
        slot_mapping[b] = static_cast<int64_t>(row[j]) * bs + pos % bs;
    }
    *n_copies = nc;
    return KVC_OK;
}

kvc_status kv_append(kvc_handle h, int layer, const void* k_new, const void* v_new, const int64_t* slot_mapping, int n,
                     void* stream) {
    if (!h) return fail(KVC_ERR_INVALID, "null handle");
    if (!h->k_pool) return fail(KVC_ERR_INVALID, "host-only cache has no device pools");
    if (layer < 0 || layer >= h->cfg.num_layers) return fail(KVC_ERR_INVALID, "layer %d out of range", layer);
    if (n < 0) return fail(KVC_ERR_INVALID, "negative n");
    if (n == 0) return KVC_OK;
    if (!k_new || !v_new || !slot_mapping) return fail(KVC_ERR_INVALID, "null pointer");
    if (!aligned16(k_new) || !aligned16(v_new)) return fail(KVC_ERR_INVALID, "k_new/v_new must be 16-byte aligned");
    if (g_checked.load()) {
        std::vector<int64_t> s;
        kvc_status st = copy_to_host(s, slot_mapping, static_cast<size_t>(n), as_stream(stream));
        if (st != KVC_OK) return st;
        const int64_t cap = static_cast<int64_t>(h->cfg.num_blocks) * h->cfg.block_size;
        for (int t = 0; t < n; ++t)
            if (s[t] >= cap) return fail(KVC_ERR_CAPACITY, "slot %lld of token %d beyond the pool (%lld slots)", (long long)s[t], t, (long long)cap);
    }
    void *kl, *vl;
    kv_cache_layer(h, layer, &kl, &vl);
    unsigned* err = nullptr;
    cudaError_t e = kvc::device_error_word(&err);
    if (e != cudaSuccess) return cuda_fail(e, "device error word");
    e = kvc::launch_append(static_cast<const __half*>(k_new), static_cast<const __half*>(v_new), slot_mapping, n,
                           static_cast<__half*>(kl), static_cast<__half*>(vl), h->cfg.num_blocks, h->cfg.num_kv_heads,
                           h->cfg.head_dim, err, as_stream(stream));
    if (e != cudaSuccess) return cuda_fail(e, "kv_append launch");
    return KVC_OK;
}

static kvc_status check_decode_shape(int B, int Hq, int Hkv, int head_dim, int block_size, int max_context_len) {
    if (B < 0 || Hq < 1 || Hkv < 1 || max_context_len < 1) return fail(KVC_ERR_INVALID, "bad sizes");
    if (Hq % Hkv) return fail(KVC_ERR_INVALID, "Hq (%d) must be a multiple of Hkv (%d)", Hq, Hkv);
    if (Hq / Hkv > kvc::kMaxGroupHeads)
        return fail(KVC_ERR_UNSUPPORTED, "group size %d > %d not supported", Hq / Hkv, kvc::kMaxGroupHeads);
    if (head_dim != 64 && head_dim != 128) return fail(KVC_ERR_UNSUPPORTED, "head_dim %d not supported", head_dim);
    if (block_size != kvc::kBlockSize) return fail(KVC_ERR_UNSUPPORTED, "block_size %d not supported", block_size);
    if (B > 65535 || Hkv > 65535) return fail(KVC_ERR_UNSUPPORTED, "B and Hkv must be <= 65535");
    return KVC_OK;
}

kvc_status paged_decode_plan(int B, int Hq, int Hkv, int head_dim, int block_size, int max_context_len,
                             int blocks_per_split, int* num_splits, int* blocks_per_split_out, size_t* workspace_bytes) {
    kvc_status s = check_decode_shape(B, Hq, Hkv, head_dim, block_size, max_context_len);
    if (s != KVC_OK) return s;
    kvc::DecodePlan plan;
    cudaError_t e = kvc::decode_plan(B, Hq, Hkv, head_dim, max_context_len, blocks_per_split, &plan);
    if (e != cudaSuccess) return cuda_fail(e, "decode plan");
    if (num_splits) *num_splits = plan.num_splits;
    if (blocks_per_split_out) *blocks_per_split_out = plan.blocks_per_split;
    if (workspace_bytes) *workspace_bytes = plan.workspace_bytes;
    return KVC_OK;
}

kvc_status paged_decode_workspace_init(void* workspace, size_t bytes, void* stream) {
    if (bytes == 0) return KVC_OK;
    if (!workspace) return fail(KVC_ERR_INVALID, "null workspace");
    cudaError_t e = cudaMemsetAsync(workspace, 0, bytes, as_stream(stream));
    if (e != cudaSuccess) return cuda_fail(e, "workspace init");
    return KVC_OK;
}

kvc_status kvc_trace_read(void* records, int capacity, int* count, int clear) {
    if (!count || capacity < 0 || (capacity > 0 && !records)) return fail(KVC_ERR_INVALID, "bad arguments");
    cudaError_t e = kvc::trace_read(records, capacity, count, clear);
    if (e == cudaErrorNotSupported) return fail(KVC_ERR_UNSUPPORTED, "library built without -DKVC_TRACE=1");
    if (e != cudaSuccess) return cuda_fail(e, "trace read");
    return KVC_OK;
}

kvc_status kvc_set_launch_overlap(int on) {
    kvc::set_launch_overlap(on);
    return KVC_OK;
}

kvc_status kvc_set_multi_tc(int on) {
    kvc::set_multi_tc(on);
    return KVC_OK;
}

kvc_status kvc_set_cascade_min_saved_blocks(int blocks) {
    if (blocks < 0) return fail(KVC_ERR_INVALID, "negative block count %d", blocks);
    kvc::set_cascade_min_saved_blocks(blocks);
    return KVC_OK;
}

// The address the current device uses for p: device and managed memory as they are, pinned host memory
// through its mapping.  False for pageable host memory and unknown pointers.
static bool device_address(const void* p, void** out) {
    cudaPointerAttributes a;
    if (cudaPointerGetAttributes(&a, p) != cudaSuccess) {
        cudaGetLastError();
        return false;
    }
    if (a.type != cudaMemoryTypeDevice && a.type != cudaMemoryTypeManaged && a.type != cudaMemoryTypeHost)
        return false;
    if (!a.devicePointer) return false;
    *out = a.devicePointer;
    return true;
}

kvc_status kvc_copy_async(void* dst, const void* src, size_t bytes, unsigned flags, void* stream) {
    if (flags & ~KVC_COPY_AHEAD) return fail(KVC_ERR_INVALID, "unknown flags 0x%x", flags);
    if (bytes == 0) return KVC_OK;
    if (!dst || !src) return fail(KVC_ERR_INVALID, "null buffer");
    if ((bytes & 15u) || !aligned16(dst) || !aligned16(src))
        return fail(KVC_ERR_INVALID, "both buffers 16-byte aligned and bytes a multiple of 16 (got %zu)", bytes);
    const uintptr_t d0 = reinterpret_cast<uintptr_t>(dst), s0 = reinterpret_cast<uintptr_t>(src);
    if (d0 < s0 + bytes && s0 < d0 + bytes) return fail(KVC_ERR_INVALID, "source and destination overlap");
    void *ddev = nullptr, *sdev = nullptr;
    if (!device_address(dst, &ddev)) return fail(KVC_ERR_INVALID, "dst is neither device nor pinned host memory");
    if (!device_address(src, &sdev)) return fail(KVC_ERR_INVALID, "src is neither device nor pinned host memory");
    cudaError_t e = kvc::launch_stage_copy(ddev, sdev, bytes, (flags & KVC_COPY_AHEAD) != 0,
                                           static_cast<cudaStream_t>(stream));
    if (e != cudaSuccess) return cuda_fail(e, "staging copy launch");
    return KVC_OK;
}

static kvc_status decode_common(const void* q, const void* k_new, const void* v_new, const void* k_cache,
                                const void* v_cache, int num_blocks,
                                const int32_t* block_table, int max_blocks, const int32_t* context_lens, int B, int Hq,
                                int Hkv, int head_dim, int block_size, int max_context_len, float scale, void* out,
                                int out_dtype, void* workspace, size_t workspace_bytes, int blocks_per_split,
                                void* stream);

kvc_status paged_decode_attention(const void* q, const void* k_cache, const void* v_cache, int num_blocks,
                                  const int32_t* block_table, int max_blocks, const int32_t* context_lens, int B, int Hq,
                                  int Hkv, int head_dim, int block_size, int max_context_len, float scale, void* out,
                                  int out_dtype, void* workspace, size_t workspace_bytes, int blocks_per_split,
                                  void* stream) {
    return decode_common(q, nullptr, nullptr, k_cache, v_cache, num_blocks, block_table, max_blocks,
                         context_lens, B, Hq, Hkv, head_dim, block_size, max_context_len, scale, out, out_dtype,
                         workspace, workspace_bytes, blocks_per_split, stream);
}

kvc_status paged_decode_append_attention(const void* q, const void* k_new, const void* v_new, void* k_cache,
                                         void* v_cache, int num_blocks,
                                         const int32_t* block_table, int max_blocks, const int32_t* context_lens,
                                         int B, int Hq, int Hkv, int head_dim, int block_size, int max_context_len,
                                         float scale, void* out, int out_dtype, void* workspace,
                                         size_t workspace_bytes, int blocks_per_split, void* stream) {
    if (B > 0 && (!k_new || !v_new)) return fail(KVC_ERR_INVALID, "null k_new/v_new");
    if (!aligned16(k_new) || !aligned16(v_new)) return fail(KVC_ERR_INVALID, "k_new/v_new must be 16-byte aligned");
    return decode_common(q, k_new, v_new, k_cache, v_cache, num_blocks, block_table, max_blocks,
                         context_lens, B, Hq, Hkv, head_dim, block_size, max_context_len, scale, out, out_dtype,
                         workspace, workspace_bytes, blocks_per_split, stream);
}

// Every argument check of a decode call; in checked mode also the context lengths and the block-table
// entries, on host copies that are returned through ctx / table (left empty otherwise).
static kvc_status decode_validate(const void* q, const void* k_cache, const void* v_cache, int num_blocks,
                                  const int32_t* block_table, int max_blocks, const int32_t* context_lens, int B,
                                  int Hq, int Hkv, int head_dim, int block_size, int max_context_len, void* out,
                                  int out_dtype, int blocks_per_split, void* stream, std::vector<int32_t>& ctx,
                                  std::vector<int32_t>& table) {
    kvc_status s = check_decode_shape(B, Hq, Hkv, head_dim, block_size, max_context_len);
    if (s != KVC_OK) return s;
    if (B == 0) return KVC_OK;
    if (!q || !k_cache || !v_cache || !block_table || !context_lens || !out) return fail(KVC_ERR_INVALID, "null pointer");
    if (!aligned16(q) || !aligned16(k_cache) || !aligned16(v_cache) || !aligned16(out))
        return fail(KVC_ERR_INVALID, "q, caches and out must be 16-byte aligned");
    if (num_blocks < 1 || max_blocks < 1) return fail(KVC_ERR_INVALID, "num_blocks and max_blocks must be positive");
    if (static_cast<int64_t>(num_blocks) * Hkv * block_size >= (int64_t(1) << 31))
        return fail(KVC_ERR_UNSUPPORTED, "num_blocks * Hkv * block_size must be < 2^31");
    if (static_cast<int64_t>(max_context_len) > static_cast<int64_t>(max_blocks) * block_size)
        return fail(KVC_ERR_CAPACITY, "max_context_len %d beyond max_blocks * block_size", max_context_len);
    if (out_dtype != KVC_F16 && out_dtype != KVC_F32) return fail(KVC_ERR_INVALID, "bad out_dtype");
    if (blocks_per_split < 0) return fail(KVC_ERR_INVALID, "negative blocks_per_split");
    if (g_checked.load()) {
        kvc_status st = copy_to_host(ctx, context_lens, static_cast<size_t>(B), as_stream(stream));
        if (st == KVC_OK) st = copy_to_host(table, block_table, static_cast<size_t>(B) * max_blocks, as_stream(stream));
        if (st != KVC_OK) return st;
        for (int b = 0; b < B; ++b) {
            if (ctx[b] < 1 || ctx[b] > max_context_len)
                return fail(KVC_ERR_CAPACITY, "sequence %d: context length %d outside [1, %d]", b, ctx[b], max_context_len);
            for (int j = 0; j < (ctx[b] + block_size - 1) / block_size; ++j) {
                const int32_t blk = table[static_cast<size_t>(b) * max_blocks + j];
                if (blk < 0 || blk >= num_blocks)
                    return fail(KVC_ERR_INVALID, "sequence %d: block-table entry %d = %d outside [0, %d)", b, j, blk, num_blocks);
            }
        }
    }
    return KVC_OK;
}

static kvc::DecodeArgs decode_args(const void* q, const void* k_new, const void* v_new, const void* k_cache,
                                   const void* v_cache, int num_blocks,
                                   const int32_t* block_table, int max_blocks, const int32_t* context_lens, int B,
                                   int Hq, int Hkv, int head_dim, int max_context_len, float scale, void* out,
                                   int out_dtype, void* workspace, size_t workspace_bytes, int blocks_per_split) {
    kvc::DecodeArgs a;
    a.q = static_cast<const __half*>(q);
    a.k_new = static_cast<const __half*>(k_new);
    a.v_new = static_cast<const __half*>(v_new);
    a.k_cache = static_cast<const __half*>(k_cache);
    a.v_cache = static_cast<const __half*>(v_cache);
    a.num_blocks = num_blocks;
    a.block_table = block_table;
    a.max_blocks = max_blocks;
    a.context_lens = context_lens;
    a.B = B;
    a.Hq = Hq;
    a.Hkv = Hkv;
    a.D = head_dim;
    a.max_context_len = max_context_len;
    a.scale = scale;
    a.out = out;
    a.out_f32 = out_dtype == KVC_F32;
    a.workspace = workspace;
    a.workspace_bytes = workspace_bytes;
    a.blocks_per_split = blocks_per_split;
    a.err = nullptr;
    return a;
}

static kvc_status check_workspace(size_t need, const void* workspace, size_t workspace_bytes) {
    if (need > workspace_bytes || (need && !workspace))
        return fail(KVC_ERR_INVALID, "workspace too small: need %zu bytes", need);
    if (need && !aligned16(workspace)) return fail(KVC_ERR_INVALID, "workspace must be 16-byte aligned");
    return KVC_OK;
}

static kvc_status decode_common(const void* q, const void* k_new, const void* v_new, const void* k_cache,
                                const void* v_cache, int num_blocks,
                                const int32_t* block_table, int max_blocks, const int32_t* context_lens, int B, int Hq,
                                int Hkv, int head_dim, int block_size, int max_context_len, float scale, void* out,
                                int out_dtype, void* workspace, size_t workspace_bytes, int blocks_per_split,
                                void* stream) {
    std::vector<int32_t> ctx, table;
    kvc_status s = decode_validate(q, k_cache, v_cache, num_blocks, block_table, max_blocks, context_lens, B, Hq, Hkv,
                                   head_dim, block_size, max_context_len, out, out_dtype, blocks_per_split, stream, ctx,
                                   table);
    if (s != KVC_OK || B == 0) return s;
    kvc::DecodeArgs a = decode_args(q, k_new, v_new, k_cache, v_cache, num_blocks, block_table,
                                    max_blocks, context_lens, B, Hq, Hkv, head_dim, max_context_len, scale, out,
                                    out_dtype, workspace, workspace_bytes, blocks_per_split);
    kvc::DecodePlan plan;
    cudaError_t e = kvc::decode_plan(B, Hq, Hkv, head_dim, max_context_len, blocks_per_split, &plan);
    if (e != cudaSuccess) return cuda_fail(e, "decode plan");
    s = check_workspace(plan.workspace_bytes, workspace, workspace_bytes);
    if (s != KVC_OK) return s;
    e = kvc::device_error_word(&a.err);
    if (e != cudaSuccess) return cuda_fail(e, "device error word");
    e = kvc::launch_decode(a, as_stream(stream));
    if (e != cudaSuccess) return cuda_fail(e, k_new ? "paged_decode_append_attention launch" : "paged_decode_attention launch");
    return KVC_OK;
}

kvc_status kv_cascade_groups(const int32_t* block_table, int B, int max_blocks, const int32_t* context_lens,
                             int block_size, int max_group, int32_t* group_start, int* n_groups,
                             int32_t* shared_blocks, int* max_shared) {
    if (B < 0 || max_blocks < 1 || block_size < 1) return fail(KVC_ERR_INVALID, "bad sizes");
    if (max_group < 1 || max_group > kvc::kMaxGroupSize)
        return fail(KVC_ERR_INVALID, "max_group %d outside [1, %d]", max_group, kvc::kMaxGroupSize);
    if (B > 0 && (!block_table || !context_lens || !group_start || !n_groups || !shared_blocks || !max_shared))
        return fail(KVC_ERR_INVALID, "null pointer");
    int ng = 0, mx = 0;
    group_start[0] = 0;
    for (int g0 = 0; g0 < B;) {
        const int32_t* r0 = block_table + static_cast<size_t>(g0) * max_blocks;
        int g1 = g0 + 1;  // members: consecutive rows that start with the same block, at most max_group
        while (g1 < B && g1 - g0 < max_group && block_table[static_cast<size_t>(g1) * max_blocks] == r0[0]) ++g1;
        int shared = 0;
        if (g1 - g0 > 1) {
            int cap = max_blocks;
            for (int b = g0; b < g1; ++b) {
                if (context_lens[b] < 1) return fail(KVC_ERR_INVALID, "sequence %d: context length %d", b, context_lens[b]);
                cap = std::min(cap, (context_lens[b] - 1) / block_size);
            }
            while (shared < cap) {
                bool same = true;
                for (int b = g0 + 1; b < g1 && same; ++b)
                    same = block_table[static_cast<size_t>(b) * max_blocks + shared] == r0[shared];
                if (!same) break;
                ++shared;
            }
        }
        for (int b = g0; b < g1; ++b) shared_blocks[b] = shared;
        mx = std::max(mx, shared);
        group_start[++ng] = g1;
        g0 = g1;
    }
    *n_groups = ng;
    *max_shared = mx;
    return KVC_OK;
}

kvc_status paged_decode_cascade_plan(int B, int Hq, int Hkv, int head_dim, int block_size, int max_context_len,
                                     int n_groups, int max_shared_blocks, size_t* workspace_bytes) {
    kvc_status s = check_decode_shape(B, Hq, Hkv, head_dim, block_size, max_context_len);
    if (s != KVC_OK) return s;
    if (n_groups < 0 || max_shared_blocks < 0) return fail(KVC_ERR_INVALID, "bad group sizes");
    kvc::CascadePlan plan;
    cudaError_t e = kvc::cascade_plan(B, Hq, Hkv, head_dim, max_context_len, std::max(n_groups, 1),
                                      max_shared_blocks, &plan);
    if (e != cudaSuccess) return cuda_fail(e, "cascade plan");
    if (workspace_bytes) *workspace_bytes = plan.workspace_bytes;
    return KVC_OK;
}

kvc_status paged_decode_cascade_attention(const void* q, const void* k_cache, const void* v_cache, int num_blocks,
                                          const int32_t* block_table, int max_blocks, const int32_t* context_lens,
                                          const int32_t* group_start, const int32_t* shared_blocks, int n_groups,
                                          int max_shared_blocks, int B, int Hq, int Hkv, int head_dim,
                                          int block_size, int max_context_len, float scale, void* out, int out_dtype,
                                          void* workspace, size_t workspace_bytes, void* stream) {
    std::vector<int32_t> ctx, table;
    kvc_status s = decode_validate(q, k_cache, v_cache, num_blocks, block_table, max_blocks, context_lens, B, Hq, Hkv,
                                   head_dim, block_size, max_context_len, out, out_dtype, 0, stream, ctx, table);
    if (s != KVC_OK || B == 0) return s;
    if (!group_start || !shared_blocks) return fail(KVC_ERR_INVALID, "null group_start / shared_blocks");
    if (n_groups < 1 || n_groups > B) return fail(KVC_ERR_INVALID, "n_groups %d outside [1, B = %d]", n_groups, B);
    if (max_shared_blocks < 0 || max_shared_blocks >= max_blocks)
        return fail(KVC_ERR_INVALID, "max_shared_blocks %d outside [0, max_blocks)", max_shared_blocks);
    if (g_checked.load()) {
        std::vector<int32_t> gs, sh;
        s = copy_to_host(gs, group_start, static_cast<size_t>(n_groups) + 1, as_stream(stream));
        if (s == KVC_OK) s = copy_to_host(sh, shared_blocks, static_cast<size_t>(B), as_stream(stream));
        if (s != KVC_OK) return s;
        if (gs[0] != 0 || gs[n_groups] != B) return fail(KVC_ERR_INVALID, "group_start must run from 0 to B");
        for (int g = 0; g < n_groups; ++g) {
            const int g0 = gs[g], g1 = gs[g + 1];
            if (g1 <= g0 || g1 - g0 > kvc::kMaxGroupSize)
                return fail(KVC_ERR_INVALID, "group %d: %d members (1..%d)", g, g1 - g0, kvc::kMaxGroupSize);
            for (int b = g0; b < g1; ++b) {
                if (sh[b] != sh[g0]) return fail(KVC_ERR_INVALID, "group %d: members share different block counts", g);
                if (sh[b] < 0 || sh[b] > max_shared_blocks || static_cast<int64_t>(sh[b]) * block_size >= ctx[b])
                    return fail(KVC_ERR_INVALID, "sequence %d: %d shared blocks do not fit its context %d (or the bound %d)",
                                b, sh[b], ctx[b], max_shared_blocks);
                for (int j = 0; j < sh[b]; ++j)
                    if (table[static_cast<size_t>(b) * max_blocks + j] != table[static_cast<size_t>(g0) * max_blocks + j])
                        return fail(KVC_ERR_INVALID, "sequence %d: block %d is not the group's shared block", b, j);
            }
        }
    }
    kvc::DecodeArgs a = decode_args(q, nullptr, nullptr, k_cache, v_cache, num_blocks, block_table,
                                    max_blocks, context_lens, B, Hq, Hkv, head_dim, max_context_len, scale, out,
                                    out_dtype, workspace, workspace_bytes, 0);
    kvc::CascadePlan plan;
    cudaError_t e = kvc::cascade_plan(B, Hq, Hkv, head_dim, max_context_len, n_groups, max_shared_blocks, &plan);
    if (e != cudaSuccess) return cuda_fail(e, "cascade plan");
    s = check_workspace(plan.workspace_bytes, workspace, workspace_bytes);
    if (s != KVC_OK) return s;
    e = kvc::device_error_word(&a.err);
    if (e != cudaSuccess) return cuda_fail(e, "device error word");
    e = kvc::launch_cascade(a, group_start, shared_blocks, n_groups, max_shared_blocks, as_stream(stream));
    if (e != cudaSuccess) return cuda_fail(e, "paged_decode_cascade_attention launch");
    return KVC_OK;
}

kvc_status kv_fp8_record_bytes(int head_dim, size_t* bytes) {
    if (head_dim != 64 && head_dim != 128) return fail(KVC_ERR_UNSUPPORTED, "head_dim %d not supported", head_dim);
    if (!bytes) return fail(KVC_ERR_INVALID, "null pointer");
    *bytes = static_cast<size_t>(kvc::fp8_record_bytes(head_dim));
    return KVC_OK;
}

kvc_status kv_append_fp8(const void* k_new, const void* v_new, const int64_t* slot_mapping, int n, void* kv_fp8,
                         int num_blocks, int Hkv, int head_dim, int block_size, void* stream) {
    if (n < 0 || num_blocks < 1 || Hkv < 1) return fail(KVC_ERR_INVALID, "bad sizes");
    if (head_dim != 64 && head_dim != 128) return fail(KVC_ERR_UNSUPPORTED, "head_dim %d not supported", head_dim);
    if (block_size != kvc::kBlockSize) return fail(KVC_ERR_UNSUPPORTED, "block_size %d not supported", block_size);
    if (n == 0) return KVC_OK;
    if (!k_new || !v_new || !slot_mapping || !kv_fp8) return fail(KVC_ERR_INVALID, "null pointer");
    if (!aligned16(k_new) || !aligned16(v_new) || !aligned16(kv_fp8))
        return fail(KVC_ERR_INVALID, "device buffers must be 16-byte aligned");
    if (g_checked.load()) {
        std::vector<int64_t> sl;
        kvc_status st = copy_to_host(sl, slot_mapping, static_cast<size_t>(n), as_stream(stream));
        if (st != KVC_OK) return st;
        for (int t = 0; t < n; ++t)
            if (sl[t] >= static_cast<int64_t>(num_blocks) * block_size)
                return fail(KVC_ERR_CAPACITY, "token %d: slot %lld beyond the pool", t, static_cast<long long>(sl[t]));
    }
    unsigned* err = nullptr;
    cudaError_t e = kvc::device_error_word(&err);
    if (e != cudaSuccess) return cuda_fail(e, "device error word");
    e = kvc::launch_append_fp8(static_cast<const __half*>(k_new), static_cast<const __half*>(v_new), slot_mapping, n,
                               static_cast<uint8_t*>(kv_fp8), num_blocks, Hkv, head_dim, err, as_stream(stream));
    if (e != cudaSuccess) return cuda_fail(e, "kv_append_fp8 launch");
    return KVC_OK;
}

kvc_status paged_decode_attention_fp8(const void* q, const void* kv_fp8, int num_blocks, const int32_t* block_table,
                                      int max_blocks, const int32_t* context_lens, int B, int Hq, int Hkv,
                                      int head_dim, int block_size, int max_context_len, float scale, void* out,
                                      int out_dtype, void* workspace, size_t workspace_bytes, int blocks_per_split,
                                      void* stream) {
    std::vector<int32_t> ctx, table;
    kvc_status s = decode_validate(q, kv_fp8, kv_fp8, num_blocks, block_table, max_blocks, context_lens, B, Hq, Hkv,
                                   head_dim, block_size, max_context_len, out, out_dtype, blocks_per_split, stream, ctx,
                                   table);
    if (s != KVC_OK || B == 0) return s;
    kvc::DecodeArgs a = decode_args(q, nullptr, nullptr, nullptr, nullptr, num_blocks, block_table,
                                    max_blocks, context_lens, B, Hq, Hkv, head_dim, max_context_len, scale, out,
                                    out_dtype, workspace, workspace_bytes, blocks_per_split);
    a.kv_fp8 = static_cast<const uint8_t*>(kv_fp8);
    kvc::DecodePlan plan;
    cudaError_t e = kvc::decode_plan(B, Hq, Hkv, head_dim, max_context_len, blocks_per_split, &plan);
    if (e != cudaSuccess) return cuda_fail(e, "decode plan");
    s = check_workspace(plan.workspace_bytes, workspace, workspace_bytes);
    if (s != KVC_OK) return s;
    e = kvc::device_error_word(&a.err);
    if (e != cudaSuccess) return cuda_fail(e, "device error word");
    e = kvc::launch_decode(a, as_stream(stream));
    if (e != cudaSuccess) return cuda_fail(e, "paged_decode_attention_fp8 launch");
    return KVC_OK;
}

kvc_status paged_decode_multi_plan(int B, int Hq, int Hkv, int head_dim, int block_size, int max_context_len,
                                   int q_len, size_t* workspace_bytes) {
    kvc_status s = check_decode_shape(B, Hq, Hkv, head_dim, block_size, max_context_len);
    if (s != KVC_OK) return s;
    if (q_len < 1 || q_len > kvc::kMaxQueryTokens)
        return fail(KVC_ERR_UNSUPPORTED, "q_len %d outside [1, %d]", q_len, kvc::kMaxQueryTokens);
    kvc::MultiPlan plan;
    cudaError_t e = kvc::multi_plan(B, Hq, Hkv, head_dim, max_context_len, q_len, &plan);
    if (e != cudaSuccess) return cuda_fail(e, "multi-token plan");
    if (workspace_bytes) *workspace_bytes = plan.workspace_bytes;
    return KVC_OK;
}

kvc_status paged_decode_multi_attention(const void* q, const void* k_cache, const void* v_cache, int num_blocks,
                                        const int32_t* block_table, int max_blocks, const int32_t* context_lens,
                                        int q_len, int B, int Hq, int Hkv, int head_dim, int block_size,
                                        int max_context_len, float scale, void* out, int out_dtype, void* workspace,
                                        size_t workspace_bytes, void* stream) {
    if (q_len < 1 || q_len > kvc::kMaxQueryTokens)
        return fail(KVC_ERR_UNSUPPORTED, "q_len %d outside [1, %d]", q_len, kvc::kMaxQueryTokens);
    std::vector<int32_t> ctx, table;
    kvc_status s = decode_validate(q, k_cache, v_cache, num_blocks, block_table, max_blocks, context_lens, B, Hq, Hkv,
                                   head_dim, block_size, max_context_len, out, out_dtype, 0, stream, ctx, table);
    if (s != KVC_OK || B == 0) return s;
    if (g_checked.load())
        for (int b = 0; b < B; ++b)
            if (ctx[b] < q_len)
                return fail(KVC_ERR_CAPACITY, "sequence %d: context length %d below q_len %d", b, ctx[b], q_len);
    kvc::DecodeArgs a = decode_args(q, nullptr, nullptr, k_cache, v_cache, num_blocks, block_table,
                                    max_blocks, context_lens, B, Hq, Hkv, head_dim, max_context_len, scale, out,
                                    out_dtype, workspace, workspace_bytes, 0);
    kvc::MultiPlan plan;
    cudaError_t e = kvc::multi_plan(B, Hq, Hkv, head_dim, max_context_len, q_len, &plan);
    if (e != cudaSuccess) return cuda_fail(e, "multi-token plan");
    s = check_workspace(plan.workspace_bytes, workspace, workspace_bytes);
    if (s != KVC_OK) return s;
    e = kvc::device_error_word(&a.err);
    if (e != cudaSuccess) return cuda_fail(e, "device error word");
    e = kvc::launch_multi(a, q_len, as_stream(stream));
    if (e != cudaSuccess) return cuda_fail(e, "paged_decode_multi_attention launch");
    return KVC_OK;
}

// ---- tree-drafted decoding ----------------------------------------------------
// whether `bytes_a` bytes from a and `bytes_b` from b share any
static bool overlap(const void* a, int64_t bytes_a, const void* b, int64_t bytes_b) {
    const uintptr_t x = reinterpret_cast<uintptr_t>(a), y = reinterpret_cast<uintptr_t>(b);
    return a && b && x < y + static_cast<uintptr_t>(bytes_b) && y < x + static_cast<uintptr_t>(bytes_a);
}
struct Span {
    const void* at;  // null: left out
    int64_t bytes;
};
// n rows of `row` elements of `size` bytes, `stride` elements apart
static Span rows_span(const void* at, int64_t n, int64_t stride, int64_t row, int64_t size) {
    const __int128 bytes = (static_cast<__int128>(n - 1) * stride + row) * size, most = __int128(1) << 56;
    return {at, static_cast<int64_t>(std::min(bytes, most))};
}
// whether each of some arrays of elements of `size` bytes starts at one (a misaligned load is a fault on the device)
static bool aligned_to(uintptr_t size, std::initializer_list<const void*> arrays) {
    for (const void* a : arrays)
        if (reinterpret_cast<uintptr_t>(a) % size) return false;
    return true;
}
// Outputs that share memory with an input or with each other: other CTAs may still read what one has written.
static kvc_status check_overlap(std::initializer_list<Span> out, std::initializer_list<Span> in) {
    for (const Span* o = out.begin(); o != out.end(); ++o) {
        for (const Span& i : in)
            if (overlap(o->at, o->bytes, i.at, i.bytes)) return fail(KVC_ERR_INVALID, "an output overlaps what the call reads");
        for (const Span* other = out.begin(); other != o; ++other)
            if (overlap(o->at, o->bytes, other->at, other->bytes)) return fail(KVC_ERR_INVALID, "an output overlaps another");
    }
    return KVC_OK;
}

kvc_status kv_tree_masks(const int32_t* parents, const int32_t* tree_lens, int B, int T, uint64_t* masks,
                         int32_t* depths) {
    if (B < 0 || T < 1) return fail(KVC_ERR_INVALID, "bad sizes");
    if (T > kvc::kMaxTreeNodes) return fail(KVC_ERR_UNSUPPORTED, "trees of %d nodes not supported (%d)", T, kvc::kMaxTreeNodes);
    if (B > 0 && (!parents || !masks)) return fail(KVC_ERR_INVALID, "null pointer");
    const int64_t nodes = static_cast<int64_t>(B) * T;
    kvc_status s = check_overlap({{masks, nodes * 8}, {depths, nodes * 4}}, {{parents, nodes * 4}, {tree_lens, B * int64_t(4)}});
    if (s != KVC_OK) return s;
    for (int b = 0; b < B; ++b) {  // everything is checked before anything is written
        const int len = tree_lens ? tree_lens[b] : T;
        if (len < 0 || len > T) return fail(KVC_ERR_INVALID, "sequence %d: tree length %d outside [0, %d]", b, len, T);
        for (int t = 1; t < len; ++t) {
            const int32_t par = parents[static_cast<size_t>(b) * T + t];
            if (par < 0 || par >= t) return fail(KVC_ERR_INVALID, "sequence %d: parent %d of node %d", b, par, t);
        }
    }
    for (int b = 0; b < B; ++b) {
        const size_t at = static_cast<size_t>(b) * T;
        const int len = tree_lens ? tree_lens[b] : T;
        for (int t = 0; t < T; ++t) {
            const bool in = t < len, child = in && t > 0;
            const size_t par = child ? at + parents[at + t] : at;
            masks[at + t] = in ? (uint64_t(1) << t) | (child ? masks[par] : 0) : 0;
            if (depths) depths[at + t] = child ? depths[par] + 1 : 0;
        }
    }
    return KVC_OK;
}

kvc_status kv_rope_turns(const double* inv_freq, int n, uint64_t* turns) {
    if (n < 0 || (n > 0 && (!inv_freq || !turns))) return fail(KVC_ERR_INVALID, "bad arguments");
    for (int i = 0; i < n; ++i)
        if (!(inv_freq[i] >= 0.0) || !std::isfinite(inv_freq[i]))
            return fail(KVC_ERR_INVALID, "frequency %d is negative or not finite", i);
    for (int i = 0; i < n; ++i) {
        // whole turns drop out; the fraction times 2^64 is below 2^64 (its double is at most 1 - 2^-53)
        double t = inv_freq[i] * 0.15915494309189535;  // 1 / (2 pi)
        t -= std::floor(t);
        turns[i] = static_cast<uint64_t>(std::nearbyint(std::ldexp(t, 64)));
    }
    return KVC_OK;
}

kvc_status kv_append_rope(const void* q, int64_t q_stride, const void* k, int64_t k_stride, const void* v,
                          int64_t v_stride, int n, int Hq, int Hkv, int head_dim, const void* q_weight,
                          const void* k_weight, float eps, const uint64_t* turns, int rot_dim, int interleaved,
                          const int32_t* positions, void* q_out, void* k_out, void* v_out, void* k_cache,
                          void* v_cache, int num_blocks, int block_size, const int64_t* slot_mapping, void* stream) {
    if (n < 0 || Hq < 1 || Hkv < 1) return fail(KVC_ERR_INVALID, "bad sizes");
    if (Hq > 65535 || Hkv > 65535) return fail(KVC_ERR_UNSUPPORTED, "Hq and Hkv must be <= 65535");
    if (head_dim != 64 && head_dim != 128) return fail(KVC_ERR_UNSUPPORTED, "head_dim %d not supported", head_dim);
    if (rot_dim < 0 || rot_dim > head_dim || rot_dim % 16)
        return fail(KVC_ERR_UNSUPPORTED, "rot_dim %d is not a multiple of 16 up to head_dim", rot_dim);
    if (interleaved != 0 && interleaved != 1) return fail(KVC_ERR_INVALID, "interleaved must be 0 or 1");
    if ((q_weight || k_weight) && !(eps >= 0.f && std::isfinite(eps)))
        return fail(KVC_ERR_INVALID, "eps must be finite and not negative");
    const bool cache = k_cache || v_cache || slot_mapping;
    if (cache && block_size != kvc::kBlockSize) return fail(KVC_ERR_UNSUPPORTED, "block_size %d not supported", block_size);
    if (n == 0) return KVC_OK;
    if (!q || !k || !v || !q_out) return fail(KVC_ERR_INVALID, "null pointer");
    if (rot_dim > 0 && (!turns || !positions)) return fail(KVC_ERR_INVALID, "rotation without turns or positions");
    if (cache && (!k_cache || !v_cache || !slot_mapping))
        return fail(KVC_ERR_INVALID, "k_cache, v_cache and slot_mapping: all or none");
    if (cache && num_blocks < 1) return fail(KVC_ERR_INVALID, "num_blocks must be positive");
    for (const void* ptr : {q, k, v, q_weight, k_weight, static_cast<const void*>(q_out), static_cast<const void*>(k_out),
                            static_cast<const void*>(v_out), static_cast<const void*>(k_cache),
                            static_cast<const void*>(v_cache)})
        if (!aligned16(ptr)) return fail(KVC_ERR_INVALID, "device buffers must be 16-byte aligned");
    if (!aligned_to(4, {rot_dim ? positions : nullptr}) || !aligned_to(8, {rot_dim ? turns : nullptr, slot_mapping}))
        return fail(KVC_ERR_INVALID, "positions, turns and slot_mapping must be aligned to their types");
    const int64_t qrow = static_cast<int64_t>(Hq) * head_dim, krow = static_cast<int64_t>(Hkv) * head_dim;
    if (q_stride % 8 || k_stride % 8 || v_stride % 8 || q_stride < qrow || k_stride < krow || v_stride < krow)
        return fail(KVC_ERR_INVALID, "token strides must be multiples of 8 elements and hold a token's heads");
    if ((q_out == q && q_stride != qrow) || (k_out == k && k_stride != krow) || (v_out == v && v_stride != krow))
        return fail(KVC_ERR_INVALID, "in place only where the rows are packed");
    {
        // in place: an output that is its own input's rows
        const int64_t cache_bytes = static_cast<int64_t>(num_blocks) * krow * block_size * 2;
        const Span q_in = rows_span(q, n, q_stride, qrow, 2), k_in = rows_span(k, n, k_stride, krow, 2),
                   v_in = rows_span(v, n, v_stride, krow, 2);
        const Span none = {nullptr, 0}, q_o = {q_out, n * qrow * 2}, k_o = {k_out, n * krow * 2}, v_o = {v_out, n * krow * 2};
        const Span kc = {k_cache, cache_bytes}, vc = {v_cache, cache_bytes};
        const Span qw = {q_weight, head_dim * 2}, kw = {k_weight, head_dim * 2};
        const Span tn = {rot_dim ? turns : nullptr, rot_dim * 4}, ps = {rot_dim ? positions : nullptr, n * int64_t(4)};
        const Span sl = {slot_mapping, n * int64_t(8)};
        for (const auto& [o, own, a, b] : {std::tuple(q_o, q_in, k_in, v_in), std::tuple(k_o, k_in, q_in, v_in),
                                           std::tuple(v_o, v_in, q_in, k_in)}) {
            kvc_status st = check_overlap({o}, {o.at == own.at ? none : own, a, b});
            if (st != KVC_OK) return st;
        }
        kvc_status st = check_overlap({kc, vc}, {q_in, k_in, v_in});
        if (st == KVC_OK) st = check_overlap({q_o, k_o, v_o, kc, vc}, {qw, kw, tn, ps, sl});
        if (st != KVC_OK) return st;
    }
    if (cache) {
        kvc_status st = checked([&]() -> kvc_status {
            std::vector<int64_t> sl;
            kvc_status e = copy_to_host(sl, slot_mapping, static_cast<size_t>(n), as_stream(stream));
            if (e != KVC_OK) return e;
            for (int t = 0; t < n; ++t)
                if (sl[t] >= static_cast<int64_t>(num_blocks) * block_size)
                    return fail(KVC_ERR_CAPACITY, "token %d: slot %lld beyond the pool", t, static_cast<long long>(sl[t]));
            return KVC_OK;
        });
        if (st != KVC_OK) return st;
    }
    kvc::RopeArgs a;
    a.q = static_cast<const __half*>(q);
    a.k = static_cast<const __half*>(k);
    a.v = static_cast<const __half*>(v);
    a.q_stride = q_stride;
    a.k_stride = k_stride;
    a.v_stride = v_stride;
    a.n = n;
    a.Hq = Hq;
    a.Hkv = Hkv;
    a.D = head_dim;
    a.q_weight = static_cast<const __half*>(q_weight);
    a.k_weight = static_cast<const __half*>(k_weight);
    a.eps = eps;
    a.turns = turns;
    a.rot_dim = rot_dim;
    a.interleaved = interleaved;
    a.positions = positions;
    a.q_out = static_cast<__half*>(q_out);
    a.k_out = static_cast<__half*>(k_out);
    a.v_out = static_cast<__half*>(v_out);
    a.k_cache = static_cast<__half*>(k_cache);
    a.v_cache = static_cast<__half*>(v_cache);
    a.num_blocks = num_blocks;
    a.slots = slot_mapping;
    cudaError_t e = kvc::device_error_word(&a.err);
    if (e != cudaSuccess) return cuda_fail(e, "device error word");
    e = kvc::launch_append_rope(a, as_stream(stream));
    if (e != cudaSuccess) return cuda_fail(e, "kv_append_rope launch");
    return KVC_OK;
}

static kvc_status check_tree_shape(int B, int Hq, int Hkv, int head_dim, int block_size, int max_context_len, int T) {
    kvc_status s = check_decode_shape(B, Hq, Hkv, head_dim, block_size, max_context_len);
    if (s != KVC_OK) return s;
    if (T < 1 || T > kvc::kMaxTreeNodes)
        return fail(KVC_ERR_UNSUPPORTED, "trees of %d nodes not supported (1..%d)", T, kvc::kMaxTreeNodes);
    if (max_context_len > kvc::kMaxTreeContext)  // key positions and tiles are 32-bit, with room behind the last one
        return fail(KVC_ERR_UNSUPPORTED, "max_context_len must be <= %d", kvc::kMaxTreeContext);
    return KVC_OK;
}

kvc_status paged_decode_tree_plan(int B, int Hq, int Hkv, int head_dim, int block_size, int max_context_len, int T,
                                  size_t* workspace_bytes) {
    kvc_status s = check_tree_shape(B, Hq, Hkv, head_dim, block_size, max_context_len, T);
    if (s != KVC_OK) return s;
    kvc::TreePlan plan;
    cudaError_t e = kvc::tree_plan(B, Hq, Hkv, head_dim, max_context_len, T, &plan);
    if (e != cudaSuccess) return cuda_fail(e, "tree plan");
    if (workspace_bytes) *workspace_bytes = plan.workspace_bytes;
    return KVC_OK;
}

kvc_status paged_decode_tree_attention(const void* q, const void* k_cache, const void* v_cache, int num_blocks,
                                       const int32_t* block_table, int max_blocks, const int32_t* context_lens,
                                       const uint64_t* masks, const int32_t* tree_lens, int T, int B, int Hq, int Hkv,
                                       int head_dim, int block_size, int max_context_len, float scale, void* out,
                                       int out_dtype, void* workspace, size_t workspace_bytes, void* stream) {
    kvc_status s = check_tree_shape(B, Hq, Hkv, head_dim, block_size, max_context_len, T);
    if (s != KVC_OK || B == 0) return s;
    if (!q || !k_cache || !v_cache || !block_table || !context_lens || !masks || !out)
        return fail(KVC_ERR_INVALID, "null pointer");
    if (!aligned16(q) || !aligned16(k_cache) || !aligned16(v_cache) || !aligned16(out))
        return fail(KVC_ERR_INVALID, "q, caches and out must be 16-byte aligned");
    if (!aligned_to(8, {masks})) return fail(KVC_ERR_INVALID, "masks must be 8-byte aligned");
    if (!aligned_to(4, {block_table, context_lens, tree_lens}))
        return fail(KVC_ERR_INVALID, "block_table, context_lens and tree_lens must be 4-byte aligned");
    if (num_blocks < 1 || max_blocks < 1) return fail(KVC_ERR_INVALID, "num_blocks and max_blocks must be positive");
    if (static_cast<int64_t>(num_blocks) * Hkv * block_size >= (int64_t(1) << 31))
        return fail(KVC_ERR_UNSUPPORTED, "num_blocks * Hkv * block_size must be < 2^31");
    if (static_cast<int64_t>(max_context_len) > static_cast<int64_t>(max_blocks) * block_size)
        return fail(KVC_ERR_CAPACITY, "max_context_len %d beyond max_blocks * block_size", max_context_len);
    if (out_dtype != KVC_F16 && out_dtype != KVC_F32) return fail(KVC_ERR_INVALID, "bad out_dtype");
    if (!std::isfinite(scale)) return fail(KVC_ERR_INVALID, "scale is not finite");
    const int64_t rows = static_cast<int64_t>(B) * T * Hq * head_dim;
    const int64_t cache = static_cast<int64_t>(num_blocks) * Hkv * block_size * head_dim * 2;
    const Span in[] = {{q, rows * 2}, {k_cache, cache}, {v_cache, cache}, {block_table, static_cast<int64_t>(B) * max_blocks * 4},
                       {context_lens, B * int64_t(4)}, {masks, static_cast<int64_t>(B) * T * 8}, {tree_lens, B * int64_t(4)}};
    const Span out_span = {out, rows * (out_dtype == KVC_F32 ? 4 : 2)};
    s = check_overlap({out_span}, {in[0], in[1], in[2], in[3], in[4], in[5], in[6]});
    if (s != KVC_OK) return s;
    s = checked([&]() -> kvc_status {
        std::vector<int32_t> ctx, tree, table;
        kvc_status e = copy_to_host(ctx, context_lens, static_cast<size_t>(B), as_stream(stream));
        if (e == KVC_OK && tree_lens) e = copy_to_host(tree, tree_lens, static_cast<size_t>(B), as_stream(stream));
        if (e == KVC_OK) e = copy_to_host(table, block_table, static_cast<size_t>(B) * max_blocks, as_stream(stream));
        if (e != KVC_OK) return e;
        for (int b = 0; b < B; ++b) {
            const int32_t len = tree_lens ? tree[b] : T;
            if (len < 0 || len > T) return fail(KVC_ERR_INVALID, "sequence %d: tree length %d outside [0, %d]", b, len, T);
            if (ctx[b] < len || ctx[b] > max_context_len)
                return fail(KVC_ERR_CAPACITY, "sequence %d: context length %d outside [%d, %d]", b, ctx[b], len, max_context_len);
            for (int j = 0; j < (ctx[b] + block_size - 1) / block_size; ++j) {
                const int32_t blk = table[static_cast<size_t>(b) * max_blocks + j];
                if (blk < 0 || blk >= num_blocks)
                    return fail(KVC_ERR_INVALID, "sequence %d: block-table entry %d = %d outside [0, %d)", b, j, blk, num_blocks);
            }
        }
        return KVC_OK;
    });
    if (s != KVC_OK) return s;
    kvc::TreePlan plan;
    cudaError_t e = kvc::tree_plan(B, Hq, Hkv, head_dim, max_context_len, T, &plan);
    if (e != cudaSuccess) return cuda_fail(e, "tree plan");
    s = check_workspace(plan.workspace_bytes, workspace, workspace_bytes);
    if (s == KVC_OK && plan.workspace_bytes)
        s = check_overlap({{workspace, static_cast<int64_t>(plan.workspace_bytes)}},
                          {out_span, in[0], in[1], in[2], in[3], in[4], in[5], in[6]});
    if (s != KVC_OK) return s;
    kvc::TreeArgs a;
    a.q = static_cast<const __half*>(q);
    a.k_cache = static_cast<const __half*>(k_cache);
    a.v_cache = static_cast<const __half*>(v_cache);
    a.num_blocks = num_blocks;
    a.block_table = block_table;
    a.max_blocks = max_blocks;
    a.context_lens = context_lens;
    a.masks = masks;
    a.tree_lens = tree_lens;
    a.T = T;
    a.B = B;
    a.Hq = Hq;
    a.Hkv = Hkv;
    a.D = head_dim;
    a.max_context_len = max_context_len;
    a.scale = scale;
    a.out = out;
    a.out_f32 = out_dtype == KVC_F32;
    a.workspace = workspace;
    a.workspace_bytes = workspace_bytes;
    e = kvc::device_error_word(&a.err);
    if (e != cudaSuccess) return cuda_fail(e, "device error word");
    e = kvc::launch_tree(a, as_stream(stream));
    if (e != cudaSuccess) return cuda_fail(e, "paged_decode_tree_attention launch");
    return KVC_OK;
}

kvc_status draft_tree_verify(const void* target_probs, int64_t p_stride, const void* draft_probs, int64_t q_stride,
                             int prob_dtype, const int32_t* tokens, const int32_t* parents, const int32_t* tree_lens,
                             const float* uniforms, int B, int T, int V, int distinct, int32_t* path,
                             int32_t* path_len, int32_t* next_token, void* stream) {
    if (B < 0 || V < 1) return fail(KVC_ERR_INVALID, "bad sizes");
    if (T < 1 || T > kvc::kMaxTreeNodes)
        return fail(KVC_ERR_UNSUPPORTED, "trees of %d nodes not supported (1..%d)", T, kvc::kMaxTreeNodes);
    if (B > 65535 || V > (1 << 24)) return fail(KVC_ERR_UNSUPPORTED, "B must be <= 65535 and V <= 2^24");
    if (prob_dtype != KVC_F16 && prob_dtype != KVC_F32) return fail(KVC_ERR_INVALID, "bad prob_dtype");
    if (distinct != 0 && distinct != 1) return fail(KVC_ERR_INVALID, "distinct must be 0 or 1");
    if (p_stride < V || q_stride < V) return fail(KVC_ERR_INVALID, "row strides must be at least V");
    if (B == 0) return KVC_OK;
    if (!target_probs || !draft_probs || !tokens || !parents || !uniforms || !path || !path_len || !next_token)
        return fail(KVC_ERR_INVALID, "null pointer");
    const uintptr_t size = prob_dtype == KVC_F32 ? 4 : 2;
    if (!aligned_to(size, {target_probs, draft_probs}))
        return fail(KVC_ERR_INVALID, "probabilities must be aligned to their type");
    if (!aligned_to(4, {tokens, parents, tree_lens, uniforms, path, path_len, next_token}))
        return fail(KVC_ERR_INVALID, "the tree's arrays must be 4-byte aligned");
    const int64_t nodes_bytes = static_cast<int64_t>(B) * T * 4, per = B * int64_t(4);
    kvc_status s = check_overlap({{path, nodes_bytes}, {path_len, per}, {next_token, per}},
                                 {rows_span(target_probs, static_cast<int64_t>(B) * T, p_stride, V, size),
                                  rows_span(draft_probs, static_cast<int64_t>(B) * T, q_stride, V, size),
                                  {tokens, nodes_bytes}, {parents, nodes_bytes}, {uniforms, nodes_bytes}, {tree_lens, per}});
    if (s != KVC_OK) return s;
    s = checked([&]() -> kvc_status {
        std::vector<int32_t> tok, par, len;
        const size_t n = static_cast<size_t>(B) * T;
        kvc_status e = copy_to_host(tok, tokens, n, as_stream(stream));
        if (e == KVC_OK) e = copy_to_host(par, parents, n, as_stream(stream));
        if (e == KVC_OK && tree_lens) e = copy_to_host(len, tree_lens, static_cast<size_t>(B), as_stream(stream));
        if (e != KVC_OK) return e;
        for (int b = 0; b < B; ++b) {
            const int32_t nodes = tree_lens ? len[b] : T;
            if (nodes < 0 || nodes > T) return fail(KVC_ERR_INVALID, "sequence %d: tree length %d outside [0, %d]", b, nodes, T);
            for (int t = 1; t < nodes; ++t) {
                const size_t at = static_cast<size_t>(b) * T + t;
                if (par[at] < 0 || par[at] >= t) return fail(KVC_ERR_INVALID, "sequence %d: parent %d of node %d", b, par[at], t);
                if (tok[at] < 0 || tok[at] >= V) return fail(KVC_ERR_INVALID, "sequence %d: token %d of node %d", b, tok[at], t);
            }
        }
        return KVC_OK;
    });
    if (s != KVC_OK) return s;
    kvc::VerifyArgs a;
    a.p = target_probs;
    a.q = draft_probs;
    a.p_stride = p_stride;
    a.q_stride = q_stride;
    a.probs_f32 = prob_dtype == KVC_F32;
    a.tokens = tokens;
    a.parents = parents;
    a.tree_lens = tree_lens;
    a.uniforms = uniforms;
    a.B = B;
    a.T = T;
    a.V = V;
    a.distinct = distinct;
    a.path = path;
    a.path_len = path_len;
    a.next_token = next_token;
    cudaError_t e = kvc::device_error_word(&a.err);
    if (e != cudaSuccess) return cuda_fail(e, "device error word");
    e = kvc::launch_tree_verify(a, as_stream(stream));
    if (e != cudaSuccess) return cuda_fail(e, "draft_tree_verify launch");
    return KVC_OK;
}

kvc_status kv_tree_commit(kvc_handle h, const int32_t* block_table, int max_blocks, const int32_t* context_lens,
                          const int32_t* tree_lens, const int32_t* path, const int32_t* path_len, int P, int B,
                          int32_t* new_context_lens, void* stream) {
    if (!h) return fail(KVC_ERR_INVALID, "null handle");
    if (!h->k_pool) return fail(KVC_ERR_INVALID, "host-only cache has no device pools");
    if (B < 0 || max_blocks < 1) return fail(KVC_ERR_INVALID, "bad sizes");
    if (P < 1 || P > kvc::kMaxTreeNodes)
        return fail(KVC_ERR_UNSUPPORTED, "paths of %d nodes not supported (1..%d)", P, kvc::kMaxTreeNodes);
    if (B > 65535) return fail(KVC_ERR_UNSUPPORTED, "B must be <= 65535");
    if (B == 0) return KVC_OK;
    if (!block_table || !context_lens || !path || !path_len || !new_context_lens) return fail(KVC_ERR_INVALID, "null pointer");
    if (!aligned_to(4, {block_table, context_lens, tree_lens, path, path_len, new_context_lens}))
        return fail(KVC_ERR_INVALID, "the arrays must be 4-byte aligned");
    const int64_t per = static_cast<int64_t>(B) * 4;
    const int64_t layer = static_cast<int64_t>(h->cfg.num_blocks) * h->cfg.num_kv_heads * h->cfg.block_size * h->cfg.head_dim;
    kvc_status s = check_overlap({{new_context_lens, per}, rows_span(h->k_pool, h->cfg.num_layers, layer, layer, 2),
                                  rows_span(h->v_pool, h->cfg.num_layers, layer, layer, 2)},
                                 {{context_lens, per}, {tree_lens, per}, {path_len, per}, {path, per * P},
                                  {block_table, per * max_blocks}});
    if (s != KVC_OK) return s;
    s = checked([&]() -> kvc_status {
        std::vector<int32_t> ctx, tree, nodes, len, table;
        kvc_status e = copy_to_host(ctx, context_lens, static_cast<size_t>(B), as_stream(stream));
        if (e == KVC_OK && tree_lens) e = copy_to_host(tree, tree_lens, static_cast<size_t>(B), as_stream(stream));
        if (e == KVC_OK) e = copy_to_host(nodes, path, static_cast<size_t>(B) * P, as_stream(stream));
        if (e == KVC_OK) e = copy_to_host(len, path_len, static_cast<size_t>(B), as_stream(stream));
        if (e == KVC_OK) e = copy_to_host(table, block_table, static_cast<size_t>(B) * max_blocks, as_stream(stream));
        if (e != KVC_OK) return e;
        for (int b = 0; b < B; ++b) {
            const int32_t size = tree_lens ? tree[b] : P;
            if (size < 0 || size > kvc::kMaxTreeNodes || ctx[b] < size ||
                ctx[b] > static_cast<int64_t>(max_blocks) * kvc::kBlockSize)
                return fail(KVC_ERR_CAPACITY, "sequence %d: context %d with a tree of %d", b, ctx[b], size);
            if (len[b] < 0 || len[b] > P || len[b] > size)
                return fail(KVC_ERR_INVALID, "sequence %d: path length %d", b, len[b]);
            int32_t last = -1;
            for (int i = 0; i < len[b]; ++i) {
                const int32_t node = nodes[static_cast<size_t>(b) * P + i];
                if (node <= last || node >= size || (i == 0 && node != 0))
                    return fail(KVC_ERR_INVALID, "sequence %d: node %d at place %d of its path", b, node, i);
                last = node;
                if (node == i) continue;
                const int32_t base = ctx[b] - size;
                for (const int32_t pos : {base + i, base + node}) {
                    const int32_t blk = table[static_cast<size_t>(b) * max_blocks + pos / kvc::kBlockSize];
                    if (blk < 0 || blk >= h->cfg.num_blocks)
                        return fail(KVC_ERR_INVALID, "sequence %d: block %d of position %d", b, blk, pos);
                }
            }
        }
        return KVC_OK;
    });
    if (s != KVC_OK) return s;
    kvc::CommitArgs a;
    a.k_pool = static_cast<__half*>(h->k_pool);
    a.v_pool = static_cast<__half*>(h->v_pool);
    a.L = h->cfg.num_layers;
    a.num_blocks = h->cfg.num_blocks;
    a.Hkv = h->cfg.num_kv_heads;
    a.D = h->cfg.head_dim;
    a.block_table = block_table;
    a.max_blocks = max_blocks;
    a.context_lens = context_lens;
    a.tree_lens = tree_lens;
    a.path = path;
    a.path_len = path_len;
    a.P = P;
    a.B = B;
    a.new_context_lens = new_context_lens;
    cudaError_t e = kvc::device_error_word(&a.err);
    if (e != cudaSuccess) return cuda_fail(e, "device error word");
    e = kvc::launch_tree_commit(a, as_stream(stream));
    if (e != cudaSuccess) return cuda_fail(e, "kv_tree_commit launch");
    return KVC_OK;
}

// ---- windows, the block-scaled cache, tables built on the GPU ------------------
static kvc_status check_window(int window, int sinks, int least) {
    if (window < least || sinks < 0) return fail(KVC_ERR_INVALID, "window must be at least %d and sinks not negative", least);
    if (window == 0 && sinks != 0) return fail(KVC_ERR_INVALID, "sinks without a window");
    if (window > kvc::kMaxWindow || sinks > kvc::kMaxWindow)
        return fail(KVC_ERR_UNSUPPORTED, "window and sinks must be <= %d", kvc::kMaxWindow);
    return KVC_OK;
}

kvc_status kv_block_tables(const int32_t* lens_before, const int32_t* lens_after, int B, const int32_t* free_blocks,
                           int num_free, const int32_t* placed, int window, int sinks, int32_t* block_table,
                           int max_blocks, int block_size, int32_t* new_placed, int32_t* cu_tokens,
                           int64_t* slot_mapping, int32_t* positions, int num_slots, void* stream) {
    if (B < 0 || num_free < 0 || num_slots < 0 || max_blocks < 1) return fail(KVC_ERR_INVALID, "bad sizes");
    if (B > 65535) return fail(KVC_ERR_UNSUPPORTED, "B must be <= 65535");
    if (block_size != kvc::kBlockSize) return fail(KVC_ERR_UNSUPPORTED, "block_size %d not supported", block_size);
    if (max_blocks > kvc::kMaxTableBlocks) return fail(KVC_ERR_UNSUPPORTED, "max_blocks * block_size must be < 2^31");
    kvc_status s = check_window(window, sinks, 0);
    if (s != KVC_OK) return s;
    if (!placed || !new_placed || !cu_tokens || (B > 0 && (!lens_after || !block_table)) ||
        (num_free > 0 && !free_blocks) || (num_slots > 0 && !slot_mapping))
        return fail(KVC_ERR_INVALID, "null pointer");
    if (!aligned_to(4, {lens_before, lens_after, free_blocks, placed, block_table, new_placed, cu_tokens, positions}) ||
        !aligned_to(8, {slot_mapping}))
        return fail(KVC_ERR_INVALID, "the arrays must be aligned to their types");
    const int64_t per = static_cast<int64_t>(B) * 4;
    s = check_overlap({{block_table, per * max_blocks}, {new_placed, 4}, {cu_tokens, per + 4},
                       {slot_mapping, num_slots * int64_t(8)}, {positions, num_slots * int64_t(4)}},
                      {{lens_before, per}, {lens_after, per}, {free_blocks, num_free * int64_t(4)}, {placed, 4}});
    if (s != KVC_OK) return s;
    s = checked([&]() -> kvc_status {
        std::vector<int32_t> before, after, used;
        kvc_status e = copy_to_host(after, lens_after, static_cast<size_t>(B), as_stream(stream));
        if (e == KVC_OK && lens_before) e = copy_to_host(before, lens_before, static_cast<size_t>(B), as_stream(stream));
        if (e == KVC_OK) e = copy_to_host(used, placed, 1, as_stream(stream));
        if (e != KVC_OK) return e;
        if (used[0] < 0 || used[0] > num_free)
            return fail(KVC_ERR_INVALID, "%d of the %d blocks are placed", used[0], num_free);
        int64_t need = 0, tokens = 0;
        const int64_t most = window > 0 ? (sinks + block_size - 1) / block_size + (window + 2 * block_size - 2) / block_size
                                        : max_blocks;
        for (int b = 0; b < B; ++b) {
            const int64_t from = lens_before ? before[b] : 0, to = after[b];
            if (from < 0 || to < from) return fail(KVC_ERR_INVALID, "sequence %d: lengths %lld and %lld", b,
                                                   static_cast<long long>(from), static_cast<long long>(to));
            if (to > static_cast<int64_t>(max_blocks) * block_size)
                return fail(KVC_ERR_CAPACITY, "sequence %d: length %lld beyond the table", b, static_cast<long long>(to));
            need += std::min<int64_t>((to + block_size - 1) / block_size, most) -
                    std::min<int64_t>((from + block_size - 1) / block_size, most);
            tokens += to - from;
        }
        if (need > num_free - used[0])
            return fail(KVC_ERR_OOM, "the step needs %lld blocks, %d are left", static_cast<long long>(need), num_free - used[0]);
        if (tokens > num_slots)
            return fail(KVC_ERR_CAPACITY, "the step has %lld tokens, there is room for %d", static_cast<long long>(tokens), num_slots);
        return KVC_OK;
    });
    if (s != KVC_OK) return s;
    kvc::BlockTableArgs a;
    a.lens_before = lens_before;
    a.lens_after = lens_after;
    a.free_blocks = free_blocks;
    a.placed = placed;
    a.B = B;
    a.num_free = num_free;
    a.window = window;
    a.sinks = sinks;
    a.block_table = block_table;
    a.max_blocks = max_blocks;
    a.new_placed = new_placed;
    a.cu_tokens = cu_tokens;
    a.slots = slot_mapping;
    a.positions = positions;
    a.num_slots = num_slots;
    cudaError_t e = kvc::device_error_word(&a.err);
    if (e != cudaSuccess) return cuda_fail(e, "device error word");
    e = kvc::launch_block_tables(a, as_stream(stream));
    if (e != cudaSuccess) return cuda_fail(e, "kv_block_tables launch");
    return KVC_OK;
}

// The block-scaled cache's own limits.
static kvc_status check_block_codes(const void* codes, const float* scales, int num_blocks, int Hkv, int block_size) {
    if (num_blocks < 1) return fail(KVC_ERR_INVALID, "num_blocks must be positive");
    if (!codes || !scales) return fail(KVC_ERR_INVALID, "null pointer");
    if (!aligned16(codes) || !aligned16(scales)) return fail(KVC_ERR_INVALID, "codes and scales must be 16-byte aligned");
    if (static_cast<int64_t>(num_blocks) * Hkv * block_size >= (int64_t(1) << 30))
        return fail(KVC_ERR_UNSUPPORTED, "num_blocks * Hkv * block_size must be < 2^30");
    return KVC_OK;
}

kvc_status kv_append_fp8_block(const void* k_new, int64_t k_stride, const void* v_new, int64_t v_stride, int n,
                               const int64_t* slot_mapping, void* codes, float* scales, int num_blocks, int Hkv,
                               int head_dim, int block_size, void* stream) {
    if (n < 0 || Hkv < 1) return fail(KVC_ERR_INVALID, "bad sizes");
    if (Hkv > 65535) return fail(KVC_ERR_UNSUPPORTED, "Hkv must be <= 65535");
    if (head_dim != 64 && head_dim != 128) return fail(KVC_ERR_UNSUPPORTED, "head_dim %d not supported", head_dim);
    if (block_size != kvc::kBlockSize) return fail(KVC_ERR_UNSUPPORTED, "block_size %d not supported", block_size);
    if (n == 0) return KVC_OK;
    if (!k_new || !v_new || !slot_mapping) return fail(KVC_ERR_INVALID, "null pointer");
    kvc_status s = check_block_codes(codes, scales, num_blocks, Hkv, block_size);
    if (s != KVC_OK) return s;
    if (!aligned16(k_new) || !aligned16(v_new)) return fail(KVC_ERR_INVALID, "k_new and v_new must be 16-byte aligned");
    if (!aligned_to(8, {slot_mapping})) return fail(KVC_ERR_INVALID, "slot_mapping must be 8-byte aligned");
    const int64_t row = static_cast<int64_t>(Hkv) * head_dim, tiles = static_cast<int64_t>(num_blocks) * Hkv * 2;
    if (k_stride % 8 || v_stride % 8 || k_stride < row || v_stride < row)
        return fail(KVC_ERR_INVALID, "token strides must be multiples of 8 elements and hold a token's heads");
    s = check_overlap({{codes, tiles * block_size * head_dim}, {scales, tiles * 4}},
                      {rows_span(k_new, n, k_stride, row, 2), rows_span(v_new, n, v_stride, row, 2),
                       {slot_mapping, n * int64_t(8)}});
    if (s != KVC_OK) return s;
    s = checked([&]() -> kvc_status {
        std::vector<int64_t> sl;
        kvc_status e = copy_to_host(sl, slot_mapping, static_cast<size_t>(n), as_stream(stream));
        if (e != KVC_OK) return e;
        std::unordered_map<int64_t, int> seen;  // block -> its last token
        for (int t = 0; t < n; ++t) {
            if (sl[t] < 0) continue;
            if (sl[t] >= static_cast<int64_t>(num_blocks) * block_size)
                return fail(KVC_ERR_CAPACITY, "token %d: slot %lld beyond the cache", t, static_cast<long long>(sl[t]));
            const auto [at, fresh] = seen.try_emplace(sl[t] / block_size, t);
            if (!fresh && (at->second != t - 1 || sl[t - 1] + 1 != sl[t]))
                return fail(KVC_ERR_INVALID, "token %d: its block's tokens are not consecutive", t);
            at->second = t;
        }
        return KVC_OK;
    });
    if (s != KVC_OK) return s;
    kvc::AppendFp8BlockArgs a;
    a.k = static_cast<const __half*>(k_new);
    a.v = static_cast<const __half*>(v_new);
    a.k_stride = k_stride;
    a.v_stride = v_stride;
    a.slots = slot_mapping;
    a.n = n;
    a.codes = static_cast<uint8_t*>(codes);
    a.scales = scales;
    a.num_blocks = num_blocks;
    a.Hkv = Hkv;
    a.D = head_dim;
    cudaError_t e = kvc::device_error_word(&a.err);
    if (e != cudaSuccess) return cuda_fail(e, "device error word");
    e = kvc::launch_append_fp8_block(a, as_stream(stream));
    if (e != cudaSuccess) return cuda_fail(e, "kv_append_fp8_block launch");
    return KVC_OK;
}

static kvc_status window_plan(int B, int Hq, int Hkv, int head_dim, int block_size, int max_context_len, int window,
                              int sinks, bool block8, size_t* workspace_bytes) {
    kvc_status s = check_decode_shape(B, Hq, Hkv, head_dim, block_size, max_context_len);
    if (s == KVC_OK) s = check_window(window, sinks, block8 ? 0 : 1);
    if (s != KVC_OK) return s;
    kvc::DecodePlan plan;
    cudaError_t e = kvc::decode_window_plan(B, Hq, Hkv, head_dim, max_context_len, window, sinks, block8, &plan);
    if (e != cudaSuccess) return cuda_fail(e, "decode plan");
    if (workspace_bytes) *workspace_bytes = plan.workspace_bytes;
    return KVC_OK;
}

kvc_status paged_decode_window_plan(int B, int Hq, int Hkv, int head_dim, int block_size, int max_context_len,
                                    int window, int sinks, size_t* workspace_bytes) {
    return window_plan(B, Hq, Hkv, head_dim, block_size, max_context_len, window, sinks, false, workspace_bytes);
}

kvc_status paged_decode_fp8_block_plan(int B, int Hq, int Hkv, int head_dim, int block_size, int max_context_len,
                                       int window, int sinks, size_t* workspace_bytes) {
    return window_plan(B, Hq, Hkv, head_dim, block_size, max_context_len, window, sinks, true, workspace_bytes);
}

// The two decode calls behind their own arguments' checks; a holds everything but the workspace and the error word.
static kvc_status decode_window(kvc::DecodeArgs& a, std::initializer_list<Span> caches, int out_dtype, void* workspace,
                                size_t workspace_bytes, const char* name, void* stream) {
    if (!a.q || !a.block_table || !a.context_lens || !a.out) return fail(KVC_ERR_INVALID, "null pointer");
    if (!aligned16(a.q) || !aligned16(a.out)) return fail(KVC_ERR_INVALID, "q and out must be 16-byte aligned");
    if (!aligned_to(4, {a.block_table, a.context_lens}))
        return fail(KVC_ERR_INVALID, "block_table and context_lens must be 4-byte aligned");
    if (a.max_blocks < 1) return fail(KVC_ERR_INVALID, "max_blocks must be positive");
    if (a.max_blocks > kvc::kMaxTableBlocks) return fail(KVC_ERR_UNSUPPORTED, "max_blocks * block_size must be < 2^31");
    if (a.max_context_len > a.max_blocks * kvc::kBlockSize)
        return fail(KVC_ERR_CAPACITY, "max_context_len %d beyond max_blocks * block_size", a.max_context_len);
    if (out_dtype != KVC_F16 && out_dtype != KVC_F32) return fail(KVC_ERR_INVALID, "bad out_dtype");
    if (!std::isfinite(a.scale)) return fail(KVC_ERR_INVALID, "scale is not finite");
    const int64_t rows = static_cast<int64_t>(a.B) * a.Hq * a.D, per = a.B * int64_t(4);
    const int64_t new_rows = static_cast<int64_t>(a.B) * a.Hkv * a.D * 2;
    const Span q = {a.q, rows * 2}, table = {a.block_table, per * a.max_blocks}, lens = {a.context_lens, per},
               kn = {a.k_new, new_rows}, vn = {a.v_new, new_rows}, out = {a.out, rows * (out_dtype == KVC_F32 ? 4 : 2)};
    kvc_status s = check_overlap({out}, caches);
    if (s == KVC_OK) s = check_overlap({out}, {q, table, lens, kn, vn});
    if (s == KVC_OK && a.k_new) {  // the caches are written too
        const Span k = *caches.begin(), v = *(caches.begin() + 1);
        s = check_overlap({k, v}, {q, table, lens, kn, vn});
    }
    if (s != KVC_OK) return s;
    s = checked([&]() -> kvc_status {
        std::vector<int32_t> ctx, entries;
        kvc_status e = copy_to_host(ctx, a.context_lens, static_cast<size_t>(a.B), as_stream(stream));
        if (e == KVC_OK) e = copy_to_host(entries, a.block_table, static_cast<size_t>(a.B) * a.max_blocks, as_stream(stream));
        if (e != KVC_OK) return e;
        for (int b = 0; b < a.B; ++b) {
            if (ctx[b] < 1 || ctx[b] > a.max_context_len)
                return fail(KVC_ERR_CAPACITY, "sequence %d: context length %d outside [1, %d]", b, ctx[b], a.max_context_len);
            const kvc::Visible v = kvc::visible_blocks(ctx[b], a.window, a.sinks);
            for (int i = 0; i < v.nblk; ++i) {
                const int j = i < v.ns ? i : i - v.ns + v.w0;
                const int32_t blk = entries[static_cast<size_t>(b) * a.max_blocks + j];
                if (blk < 0 || blk >= a.num_blocks)
                    return fail(KVC_ERR_INVALID, "sequence %d: block-table entry %d = %d outside [0, %d)", b, j, blk, a.num_blocks);
            }
        }
        return KVC_OK;
    });
    if (s != KVC_OK) return s;
    kvc::DecodePlan plan;
    cudaError_t e = kvc::decode_window_plan(a.B, a.Hq, a.Hkv, a.D, a.max_context_len, a.window, a.sinks,
                                            a.codes != nullptr, &plan);
    if (e != cudaSuccess) return cuda_fail(e, "decode plan");
    s = check_workspace(plan.workspace_bytes, workspace, workspace_bytes);
    if (s == KVC_OK && plan.workspace_bytes) {
        const Span ws = {workspace, static_cast<int64_t>(plan.workspace_bytes)};
        s = check_overlap({ws}, caches);
        if (s == KVC_OK) s = check_overlap({ws}, {out, q, table, lens, kn, vn});
    }
    if (s != KVC_OK) return s;
    a.out_f32 = out_dtype == KVC_F32;
    a.workspace = workspace;
    a.workspace_bytes = workspace_bytes;
    a.blocks_per_split = 0;
    e = kvc::device_error_word(&a.err);
    if (e != cudaSuccess) return cuda_fail(e, "device error word");
    e = kvc::launch_decode_window(a, plan, as_stream(stream));
    if (e != cudaSuccess) return cuda_fail(e, name);
    return KVC_OK;
}

kvc_status paged_decode_window_attention(const void* q, const void* k_new, const void* v_new, void* k_cache,
                                         void* v_cache, int num_blocks, const int32_t* block_table, int max_blocks,
                                         const int32_t* context_lens, int window, int sinks, int B, int Hq, int Hkv,
                                         int head_dim, int block_size, int max_context_len, float scale, void* out,
                                         int out_dtype, void* workspace, size_t workspace_bytes, void* stream) {
    kvc_status s = check_decode_shape(B, Hq, Hkv, head_dim, block_size, max_context_len);
    if (s == KVC_OK) s = check_window(window, sinks, 1);
    if (s != KVC_OK || B == 0) return s;
    if (!k_cache || !v_cache) return fail(KVC_ERR_INVALID, "null pointer");
    if ((k_new == nullptr) != (v_new == nullptr)) return fail(KVC_ERR_INVALID, "k_new and v_new: both or neither");
    if (!aligned16(k_cache) || !aligned16(v_cache) || !aligned16(k_new) || !aligned16(v_new))
        return fail(KVC_ERR_INVALID, "caches, k_new and v_new must be 16-byte aligned");
    if (num_blocks < 1) return fail(KVC_ERR_INVALID, "num_blocks must be positive");
    if (static_cast<int64_t>(num_blocks) * Hkv * block_size >= (int64_t(1) << 31))
        return fail(KVC_ERR_UNSUPPORTED, "num_blocks * Hkv * block_size must be < 2^31");
    kvc::DecodeArgs a = decode_args(q, k_new, v_new, k_cache, v_cache, num_blocks, block_table, max_blocks, context_lens,
                                    B, Hq, Hkv, head_dim, max_context_len, scale, out, out_dtype, nullptr, 0, 0);
    a.window = window;
    a.sinks = sinks;
    const int64_t cache = static_cast<int64_t>(num_blocks) * Hkv * block_size * head_dim * 2;
    return decode_window(a, {{k_cache, cache}, {v_cache, cache}}, out_dtype, workspace, workspace_bytes,
                         "paged_decode_window_attention launch", stream);
}

kvc_status paged_decode_attention_fp8_block(const void* q, const void* codes, const float* scales, int num_blocks,
                                            const int32_t* block_table, int max_blocks, const int32_t* context_lens,
                                            int window, int sinks, int B, int Hq, int Hkv, int head_dim,
                                            int block_size, int max_context_len, float scale, void* out, int out_dtype,
                                            void* workspace, size_t workspace_bytes, void* stream) {
    kvc_status s = check_decode_shape(B, Hq, Hkv, head_dim, block_size, max_context_len);
    if (s == KVC_OK) s = check_window(window, sinks, 0);
    if (s != KVC_OK || B == 0) return s;
    s = check_block_codes(codes, scales, num_blocks, Hkv, block_size);
    if (s != KVC_OK) return s;
    kvc::DecodeArgs a = decode_args(q, nullptr, nullptr, nullptr, nullptr, num_blocks, block_table, max_blocks,
                                    context_lens, B, Hq, Hkv, head_dim, max_context_len, scale, out, out_dtype, nullptr,
                                    0, 0);
    a.codes = static_cast<const uint8_t*>(codes);
    a.scales = scales;
    a.window = window;
    a.sinks = sinks;
    const int64_t tiles = static_cast<int64_t>(num_blocks) * Hkv * 2;
    return decode_window(a, {{codes, tiles * block_size * head_dim}, {scales, tiles * 4}}, out_dtype, workspace,
                         workspace_bytes, "paged_decode_attention_fp8_block launch", stream);
}

kvc_status kvc_call(int which, const void* words, int count, void* stream) {
    if (!words) return fail(KVC_ERR_INVALID, "null pointer");
    switch (which) {
        case KVC_CALL_APPEND_ROPE: return call_with_words(kv_append_rope, words, count, stream);
        case KVC_CALL_TREE_ATTENTION: return call_with_words(paged_decode_tree_attention, words, count, stream);
        case KVC_CALL_TREE_VERIFY: return call_with_words(draft_tree_verify, words, count, stream);
        case KVC_CALL_TREE_COMMIT: return call_with_words(kv_tree_commit, words, count, stream);
        case KVC_CALL_BLOCK_TABLES: return call_with_words(kv_block_tables, words, count, stream);
        case KVC_CALL_APPEND_FP8_BLOCK: return call_with_words(kv_append_fp8_block, words, count, stream);
        case KVC_CALL_ATTENTION_FP8_BLOCK: return call_with_words(paged_decode_attention_fp8_block, words, count, stream);
        case KVC_CALL_WINDOW_ATTENTION: return call_with_words(paged_decode_window_attention, words, count, stream);
        case KVC_CALL_PREFILL_WINDOW: return call_with_words(prefill_window_attention, words, count, stream);
        default: return fail(KVC_ERR_INVALID, "unknown call %d", which);
    }
}

// (window 0: none)
static kvc_status prefill_common(const void* q, const void* k, const void* v, const int32_t* cu_seqlens, int nseq,
                                 int total_tokens, int max_seqlen, int Hq, int Hkv, int head_dim, float scale,
                                 int causal, int window, int sinks, int p_precision, void* out, int out_dtype,
                                 const char* name, void* stream) {
    if (p_precision != KVC_PREFILL_P_F16 && p_precision != KVC_PREFILL_P_SPLIT)
        return fail(KVC_ERR_INVALID, "bad p_precision %d", p_precision);
    if (nseq < 0 || total_tokens < 0 || max_seqlen < 0 || Hq < 1 || Hkv < 1) return fail(KVC_ERR_INVALID, "bad sizes");
    if (Hq % Hkv) return fail(KVC_ERR_INVALID, "Hq (%d) must be a multiple of Hkv (%d)", Hq, Hkv);
    if (head_dim != 64 && head_dim != 128) return fail(KVC_ERR_UNSUPPORTED, "head_dim %d not supported", head_dim);
    if (out_dtype != KVC_F16 && out_dtype != KVC_F32) return fail(KVC_ERR_INVALID, "bad out_dtype");
    if (nseq == 0 || total_tokens == 0) return KVC_OK;
    if (!q || !k || !v || !cu_seqlens || !out) return fail(KVC_ERR_INVALID, "null pointer");
    if (!aligned16(q) || !aligned16(k) || !aligned16(v) || !aligned16(out))
        return fail(KVC_ERR_INVALID, "q, k, v and out must be 16-byte aligned");
    if (static_cast<int64_t>(nseq) * ((max_seqlen + 127) / 128) * Hq > 2147483647LL)
        return fail(KVC_ERR_UNSUPPORTED, "grid too large");
    if (g_checked.load()) {
        std::vector<int32_t> cu;
        kvc_status st = copy_to_host(cu, cu_seqlens, static_cast<size_t>(nseq) + 1, as_stream(stream));
        if (st != KVC_OK) return st;
        if (cu[0] != 0 || cu[nseq] != total_tokens) return fail(KVC_ERR_INVALID, "cu_seqlens must run from 0 to total_tokens");
        for (int s = 0; s < nseq; ++s)
            if (cu[s + 1] < cu[s] || cu[s + 1] - cu[s] > max_seqlen)
                return fail(KVC_ERR_INVALID, "segment %d: length %d outside [0, max_seqlen]", s, cu[s + 1] - cu[s]);
    }
    kvc::PrefillArgs a;
    a.q = static_cast<const __half*>(q);
    a.k = static_cast<const __half*>(k);
    a.v = static_cast<const __half*>(v);
    a.cu_seqlens = cu_seqlens;
    a.nseq = nseq;
    a.total_tokens = total_tokens;
    a.max_seqlen = max_seqlen;
    a.Hq = Hq;
    a.Hkv = Hkv;
    a.D = head_dim;
    a.scale = scale;
    a.causal = causal ? 1 : 0;
    a.out = out;
    a.out_f32 = out_dtype == KVC_F32;
    a.window = window;
    a.sinks = sinks;
    a.split_p = p_precision == KVC_PREFILL_P_SPLIT;
    cudaError_t e = kvc::device_error_word(&a.err);
    if (e != cudaSuccess) return cuda_fail(e, "device error word");
    e = kvc::launch_prefill(a, as_stream(stream));
    if (e != cudaSuccess) return cuda_fail(e, name);
    return KVC_OK;
}

kvc_status prefill_attention_ex(const void* q, const void* k, const void* v, const int32_t* cu_seqlens, int nseq,
                                int total_tokens, int max_seqlen, int Hq, int Hkv, int head_dim, float scale,
                                int causal, int p_precision, void* out, int out_dtype, void* stream) {
    return prefill_common(q, k, v, cu_seqlens, nseq, total_tokens, max_seqlen, Hq, Hkv, head_dim, scale, causal, 0, 0,
                          p_precision, out, out_dtype, "prefill_attention launch", stream);
}

kvc_status prefill_window_attention(const void* q, const void* k, const void* v, const int32_t* cu_seqlens, int nseq,
                                    int total_tokens, int max_seqlen, int Hq, int Hkv, int head_dim, float scale,
                                    int window, int sinks, int p_precision, void* out, int out_dtype, void* stream) {
    kvc_status s = check_window(window, sinks, 1);
    if (s != KVC_OK) return s;
    if (!std::isfinite(scale)) return fail(KVC_ERR_INVALID, "scale is not finite");
    if (nseq > 0 && total_tokens > 0 && Hq > 0 && Hkv > 0 && head_dim > 0) {
        if (!aligned_to(4, {cu_seqlens})) return fail(KVC_ERR_INVALID, "cu_seqlens must be 4-byte aligned");
        const int64_t qn = static_cast<int64_t>(total_tokens) * Hq * head_dim, kn = static_cast<int64_t>(total_tokens) * Hkv * head_dim;
        s = check_overlap({{out, qn * (out_dtype == KVC_F32 ? 4 : 2)}},
                          {{q, qn * 2}, {k, kn * 2}, {v, kn * 2}, {cu_seqlens, (nseq + int64_t(1)) * 4}});
        if (s != KVC_OK) return s;
    }
    // (no segment is longer than all of the tokens, whatever max_seqlen says)
    return prefill_common(q, k, v, cu_seqlens, nseq, total_tokens, std::min(max_seqlen, total_tokens), Hq, Hkv, head_dim,
                          scale, 1, window, sinks, p_precision, out, out_dtype, "prefill_window_attention launch", stream);
}

kvc_status prefill_attention(const void* q, const void* k, const void* v, const int32_t* cu_seqlens, int nseq,
                             int total_tokens, int max_seqlen, int Hq, int Hkv, int head_dim, float scale, int causal,
                             void* out, int out_dtype, void* stream) {
    return prefill_attention_ex(q, k, v, cu_seqlens, nseq, total_tokens, max_seqlen, Hq, Hkv, head_dim, scale, causal,
                                KVC_PREFILL_P_F16, out, out_dtype, stream);
}

}  // extern "C"
