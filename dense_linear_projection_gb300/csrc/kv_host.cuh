// Host side of the paged key-value cache shared by its translation units: the handle, argument
// checks, launches and the choice of an attention kernel's instance.
#pragma once

#include <cuda_runtime.h>

#include <cmath>

#include "kv_attend.cuh"
#include "kv_internal.h"
#include "proj.h"
#include "proj_host.h"

struct proj_kv_s {
    proj_kv_desc_t d{};
    int sm_count = 0, device = 0;
    int elem = 2;  // bytes of a cache element
    int chunk_heads = 0, chunks = 0;  // rows of a key head: query heads of each, and how many
    int key_heads = 1;                // key heads of a row: 1 or 2
    int grid = 0;                     // CTAs of an attention launch at most
    void *scratch = nullptr;          // status word, counters, partial results
    int *status = nullptr;
    uint32_t *counters = nullptr, *group_counters = nullptr;
    float *partials = nullptr;
    int64_t fault_place = -1;         // where the next prefix kernel's wait runs out (fault injection)
};

namespace projgb {

inline KvCacheView view_of(const proj_kv_s *h, const int32_t *table, int64_t table_width) {
    KvCacheView c{};
    c.page_stride = h->d.page_stride;
    c.token_stride = h->d.token_stride;
    c.head_stride = h->d.head_stride;
    c.num_pages = h->d.num_pages;
    c.table = table;
    c.table_width = table_width;
    c.page_size = h->d.page_size;
    c.kv_heads = h->d.kv_heads;
    c.head_dim = h->d.head_dim;
    return c;
}

// A bf16 row array: base and row stride whole 16-byte multiples.
inline bool rows_aligned(const void *p, int64_t stride) { return aligned16(p) && stride % 8 == 0; }

// Tokens are counted in 32 bits, with room for a tile past the last one.
inline bool fits_table(int64_t table_width, int32_t page_size) {
    return table_width >= 0 && table_width <= kMaxDim && table_width * page_size <= kMaxDim - 4095;
}

// A launch whose set-up may overlap the preceding kernel's tail.
template <typename... P, typename... A>
proj_status_t launch(void (*kernel)(P...), dim3 grid, int threads, size_t smem, void *stream, A... args) {
    if (launch_faulted()) return PROJ_ERR_CUDA;
    cudaLaunchConfig_t cfg{};
    cudaLaunchAttribute attr[1];
    cfg.gridDim = grid;
    cfg.blockDim = dim3(static_cast<unsigned>(threads));
    cfg.dynamicSmemBytes = smem;
    cfg.stream = as_stream(stream);
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    if (cudaLaunchKernelEx(&cfg, kernel, args...) != cudaSuccess) {
        cudaGetLastError();
        return PROJ_ERR_CUDA;
    }
    return PROJ_OK;
}

// The attention kernel's instance for a head width and a row's heads.
using AttendKernel = void (*)(KvAttendParams);
struct AttendInstance {
    AttendKernel kernel;
    int smem, per_sm, part, tile;  // shared memory, CTAs an SM, floats of a partial result, tokens of a tile
};

template <int kLeaves, bool kE4m3, int kDim, int kNT, int kKeyHeads>
AttendInstance instance_of() {
    using Shape = dev::AttendShape<kE4m3, kDim, kNT, kKeyHeads>;
    return {dev::kv_attend_kernel<kE4m3, kDim, kNT, kKeyHeads, kLeaves>, Shape::kSmem, Shape::kPerSm, Shape::kRowHeads * (kDim + 2),
            Shape::kTile};
}

// Two key heads a row, where the cache's rows are at most 128 bytes.
template <int kLeaves, bool kE4m3, int kDim, int kNT>
AttendInstance instance_of(int key_heads) {
    if constexpr (kDim * (kE4m3 ? 1 : 2) <= 128)
        if (key_heads == 2) return instance_of<kLeaves, kE4m3, kDim, kNT, 2>();
    return instance_of<kLeaves, kE4m3, kDim, kNT, 1>();
}

// Rows of at most 8 query heads, or 16 where the group is larger and the
// accumulators of 16 fit the registers (heads up to 128 wide).
template <int kLeaves, bool kE4m3>
AttendInstance instance_for(int head_dim, int chunk_heads, int key_heads) {
    if (head_dim <= 64) return chunk_heads <= 8 ? instance_of<kLeaves, kE4m3, 64, 1>(key_heads) : instance_of<kLeaves, kE4m3, 64, 2>(key_heads);
    if (head_dim <= 128) return chunk_heads <= 8 ? instance_of<kLeaves, kE4m3, 128, 1>(key_heads) : instance_of<kLeaves, kE4m3, 128, 2>(key_heads);
    return instance_of<kLeaves, kE4m3, 256, 1>(key_heads);
}

template <int kLeaves>
AttendInstance instance_for(const proj_kv_s *h) {
    return h->d.kv_dtype == PROJ_E4M3 ? instance_for<kLeaves, true>(h->d.head_dim, h->chunk_heads, h->key_heads)
                                      : instance_for<kLeaves, false>(h->d.head_dim, h->chunk_heads, h->key_heads);
}

// An attention kernel's arguments, checked; the outputs' own are the caller's to set.
struct AttendArgs {
    int64_t sequences;
    const void *q;
    int64_t q_stride;
    const void *k_cache, *v_cache;
    const float *k_scale, *v_scale;
    const int32_t *page_table;
    int64_t table_width;
    const int32_t *seq_lens;
    int64_t window;
    float scale;
    void *out;
    int64_t out_stride;
    float *lse;
};

// PROJ_OK with sequences > 0: `p` is filled.
inline proj_status_t attend_params(const proj_kv_s *h, const AttendArgs &a, KvAttendParams &p) {
    if (!h || !is_current(h->device) || a.sequences < 0 || a.sequences > h->d.max_sequences || a.window < 0 ||
        !std::isfinite(a.scale) || !fits_table(a.table_width, h->d.page_size))
        return PROJ_ERR_INVALID_ARG;
    const proj_kv_desc_t &d = h->d;
    if (a.q_stride < 0 || a.out_stride < int64_t(d.q_heads) * d.head_dim) return PROJ_ERR_INVALID_ARG;
    if (a.sequences == 0) return PROJ_OK;
    if (!a.q || !a.seq_lens || !a.out) return PROJ_ERR_INVALID_ARG;
    if (a.table_width > 0 && (!a.k_cache || !a.v_cache || !a.page_table)) return PROJ_ERR_INVALID_ARG;
    if (!rows_aligned(a.q, a.q_stride) || !rows_aligned(a.out, a.out_stride) || !aligned16(a.k_cache) || !aligned16(a.v_cache) ||
        reinterpret_cast<uintptr_t>(a.lse) % 4 != 0 || reinterpret_cast<uintptr_t>(a.seq_lens) % 4 != 0 ||
        reinterpret_cast<uintptr_t>(a.page_table) % 4 != 0)
        return PROJ_ERR_MISALIGNED;
    p.cache = view_of(h, a.page_table, a.table_width);
    p.sequences = a.sequences;
    p.q = static_cast<const uint16_t *>(a.q);
    p.q_stride = a.q_stride;
    p.out_stride = a.out_stride;
    p.k_cache = a.k_cache;
    p.v_cache = a.v_cache;
    p.k_scale = a.k_scale;
    p.v_scale = a.v_scale;
    p.seq_lens = a.seq_lens;
    p.window = a.window;
    p.scale = a.scale;
    p.q_heads = d.q_heads;
    p.out = static_cast<uint16_t *>(a.out);
    p.lse = a.lse;
    p.status = h->status;
    p.group = d.q_heads / d.kv_heads;
    p.chunk_heads = h->chunk_heads;
    p.chunks = h->chunks;
    p.units = d.kv_heads / h->key_heads * h->chunks;
    p.partials = h->partials;
    p.counters = h->counters;
    p.group_counters = h->group_counters;
    return PROJ_OK;
}

template <int kLeaves>
proj_status_t launch_attend(const proj_kv_s *h, const KvAttendParams &p, void *stream) {
    // No more CTAs than there can be tiles (one where every length is zero).
    const AttendInstance a = instance_for<kLeaves>(h);
    int64_t tiles = (p.cache.table_width * h->d.page_size + a.tile - 1) / a.tile;
    if (p.window > 0 && p.window / a.tile + 2 < tiles) tiles = p.window / a.tile + 2;
    const int64_t want = p.sequences * p.units * (tiles > 0 ? tiles : 1);
    return launch(a.kernel, dim3(static_cast<unsigned>(want < h->grid ? want : h->grid)), kKvThreads,
                  static_cast<size_t>(a.smem), stream, p);
}

// Allows an attention kernel its shared memory; at the handle's making, not while a graph is captured.
template <int kLeaves>
bool prepare_attend(const proj_kv_s *h) {
    const AttendInstance a = instance_for<kLeaves>(h);
    if (cudaFuncSetAttribute(a.kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, a.smem) == cudaSuccess) return true;
    cudaGetLastError();
    return false;
}

// The same for the kernels of scored and shared-prefix attention and of eviction (kv_scored.cu,
// kv_shared.cu, kv_evict.cu).
bool prepare_evict();
bool prepare_scored(const proj_kv_s *h);
bool prepare_shared(const proj_kv_s *h);

inline size_t rounded(size_t bytes) { return (bytes + 255) / 256 * 256; }

}  // namespace projgb
