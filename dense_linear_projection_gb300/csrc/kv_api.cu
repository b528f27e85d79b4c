// C ABI of the paged key-value cache (proj_kv_*): argument checks and launches.
// See include/proj.h for the contract.
#include <cuda_runtime.h>

#include <cmath>
#include <new>

#include "kv_append.cuh"
#include "kv_attend.cuh"
#include "kv_internal.h"
#include "proj.h"
#include "proj_host.h"

using namespace projgb;

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
};

namespace {

KvCacheView view_of(const proj_kv_s *h, const int32_t *table, int64_t table_width) {
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
bool rows_aligned(const void *p, int64_t stride) { return aligned16(p) && stride % 8 == 0; }

// Tokens are counted in 32 bits, with room for a tile past the last one.
bool fits_table(int64_t table_width, int32_t page_size) {
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

template <bool kE4m3>
proj_status_t launch_append(const KvAppendParams &p, dim3 grid, bool interleaved, bool vec, void *stream) {
    const int t = dev::kAppendThreads;
    if (interleaved)
        return vec ? launch(dev::kv_append_kernel<kE4m3, true, true>, grid, t, 0, stream, p)
                   : launch(dev::kv_append_kernel<kE4m3, true, false>, grid, t, 0, stream, p);
    return vec ? launch(dev::kv_append_kernel<kE4m3, false, true>, grid, t, 0, stream, p)
               : launch(dev::kv_append_kernel<kE4m3, false, false>, grid, t, 0, stream, p);
}

// The attention kernel's instance for a head width and a row's heads.
using AttendKernel = void (*)(KvAttendParams);
struct AttendInstance {
    AttendKernel kernel;
    int smem, per_sm, part, tile;  // shared memory, CTAs an SM, floats of a partial result, tokens of a tile
};

template <bool kE4m3, int kDim, int kNT, int kKeyHeads>
AttendInstance instance_of() {
    using Shape = dev::AttendShape<kE4m3, kDim, kNT, kKeyHeads>;
    return {dev::kv_attend_kernel<kE4m3, kDim, kNT, kKeyHeads>, Shape::kSmem, Shape::kPerSm, Shape::kRowHeads * (kDim + 2),
            Shape::kTile};
}

// Two key heads a row, where the cache's rows are at most 128 bytes.
template <bool kE4m3, int kDim, int kNT>
AttendInstance instance_of(int key_heads) {
    if constexpr (kDim * (kE4m3 ? 1 : 2) <= 128)
        if (key_heads == 2) return instance_of<kE4m3, kDim, kNT, 2>();
    return instance_of<kE4m3, kDim, kNT, 1>();
}

// Rows of at most 8 query heads, or 16 where the group is larger and the
// accumulators of 16 fit the registers (heads up to 128 wide).
template <bool kE4m3>
AttendInstance instance_for(int head_dim, int chunk_heads, int key_heads) {
    if (head_dim <= 64) return chunk_heads <= 8 ? instance_of<kE4m3, 64, 1>(key_heads) : instance_of<kE4m3, 64, 2>(key_heads);
    if (head_dim <= 128) return chunk_heads <= 8 ? instance_of<kE4m3, 128, 1>(key_heads) : instance_of<kE4m3, 128, 2>(key_heads);
    return instance_of<kE4m3, 256, 1>(key_heads);
}

AttendInstance instance_for(const proj_kv_s *h) {
    return h->d.kv_dtype == PROJ_E4M3 ? instance_for<true>(h->d.head_dim, h->chunk_heads, h->key_heads)
                                      : instance_for<false>(h->d.head_dim, h->chunk_heads, h->key_heads);
}

size_t rounded(size_t bytes) { return (bytes + 255) / 256 * 256; }

}  // namespace

extern "C" {

proj_status_t proj_kv_create(proj_kv_handle_t *out, const proj_kv_desc_t *desc, void *stream) {
    if (!out) return PROJ_ERR_INVALID_ARG;
    *out = nullptr;
    if (!desc) return PROJ_ERR_INVALID_ARG;
    const proj_kv_desc_t &d = *desc;
    if (d.kv_dtype != PROJ_BF16 && d.kv_dtype != PROJ_E4M3) return PROJ_ERR_UNSUPPORTED;
    if (d.num_pages < 0 || d.num_pages > kMaxDim || d.page_size < 1 || d.q_heads < 1 || d.kv_heads < 1 ||
        d.q_heads % d.kv_heads != 0 || d.head_dim < 1 || d.max_sequences < 0 || d.max_sequences > kMaxDim ||
        d.page_stride < 0 || d.token_stride < 0 || d.head_stride < 0)
        return PROJ_ERR_INVALID_ARG;
    if (d.head_dim % 16 != 0 || d.head_dim > kKvMaxDim) return PROJ_ERR_UNSUPPORTED;
    const int elem = d.kv_dtype == PROJ_E4M3 ? 1 : 2;
    if ((d.page_stride * elem) % 16 != 0 || (d.token_stride * elem) % 16 != 0 || (d.head_stride * elem) % 16 != 0)
        return PROJ_ERR_MISALIGNED;
    const int sms = gb300_sm_count();
    if (sms <= 0) return sms < 0 ? PROJ_ERR_CUDA : PROJ_ERR_UNSUPPORTED;
    proj_kv_s *h = new (std::nothrow) proj_kv_s();
    if (!h) return PROJ_ERR_OUT_OF_MEMORY;
    h->d = d;
    h->sm_count = sms;
    h->device = device_of_handle();
    h->elem = elem;
    const int group = d.q_heads / d.kv_heads, most = d.head_dim <= 128 ? 16 : 8;
    h->chunks = (group + most - 1) / most;
    h->chunk_heads = (group + h->chunks - 1) / h->chunks;
    // Two key heads a row where a token's row of one is short: longer pieces of
    // memory and half the rows (an 8-bit cache of 128-wide heads 104 -> 95 us, a
    // window over 64-wide heads 36.4 -> 33.4; with heads before tokens in memory
    // 91 -> 93 and 34.5 -> 32.6).
    const int row_bytes = (d.head_dim <= 64 ? 64 : d.head_dim <= 128 ? 128 : 256) * elem;
    if (row_bytes <= 128 && d.kv_heads % 2 == 0 && h->chunks == 1) h->key_heads = 2;
    const AttendInstance a = instance_for(h);
    if (cudaFuncSetAttribute(a.kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, a.smem) != cudaSuccess) {
        cudaGetLastError();
        delete h;
        return PROJ_ERR_CUDA;
    }
    h->grid = h->sm_count * a.per_sm;
    const size_t counters = rounded(static_cast<size_t>(d.max_sequences) * (d.kv_heads / h->key_heads) * h->chunks * 4);
    const size_t groups = rounded(static_cast<size_t>(h->grid) * 2 * 4);
    const size_t clear = 256 + counters + groups;
    const size_t bytes = clear + static_cast<size_t>(h->grid) * 2 * a.part * 4;
    if (dev_malloc(&h->scratch, bytes) != cudaSuccess) {
        cudaGetLastError();
        delete h;
        return PROJ_ERR_OUT_OF_MEMORY;
    }
    h->status = static_cast<int *>(h->scratch);
    h->counters = reinterpret_cast<uint32_t *>(static_cast<uint8_t *>(h->scratch) + 256);
    h->group_counters = reinterpret_cast<uint32_t *>(static_cast<uint8_t *>(h->scratch) + 256 + counters);
    h->partials = reinterpret_cast<float *>(static_cast<uint8_t *>(h->scratch) + clear);
    if (cudaMemsetAsync(h->scratch, 0, clear, as_stream(stream)) != cudaSuccess ||
        cudaStreamSynchronize(as_stream(stream)) != cudaSuccess) {
        cudaGetLastError();
        cudaFree(h->scratch);
        delete h;
        return PROJ_ERR_CUDA;
    }
    *out = h;
    return PROJ_OK;
}

proj_status_t proj_kv_append(proj_kv_handle_t h, int64_t tokens, const void *q, int64_t q_stride, const void *k,
                             const void *v, int64_t kv_stride, const int32_t *positions, const int32_t *seq_ids,
                             const int32_t *page_table, int64_t sequences, int64_t table_width, const float *rope,
                             int64_t rope_positions, int32_t rot_dim, int interleaved, const float *k_scale,
                             const float *v_scale, void *k_cache, void *v_cache, void *q_out, int64_t q_out_stride,
                             void *stream) {
    if (!h || !is_current(h->device) || tokens < 0 || tokens > kMaxDim || sequences < 0 || sequences > kMaxDim || rope_positions < 0 ||
        (interleaved != 0 && interleaved != 1) || !fits_table(table_width, h->d.page_size))
        return PROJ_ERR_INVALID_ARG;
    const proj_kv_desc_t &d = h->d;
    if (rope ? rot_dim < 2 || rot_dim % 2 != 0 || rot_dim > d.head_dim : rot_dim != 0) return PROJ_ERR_INVALID_ARG;
    if ((q != nullptr) != (q_out != nullptr)) return PROJ_ERR_INVALID_ARG;
    if (q && (q_stride < 0 || q_out_stride < int64_t(d.q_heads) * d.head_dim)) return PROJ_ERR_INVALID_ARG;
    if (kv_stride < 0) return PROJ_ERR_INVALID_ARG;
    if (tokens == 0) return PROJ_OK;
    if (!k || !v || !positions || !page_table || !k_cache || !v_cache) return PROJ_ERR_INVALID_ARG;
    if (!rows_aligned(k, kv_stride) || !rows_aligned(v, kv_stride) || !aligned16(k_cache) || !aligned16(v_cache) ||
        (q && (!rows_aligned(q, q_stride) || !rows_aligned(q_out, q_out_stride))) ||
        reinterpret_cast<uintptr_t>(rope) % 4 != 0 || reinterpret_cast<uintptr_t>(positions) % 4 != 0 ||
        reinterpret_cast<uintptr_t>(seq_ids) % 4 != 0 || reinterpret_cast<uintptr_t>(page_table) % 4 != 0)
        return PROJ_ERR_MISALIGNED;
    KvAppendParams p{};
    p.cache = view_of(h, page_table, table_width);
    p.tokens = tokens;
    p.sequences = sequences;
    p.rope_positions = rope_positions;
    p.q = static_cast<const uint16_t *>(q);
    p.k = static_cast<const uint16_t *>(k);
    p.v = static_cast<const uint16_t *>(v);
    p.q_stride = q_stride;
    p.kv_stride = kv_stride;
    p.q_out_stride = q_out_stride;
    p.positions = positions;
    p.seq_ids = seq_ids;
    p.rope = rope;
    p.q_heads = q ? d.q_heads : 0;
    p.rot_dim = rot_dim;
    p.k_scale = k_scale;
    p.v_scale = v_scale;
    p.k_cache = k_cache;
    p.v_cache = v_cache;
    p.q_out = static_cast<uint16_t *>(q_out);
    p.status = h->status;
    // Few tokens: the heads are spread over blocks too.
    const int units = (rot_dim / 2 + 7) / 8 + (d.head_dim - rot_dim + 15) / 16;
    const int slots = dev::kAppendThreads / units;
    const int passes = (p.q_heads + 2 * d.kv_heads + slots - 1) / slots;
    const int64_t want = 4 * int64_t(h->sm_count) / tokens;
    const int parts = static_cast<int>(want < 1 ? 1 : want < passes ? want : passes);
    const dim3 grid(static_cast<unsigned>(tokens), static_cast<unsigned>(parts));
    const bool vec = rot_dim % 16 == 0;
    return d.kv_dtype == PROJ_E4M3 ? launch_append<true>(p, grid, interleaved != 0, vec, stream)
                                   : launch_append<false>(p, grid, interleaved != 0, vec, stream);
}

proj_status_t proj_kv_attend(proj_kv_handle_t h, int64_t sequences, const void *q, int64_t q_stride,
                             const void *k_cache, const void *v_cache, const float *k_scale, const float *v_scale,
                             const int32_t *page_table, int64_t table_width, const int32_t *seq_lens, int64_t window,
                             float scale, void *out, int64_t out_stride, float *lse, void *stream) {
    if (!h || !is_current(h->device) || sequences < 0 || sequences > h->d.max_sequences || window < 0 || !std::isfinite(scale) ||
        !fits_table(table_width, h->d.page_size))
        return PROJ_ERR_INVALID_ARG;
    const proj_kv_desc_t &d = h->d;
    if (q_stride < 0 || out_stride < int64_t(d.q_heads) * d.head_dim) return PROJ_ERR_INVALID_ARG;
    if (sequences == 0) return PROJ_OK;
    if (!q || !seq_lens || !out) return PROJ_ERR_INVALID_ARG;
    if (table_width > 0 && (!k_cache || !v_cache || !page_table)) return PROJ_ERR_INVALID_ARG;
    if (!rows_aligned(q, q_stride) || !rows_aligned(out, out_stride) || !aligned16(k_cache) || !aligned16(v_cache) ||
        reinterpret_cast<uintptr_t>(lse) % 4 != 0 || reinterpret_cast<uintptr_t>(seq_lens) % 4 != 0 ||
        reinterpret_cast<uintptr_t>(page_table) % 4 != 0)
        return PROJ_ERR_MISALIGNED;
    KvAttendParams p{};
    p.cache = view_of(h, page_table, table_width);
    p.sequences = sequences;
    p.q = static_cast<const uint16_t *>(q);
    p.q_stride = q_stride;
    p.out_stride = out_stride;
    p.k_cache = k_cache;
    p.v_cache = v_cache;
    p.k_scale = k_scale;
    p.v_scale = v_scale;
    p.seq_lens = seq_lens;
    p.window = window;
    p.scale = scale;
    p.q_heads = d.q_heads;
    p.out = static_cast<uint16_t *>(out);
    p.lse = lse;
    p.status = h->status;
    p.group = d.q_heads / d.kv_heads;
    p.chunk_heads = h->chunk_heads;
    p.chunks = h->chunks;
    p.units = d.kv_heads / h->key_heads * h->chunks;
    p.partials = h->partials;
    p.counters = h->counters;
    p.group_counters = h->group_counters;
    // No more CTAs than there can be tiles (one where every length is zero).
    const AttendInstance a = instance_for(h);
    int64_t tiles = (table_width * d.page_size + a.tile - 1) / a.tile;
    if (window > 0 && window / a.tile + 2 < tiles) tiles = window / a.tile + 2;
    const int64_t want = sequences * p.units * (tiles > 0 ? tiles : 1);
    return launch(a.kernel, dim3(static_cast<unsigned>(want < h->grid ? want : h->grid)), kKvThreads,
                  static_cast<size_t>(a.smem), stream, p);
}

proj_status_t proj_kv_device_status(proj_kv_handle_t h, void *stream) {
    if (!h || !is_current(h->device)) return PROJ_ERR_INVALID_ARG;
    // Read and cleared in the stream's order: a kernel launched after this call on
    // any stream finds the word as this call leaves it.
    int word = 0;
    if (cudaMemcpyAsync(&word, h->status, sizeof word, cudaMemcpyDeviceToHost, as_stream(stream)) != cudaSuccess ||
        cudaStreamSynchronize(as_stream(stream)) != cudaSuccess) {
        cudaGetLastError();
        return PROJ_ERR_CUDA;
    }
    if (word == 0) return PROJ_OK;
    if (cudaMemsetAsync(h->status, 0, sizeof word, as_stream(stream)) != cudaSuccess ||
        cudaStreamSynchronize(as_stream(stream)) != cudaSuccess) {
        cudaGetLastError();
        return PROJ_ERR_CUDA;
    }
    return PROJ_ERR_INVALID_ARG;
}

proj_status_t proj_kv_destroy(proj_kv_handle_t h) {
    if (!h) return PROJ_OK;
    const proj_status_t st = cudaFree(h->scratch) == cudaSuccess ? PROJ_OK : PROJ_ERR_CUDA;
    delete h;
    return st;
}

}  // extern "C"
