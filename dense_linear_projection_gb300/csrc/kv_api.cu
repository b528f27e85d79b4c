// C ABI of the paged key-value cache (proj_kv_*): argument checks and launches.
// See include/proj.h for the contract.
#include <cuda_runtime.h>

#include <cmath>
#include <new>

#include "kv_append.cuh"
#include "kv_host.cuh"
#include "kv_internal.h"
#include "proj.h"
#include "proj_host.h"

using namespace projgb;

namespace {

template <bool kE4m3>
proj_status_t launch_append(const KvAppendParams &p, dim3 grid, bool interleaved, bool vec, void *stream) {
    const int t = dev::kAppendThreads;
    if (interleaved)
        return vec ? launch(dev::kv_append_kernel<kE4m3, true, true>, grid, t, 0, stream, p)
                   : launch(dev::kv_append_kernel<kE4m3, true, false>, grid, t, 0, stream, p);
    return vec ? launch(dev::kv_append_kernel<kE4m3, false, true>, grid, t, 0, stream, p)
               : launch(dev::kv_append_kernel<kE4m3, false, false>, grid, t, 0, stream, p);
}

template <bool kE4m3>
proj_status_t launch_append_norm(const KvAppendParams &p, dim3 grid, int lanes, bool interleaved, bool vec, void *stream) {
    const int t = dev::kAppendThreads;
    if (interleaved)
        return vec ? launch(dev::kv_append_norm_kernel<kE4m3, true, true>, grid, t, 0, stream, p, lanes)
                   : launch(dev::kv_append_norm_kernel<kE4m3, true, false>, grid, t, 0, stream, p, lanes);
    return vec ? launch(dev::kv_append_norm_kernel<kE4m3, false, true>, grid, t, 0, stream, p, lanes)
               : launch(dev::kv_append_norm_kernel<kE4m3, false, false>, grid, t, 0, stream, p, lanes);
}

// The norms and rotary rows of proj_kv_append_normed.
struct Norms {
    const void *q, *k;
    proj_dtype_t dtype;
    float eps;
    const int32_t *rope_rows;
};

proj_status_t append(proj_kv_handle_t h, const Norms *norms, int64_t tokens, const void *q, int64_t q_stride, const void *k,
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
    if (norms && ((norms->dtype != PROJ_BF16 && norms->dtype != PROJ_F32) || !std::isfinite(norms->eps) || norms->eps < 0.f ||
                  (norms->q && !q) || (norms->rope_rows && !rope)))
        return PROJ_ERR_INVALID_ARG;
    if (tokens == 0) return PROJ_OK;
    if (!k || !v || !positions || !page_table || !k_cache || !v_cache) return PROJ_ERR_INVALID_ARG;
    if (!rows_aligned(k, kv_stride) || !rows_aligned(v, kv_stride) || !aligned16(k_cache) || !aligned16(v_cache) ||
        (q && (!rows_aligned(q, q_stride) || !rows_aligned(q_out, q_out_stride))) ||
        reinterpret_cast<uintptr_t>(rope) % 4 != 0 || reinterpret_cast<uintptr_t>(positions) % 4 != 0 ||
        reinterpret_cast<uintptr_t>(seq_ids) % 4 != 0 || reinterpret_cast<uintptr_t>(page_table) % 4 != 0)
        return PROJ_ERR_MISALIGNED;
    if (norms && (!aligned16(norms->q) || !aligned16(norms->k) || reinterpret_cast<uintptr_t>(norms->rope_rows) % 4 != 0))
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
    int lanes = units;  // threads of a head
    if (norms) {
        for (lanes = 1; lanes < units;) lanes *= 2;
        p.rope_rows = norms->rope_rows;
        p.q_weight = norms->q;
        p.k_weight = norms->k;
        p.weight_f32 = norms->dtype == PROJ_F32;
        p.eps = norms->eps;
    }
    const int slots = dev::kAppendThreads / lanes;
    const int passes = (p.q_heads + 2 * d.kv_heads + slots - 1) / slots;
    const int64_t want = 4 * int64_t(h->sm_count) / tokens;
    const int parts = static_cast<int>(want < 1 ? 1 : want < passes ? want : passes);
    const dim3 grid(static_cast<unsigned>(tokens), static_cast<unsigned>(parts));
    const bool vec = rot_dim % 16 == 0;
    if (norms)
        return d.kv_dtype == PROJ_E4M3 ? launch_append_norm<true>(p, grid, lanes, interleaved != 0, vec, stream)
                                       : launch_append_norm<false>(p, grid, lanes, interleaved != 0, vec, stream);
    return d.kv_dtype == PROJ_E4M3 ? launch_append<true>(p, grid, interleaved != 0, vec, stream)
                                   : launch_append<false>(p, grid, interleaved != 0, vec, stream);
}

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
    h->fault_place = fault_wait_place();
    const int group = d.q_heads / d.kv_heads, most = d.head_dim <= 128 ? 16 : 8;
    h->chunks = (group + most - 1) / most;
    h->chunk_heads = (group + h->chunks - 1) / h->chunks;
    // Two key heads a row where a token's row of one is short: longer pieces of
    // memory and half the rows (an 8-bit cache of 128-wide heads 104 -> 95 us, a
    // window over 64-wide heads 36.4 -> 33.4; with heads before tokens in memory
    // 91 -> 93 and 34.5 -> 32.6).
    const int row_bytes = (d.head_dim <= 64 ? 64 : d.head_dim <= 128 ? 128 : 256) * elem;
    if (row_bytes <= 128 && d.kv_heads % 2 == 0 && h->chunks == 1) h->key_heads = 2;
    const AttendInstance a = instance_for<kAttendPlain>(h);
    if (!prepare_attend<kAttendPlain>(h) || !prepare_scored(h) || !prepare_shared(h) || !prepare_evict()) {
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
    return append(h, nullptr, tokens, q, q_stride, k, v, kv_stride, positions, seq_ids, page_table, sequences, table_width, rope,
                  rope_positions, rot_dim, interleaved, k_scale, v_scale, k_cache, v_cache, q_out, q_out_stride, stream);
}

proj_status_t proj_kv_append_normed(proj_kv_handle_t h, int64_t tokens, const void *q, int64_t q_stride, const void *k,
                                    const void *v, int64_t kv_stride, const void *q_weight, const void *k_weight,
                                    proj_dtype_t weight_dtype, float eps, const int32_t *positions, const int32_t *seq_ids,
                                    const int32_t *page_table, int64_t sequences, int64_t table_width,
                                    const int32_t *rope_rows, const float *rope, int64_t rope_positions, int32_t rot_dim,
                                    int interleaved, const float *k_scale, const float *v_scale, void *k_cache, void *v_cache,
                                    void *q_out, int64_t q_out_stride, void *stream) {
    const Norms norms{q_weight, k_weight, weight_dtype, eps, rope_rows};
    return append(h, &norms, tokens, q, q_stride, k, v, kv_stride, positions, seq_ids, page_table, sequences, table_width, rope,
                  rope_positions, rot_dim, interleaved, k_scale, v_scale, k_cache, v_cache, q_out, q_out_stride, stream);
}

proj_status_t proj_kv_attend(proj_kv_handle_t h, int64_t sequences, const void *q, int64_t q_stride,
                             const void *k_cache, const void *v_cache, const float *k_scale, const float *v_scale,
                             const int32_t *page_table, int64_t table_width, const int32_t *seq_lens, int64_t window,
                             float scale, void *out, int64_t out_stride, float *lse, void *stream) {
    KvAttendParams p{};
    const proj_status_t st = attend_params(h, {sequences, q, q_stride, k_cache, v_cache, k_scale, v_scale, page_table, table_width,
                                               seq_lens, window, scale, out, out_stride, lse}, p);
    return st != PROJ_OK || sequences == 0 ? st : launch_attend<kAttendPlain>(h, p, stream);
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
    // A wait that ran out is told first; what else was found stays for the next call.  (The bits are in
    // the word's first byte.)
    const int rest = (word & kKvErrWait) ? word & ~kKvErrWait : 0;
    if (cudaMemsetAsync(h->status, rest, 1, as_stream(stream)) != cudaSuccess ||
        cudaStreamSynchronize(as_stream(stream)) != cudaSuccess) {
        cudaGetLastError();
        return PROJ_ERR_CUDA;
    }
    return (word & kKvErrWait) ? PROJ_ERR_DEVICE_TIMEOUT : PROJ_ERR_INVALID_ARG;
}

proj_status_t proj_kv_destroy(proj_kv_handle_t h) {
    if (!h) return PROJ_OK;
    const proj_status_t st = cudaFree(h->scratch) == cudaSuccess ? PROJ_OK : PROJ_ERR_CUDA;
    delete h;
    return st;
}

}  // extern "C"
