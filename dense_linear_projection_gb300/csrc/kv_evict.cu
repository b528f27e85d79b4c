// C ABI of eviction from the paged key-value cache (proj_kv_evict): argument checks and launches.
// See include/proj.h for the contract.
#include <cuda_runtime.h>

#include "kv_evict.cuh"
#include "kv_host.cuh"
#include "proj.h"

using namespace projgb;

namespace projgb {
bool prepare_evict() {
    if (cudaFuncSetAttribute(dev::kv_evict_select_kernel<true>, cudaFuncAttributeMaxDynamicSharedMemorySize, dev::kEvictSlab * 4) ==
            cudaSuccess)
        return true;
    cudaGetLastError();
    return false;
}
}  // namespace projgb

extern "C" {

proj_status_t proj_kv_evict(proj_kv_handle_t h, int64_t sequences, const int32_t *page_table, int64_t table_width,
                            const int32_t *seq_lens, const float *scores, int64_t score_tokens, const int32_t *to_table,
                            int64_t to_width, int64_t keep, int64_t recent, void *k_cache, void *v_cache, int32_t *lens_out,
                            float *scores_out, int32_t *kept, void *stream) {
    if (!h || !is_current(h->device) || sequences < 0 || !fits_table(table_width, h->d.page_size) || !fits_table(to_width, h->d.page_size))
        return PROJ_ERR_INVALID_ARG;
    const proj_kv_desc_t &d = h->d;
    if (keep < 0 || recent < 0 || recent > keep || keep > to_width * d.page_size || score_tokens < table_width * d.page_size ||
        score_tokens > kMaxDim)
        return PROJ_ERR_INVALID_ARG;
    if (sequences > kMaxDim / d.kv_heads / kEvictMostBlocks) return PROJ_ERR_UNSUPPORTED;  // one row of blocks each
    if (sequences == 0) return PROJ_OK;
    if (!seq_lens || !lens_out || (table_width > 0 && (!page_table || !scores)) || (to_width > 0 && (!to_table || !scores_out)) ||
        (keep > 0 && (!kept || !k_cache || !v_cache)))
        return PROJ_ERR_INVALID_ARG;
    if (!aligned16(k_cache) || !aligned16(v_cache) ||
        ((reinterpret_cast<uintptr_t>(page_table) | reinterpret_cast<uintptr_t>(seq_lens) | reinterpret_cast<uintptr_t>(scores) |
          reinterpret_cast<uintptr_t>(to_table) | reinterpret_cast<uintptr_t>(lens_out) | reinterpret_cast<uintptr_t>(scores_out) |
          reinterpret_cast<uintptr_t>(kept)) % 4) != 0)
        return PROJ_ERR_MISALIGNED;
    KvEvictParams p{};
    p.cache = view_of(h, page_table, table_width);
    p.to_table = to_table;
    p.to_width = to_width;
    p.sequences = sequences;
    p.score_tokens = score_tokens;
    p.keep = keep;
    p.recent = recent;
    p.seq_lens = seq_lens;
    p.scores = scores;
    p.scores_out = scores_out;
    p.lens_out = lens_out;
    p.kept = kept;
    p.k_cache = k_cache;
    p.v_cache = v_cache;
    p.elem = h->elem;
    p.status = h->status;

    // CTAs of a row: as many as give each kEvictSpan scores, within a cluster.
    const int64_t rows = sequences * d.kv_heads;
    unsigned ranks = 1;
    while (ranks < dev::kEvictCluster && table_width * d.page_size > int64_t(ranks) * dev::kEvictSpan) ranks *= 2;
    if (launch_faulted()) return PROJ_ERR_CUDA;
    cudaLaunchConfig_t cfg{};
    cudaLaunchAttribute attr[2];
    cfg.gridDim = dim3(static_cast<unsigned>(rows) * ranks);
    cfg.blockDim = dim3(dev::kEvictThreads);
    cfg.stream = as_stream(stream);
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = ranks;
    attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    // Its scores in shared memory, where they fit (65 KiB at most).
    const int64_t span = ((table_width * d.page_size + ranks - 1) / ranks + 3) / 4 * 4;
    const bool held = span <= dev::kEvictSlab;
    cfg.dynamicSmemBytes = held ? static_cast<size_t>(span) * 4 : 0;
    if (cudaLaunchKernelEx(&cfg, held ? dev::kv_evict_select_kernel<true> : dev::kv_evict_select_kernel<false>, p) != cudaSuccess) {
        cudaGetLastError();
        return PROJ_ERR_CUDA;
    }
    if (keep == 0) return PROJ_OK;
    // Tokens of a block: 256, or fewer where that leaves SMs without one; blocks of a row: enough
    // for every SM to have kEvictMostBlocks.
    int tokens = dev::kEvictCopyThreads;
    while (tokens > 32 && rows * ((keep + tokens - 1) / tokens) < 2 * int64_t(h->sm_count)) tokens /= 2;
    int64_t of_row = (int64_t(h->sm_count) * kEvictMostBlocks + rows - 1) / rows;
    if (of_row > (keep + tokens - 1) / tokens) of_row = (keep + tokens - 1) / tokens;
    return launch(dev::kv_evict_copy_kernel, dim3(static_cast<unsigned>(rows * of_row)), dev::kEvictCopyThreads, 0, stream, p,
                  static_cast<int>(of_row), tokens);
}

}  // extern "C"
