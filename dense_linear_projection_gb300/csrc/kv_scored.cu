// C ABI of scored attention (proj_kv_attend_scored): argument checks and launches.
// See include/proj.h for the contract.
#include <cuda_runtime.h>

#include "kv_host.cuh"
#include "kv_scored.cuh"
#include "proj.h"

using namespace projgb;

namespace projgb {
bool prepare_scored(const proj_kv_s *h) { return prepare_attend<kAttendLogits>(h); }
}  // namespace projgb

namespace {

// The workspace: every row's maximum and sum, then the logits.
size_t tops_bytes(const proj_kv_s *h, int64_t sequences) { return rounded(static_cast<size_t>(sequences) * h->d.q_heads * sizeof(float2)); }

}  // namespace

extern "C" {

proj_status_t proj_kv_scored_workspace(proj_kv_handle_t h, int64_t sequences, int64_t table_width, size_t *bytes) {
    if (!bytes) return PROJ_ERR_INVALID_ARG;
    *bytes = 0;
    if (!h || sequences < 0 || sequences > h->d.max_sequences || !fits_table(table_width, h->d.page_size)) return PROJ_ERR_INVALID_ARG;
    *bytes = tops_bytes(h, sequences) + static_cast<size_t>(sequences) * h->d.q_heads * static_cast<size_t>(table_width) * h->d.page_size * 4;
    return PROJ_OK;
}

proj_status_t proj_kv_attend_scored(proj_kv_handle_t h, int64_t sequences, const void *q, int64_t q_stride,
                                    const void *k_cache, const void *v_cache, const float *k_scale, const float *v_scale,
                                    const int32_t *page_table, int64_t table_width, const int32_t *seq_lens, int64_t window,
                                    float scale, const float *scores, float *scores_out, int64_t score_tokens,
                                    void *workspace, void *out, int64_t out_stride, float *lse, void *stream) {
    KvAttendParams p{};
    const proj_status_t st = attend_params(h, {sequences, q, q_stride, k_cache, v_cache, k_scale, v_scale, page_table, table_width,
                                               seq_lens, window, scale, out, out_stride, lse}, p);
    if (st != PROJ_OK) return st;
    const int64_t table_tokens = table_width * h->d.page_size;
    if (score_tokens < table_tokens || score_tokens > kMaxDim) return PROJ_ERR_INVALID_ARG;
    if (sequences == 0) return PROJ_OK;
    if (!workspace || (score_tokens > 0 && (!scores || !scores_out))) return PROJ_ERR_INVALID_ARG;
    if (!aligned16(workspace) || reinterpret_cast<uintptr_t>(scores) % 4 != 0 || reinterpret_cast<uintptr_t>(scores_out) % 4 != 0)
        return PROJ_ERR_MISALIGNED;
    p.top = static_cast<float2 *>(workspace);
    p.logits = reinterpret_cast<float *>(static_cast<uint8_t *>(workspace) + tops_bytes(h, sequences));
    const proj_status_t first = launch_attend<kAttendLogits>(h, p, stream);
    if (first != PROJ_OK || score_tokens == 0) return first;

    KvScoreParams s{};
    s.logits = p.logits;
    s.top = p.top;
    s.scores = scores;
    s.scores_out = scores_out;
    s.seq_lens = seq_lens;
    s.sequences = sequences;
    s.table_tokens = table_tokens;
    s.score_tokens = score_tokens;
    s.window = window;
    s.kv_heads = h->d.kv_heads;
    s.group = p.group;
    // Blocks enough for every SM, no more of a row than it has tokens for.
    const bool ahead = p.group == 8 || p.group == 4;
    const int64_t at_once = int64_t(dev::kScoreThreads) * (ahead ? dev::kScoreAhead : 1);
    const int64_t rows = sequences * h->d.kv_heads, most = (score_tokens + at_once - 1) / at_once;
    int64_t of_row = (int64_t(h->sm_count) * 32 + rows - 1) / rows;
    if (of_row > most) of_row = most;
    if (rows * of_row > kMaxDim) return PROJ_ERR_UNSUPPORTED;
    const dim3 grid(static_cast<unsigned>(rows * of_row));
    const int blocks = static_cast<int>(of_row), t = dev::kScoreThreads;
    if (p.group == 8) return launch(dev::kv_score_kernel<8>, grid, t, 0, stream, s, blocks);
    if (p.group == 4) return launch(dev::kv_score_kernel<4>, grid, t, 0, stream, s, blocks);
    return launch(dev::kv_score_kernel<0>, grid, t, 0, stream, s, blocks);
}

}  // extern "C"
