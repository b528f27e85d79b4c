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

constexpr int kScoreBlocks = 32;  // of an SM, at least

// Blocks enough for every SM, no more of a row than it has tokens for.
template <int kGroup>
proj_status_t launch_score(const proj_kv_s *h, const KvScoreParams &s, void *stream) {
    const int64_t at_once = int64_t(dev::kScoreThreads) * dev::kScoreAhead<kGroup>;
    const int64_t rows = s.sequences * s.kv_heads, most = (s.score_tokens + at_once - 1) / at_once;
    int64_t of_row = (int64_t(h->sm_count) * kScoreBlocks + rows - 1) / rows;
    if (of_row > most) of_row = most;
    return launch(dev::kv_score_kernel<kGroup>, dim3(static_cast<unsigned>(rows * of_row)), dev::kScoreThreads, 0, stream, s,
                  static_cast<int>(of_row));
}

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
    // (Before anything is launched: the scores' grid has at most a block a row more than this.)
    if (sequences > (kMaxDim - int64_t(h->sm_count) * kScoreBlocks) / h->d.kv_heads) return PROJ_ERR_UNSUPPORTED;
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
    static_assert(scored_in_fours(4) && scored_in_fours(8) && scored_in_fours(12) && scored_in_fours(16) && !scored_in_fours(20));
    switch (p.group) {
        case 4: return launch_score<4>(h, s, stream);
        case 8: return launch_score<8>(h, s, stream);
        case 12: return launch_score<12>(h, s, stream);
        case 16: return launch_score<16>(h, s, stream);
        default: return launch_score<0>(h, s, stream);
    }
}

}  // extern "C"
