// Parameters of the paged key-value cache's kernels.
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

#include "proj_internal.h"

namespace projgb {

constexpr int kKvMaxDim = 256;
constexpr int kKvWarps = 4;                        // warps of an attention CTA
constexpr int kKvThreads = 32 * kKvWarps;
constexpr int kKvRowCost = 2;  // a row's start and join, in tiles (64 ragged sequences: 0, 1, 2 gave 170, 163, 161 us)
constexpr int kKvMinPlaces = 2;  // of a CTA (one head of 1000 tokens: 1, 2, 4 gave 11.7, 10.4, 11.7 us)
// Parts of a row that one CTA joins at once; more are joined in groups first
// (twice as large past kKvJoinMany parts).  A round trip to scratch takes about
// 1.3 us while the other CTAs stream, and the early groups meet before the last:
// one sequence of 131071 tokens, 38 parts a row, took 94 us with one group, 91.4
// in groups of 16 and 90.5 in groups of 8.
constexpr int kKvJoinOnce = 16, kKvJoinGroup = 8, kKvJoinMany = 128;

// Bits of the cache handle's status word, below 2^8: what a kernel found out of range.
constexpr int kKvErrPosition = 1 << 0;  // position past the page table or the rope table
constexpr int kKvErrSequence = 1 << 1;  // sequence id outside the page table
constexpr int kKvErrPage = 1 << 2;      // page outside the cache
constexpr int kKvErrLength = 1 << 3;    // length below zero or past the page table
constexpr int kKvErrRopeRow = 1 << 4;   // row outside the rope table
constexpr int kKvErrWait = 1 << 5;      // a bounded wait of the prefix kernel ran out

constexpr int kEvictMostBlocks = 32;  // of the eviction's copy, for each SM

// Where a sequence's tokens lie; strides in elements.
struct KvCacheView {
    int64_t page_stride, token_stride, head_stride;
    int64_t num_pages;
    const int32_t *table;
    int64_t table_width;
    int32_t page_size;
    int32_t kv_heads;
    int32_t head_dim;
};

struct KvAppendParams {
    KvCacheView cache;
    int64_t tokens, sequences, rope_positions;
    const uint16_t *q, *k, *v;
    int64_t q_stride, kv_stride, q_out_stride;
    const int32_t *positions, *seq_ids;
    const int32_t *rope_rows;  // the rope table's row of each token, or NULL: its position
    const void *q_weight, *k_weight;  // of the norms: bf16 or fp32 [head_dim], NULL: no norm
    int32_t weight_f32;
    float eps;
    const float *rope;
    int32_t q_heads;  // 0: keys and values only
    int32_t rot_dim;
    const float *k_scale, *v_scale;
    void *k_cache, *v_cache;
    uint16_t *q_out;
    int *status;
};

struct KvAttendParams {
    KvCacheView cache;
    int64_t sequences;
    const uint16_t *q;
    int64_t q_stride, out_stride;
    const void *k_cache, *v_cache;
    const float *k_scale, *v_scale;
    const int32_t *seq_lens;
    int64_t window;
    float scale;
    int32_t q_heads;
    int32_t group;        // query heads of a key head
    int32_t chunk_heads;  // of which a row takes this many at most
    int32_t chunks;       // rows of a key head
    int32_t units;        // rows of a sequence: kv_heads · chunks, or pairs of key heads
    float *partials;      // [CTA][row begun by another, row begun last][maxima, sums, heads × dim]
    uint32_t *counters;        // [sequence][unit], zero between runs
    uint32_t *group_counters;  // [slot of a partial result], zero between runs
    uint16_t *out;
    float *lse;
    int *status;
    // Scored attention and the own part of shared-prefix attention (kAttendLogits, kAttendPart):
    float *logits;   // [sequence][kv head][token][query head of it], in units of log 2
    float2 *top;     // [sequence][query head]: maximum of the logits; with logits 1 / Σ 2^(x − maximum), else the sum
    float *out32;    // [sequence][query head][head_dim]: the output before rounding
};

// Scored attention: numbers of query heads of a key head whose logits the second kernel reads four at a
// time, and for the last time.
__host__ __device__ constexpr bool scored_in_fours(int group) { return group % 4 == 0 && group <= 16; }

// What an attention kernel leaves beside, or instead of, the rounded output.
constexpr int kAttendPlain = 0;   // the output
constexpr int kAttendLogits = 1;  // the output, every logit, and each row's maximum and sum
constexpr int kAttendPart = 2;    // the unrounded output, and each row's maximum and sum

struct KvScoreParams {
    const float *logits;
    const float2 *top;
    const float *scores;
    float *scores_out;
    const int32_t *seq_lens;
    int64_t sequences, table_tokens, score_tokens, window;
    int32_t kv_heads, group;
};

struct KvEvictParams {
    KvCacheView cache;  // with the sequences' present table
    const int32_t *to_table;
    int64_t to_width, sequences, score_tokens, keep, recent;
    const int32_t *seq_lens;
    const float *scores;
    float *scores_out;  // [sequence][kv head][to_width · page_size]
    int32_t *lens_out, *kept;
    void *k_cache, *v_cache;
    int32_t elem;  // bytes of a cache element
    int *status;
};

// Shared-prefix attention: see kv_prefix.cuh.
struct KvPrefixParams {
    KvCacheView cache;  // its table: the prefix's pages, of which table_width are given
    int64_t sequences, prefix;
    const uint16_t *q;
    int64_t q_stride;
    const void *k_cache, *v_cache;
    const float *k_scale, *v_scale;
    float scale;
    int32_t group;
    int64_t row_tiles, tiles;  // of a key head's rows; of the prefix's tokens
    int32_t box;               // tokens of a TMA box, 0: copies instead
    float *partials;           // [unit + CTA][maxima, sums, values]
    int *status;
    int64_t wait_limit_ns;     // bounded waits give up after this long
    int64_t fault_place;       // fault injection: of a CTA's places, where a wait runs out; −1: none
};

struct KvCombineParams {
    const float *partials;
    const float2 *top;   // the own tokens' part
    const float *out32;
    int64_t sequences, row_tiles, tiles;
    int32_t ctas;        // of the prefix kernel
    int32_t kv_heads, group, head_dim;
    uint16_t *out;
    int64_t out_stride;
    float *lse;
};

}  // namespace projgb
