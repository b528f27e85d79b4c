// Device code of scored attention's second kernel: each cached token's weight, added to its score.
#pragma once

#include "kv_attend.cuh"

namespace projgb {
namespace dev {

// Mathematics.  scores_out[t] = scores[t] + Σ_h 2^(x[t,h] − m[h]) / l[h] over the query
// heads h of one key head: the softmax weights of the attention kernel before, which
// left x, m and 1 / l (a weight is known only once a row's last token is).
//
// What bounds it: bytes, 4 of x a query head and token (written by the one kernel and
// read by this one: 8 heads are 64 bytes, next to 512 of keys and values) and the
// scores.  Computing x again from the keys would read 256 bytes for those 64.
constexpr int kScoreThreads = 256;

// Four logits, not needed again.
__device__ __forceinline__ float4 load_once(const float *from, uint64_t policy) {
    float4 v;
    asm volatile("ld.global.L2::cache_hint.v4.f32 {%0, %1, %2, %3}, [%4], %5;"
                 : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w)
                 : "l"(from), "l"(policy));
    return v;
}

template <bool kVec>  // the heads of a token in whole float4s
__global__ void __launch_bounds__(kScoreThreads) kv_score_kernel(const KvScoreParams p, const int blocks_of_row) {
    griddep_launch_dependents();
    griddep_wait();
    const int64_t row = blockIdx.x / blocks_of_row, part = blockIdx.x % blocks_of_row;
    const int64_t b = row / p.kv_heads;
    int64_t n = p.seq_lens[b];
    if (n < 0 || n > p.table_tokens) n = n < 0 ? 0 : p.table_tokens;  // as the attention kernel took it
    const int64_t low = p.window > 0 && n > p.window ? n - p.window : 0;
    const float *in = p.scores + row * p.score_tokens;
    float *out = p.scores_out + row * p.score_tokens;
    const float *x = p.logits + row * p.table_tokens * p.group;
    const float2 *top = p.top + row * p.group;  // row · group: the first of the key head's query heads
    const uint64_t policy = l2_policy_evict_first();
    const bool in_place = p.scores == p.scores_out;
    const int64_t from = in_place ? low : 0, to = in_place ? n : p.score_tokens;
    for (int64_t t = from + part * kScoreThreads + threadIdx.x; t < to; t += int64_t(blocks_of_row) * kScoreThreads) {
        const float before = in[t];
        float sum = 0.f;
        if (t >= low && t < n) {
            const float *xt = x + t * p.group;
            if constexpr (kVec) {
                for (int g = 0; g < p.group; g += 4) {
                    const float4 v = load_once(xt + g, policy);
                    const float y[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const float2 r = top[g + i];
                        sum += exp2_fast(y[i] - finite_or_zero(r.x)) * r.y;
                    }
                }
            } else {
                for (int g = 0; g < p.group; ++g) {
                    const float2 r = top[g];
                    sum += exp2_fast(xt[g] - finite_or_zero(r.x)) * r.y;
                }
            }
        }
        out[t] = before + sum;
    }
}

}  // namespace dev
}  // namespace projgb
