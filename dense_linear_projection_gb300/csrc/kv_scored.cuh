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

// kGroup: query heads of a key head where these are a multiple of four up to 16: the maxima and sums stay
// in registers, the logits come in fours, of kScoreAhead tokens together.  (64 ragged sequences to 8192, 8
// key heads, whole call: 16 heads 275 us, 312 as below; over 8 bits, 4 key heads, 129 and 147; 12 heads of
// 4 key heads 135.5 and 142.5; 8 heads 20.6 us for 100 MB.)  0: other numbers, a token and a head at a
// time (1: 182, 2: 184, 3: 189, 6: 200, 7: 204; 1 and 2 in the way of the fours 178 and 180).
template <int kGroup>
constexpr int kScoreAhead = kGroup == 0 ? 1 : kGroup <= 8 ? 4 : 2;  // tokens

template <int kGroup>
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
    const int64_t step = int64_t(blocks_of_row) * kScoreThreads;
    auto weight = [&](float y, float2 r) { return exp2_fast(y - finite_or_zero(r.x)) * r.y; };
    if constexpr (kGroup > 0) {
        constexpr int kAhead = kScoreAhead<kGroup>;
        float2 held[kGroup];
#pragma unroll
        for (int g = 0; g < kGroup; ++g) held[g] = top[g];
        for (int64_t t0 = from + part * kScoreThreads + threadIdx.x; t0 < to; t0 += kAhead * step) {
            float before[kAhead];
            float4 v[kAhead][kGroup / 4];
#pragma unroll
            for (int k = 0; k < kAhead; ++k) {
                const int64_t t = t0 + k * step;
                before[k] = t < to ? in[t] : 0.f;
#pragma unroll
                for (int g = 0; g < kGroup / 4; ++g)
                    v[k][g] = t >= low && t < n ? load_once(x + t * kGroup + 4 * g, policy) : make_float4(-INFINITY, -INFINITY, -INFINITY, -INFINITY);
            }
#pragma unroll
            for (int k = 0; k < kAhead; ++k) {
                const int64_t t = t0 + k * step;
                if (t >= to) break;
                float sum = 0.f;
                if (t >= low && t < n) {
#pragma unroll
                    for (int g = 0; g < kGroup / 4; ++g)
                        sum += weight(v[k][g].x, held[4 * g]) + weight(v[k][g].y, held[4 * g + 1]) + weight(v[k][g].z, held[4 * g + 2]) +
                               weight(v[k][g].w, held[4 * g + 3]);
                }
                out[t] = before[k] + sum;
            }
        }
    } else {
        for (int64_t t = from + part * kScoreThreads + threadIdx.x; t < to; t += step) {
            float sum = 0.f;
            if (t >= low && t < n)
                for (int g = 0; g < p.group; ++g) sum += weight(x[t * p.group + g], top[g]);
            out[t] = in[t] + sum;
        }
    }
}

}  // namespace dev
}  // namespace projgb
