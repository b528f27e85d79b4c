// Device code of eviction from the paged key-value cache: which tokens of a
// sequence and key head stay, and their copy to other pages.
#pragma once

#include "kv_internal.h"
#include "proj_kernel.cuh"
#include "proj_warp.cuh"

namespace projgb {
namespace dev {

// Selection.  Of n > keep tokens the last `recent` stay, and of the m = n − recent
// before them the want = keep − recent of the highest scores, equal scores by their
// place; all in their order.  Scores are compared as 32-bit keys of the same order
// (−0 as 0, NaN above all).  Three passes over the keys' digits of 11, 11 and 10
// bits count each digit's keys and narrow down to the one key `border` of which
// some are taken: a token's place among the kept ones is then
//   (keys above the border before it) + min(keys at the border before it, rest).
//
// What bounds it: the few short passes, one after another.  The scores come from
// memory once and stay in registers (kHeld; longer rows are read again by every
// pass).  A cluster shares a long row, its counts meet in distributed shared memory,
// and every CTA of it does the same search on the sums.
constexpr int kEvictThreads = 1024;
constexpr int kEvictBins = 2048;
constexpr int kEvictSpan = 8192;    // scores of a CTA, where a cluster of at most kEvictCluster gives that
constexpr int kEvictCluster = 8;
constexpr int kEvictPer = 4;        // consecutive scores of a thread: its places are counted over these
constexpr int kEvictSlab = kEvictThreads * kEvictPer;
constexpr int kEvictHeld = 4;       // slabs in registers

__device__ __forceinline__ uint32_t score_key(float s) {
    const uint32_t u = __float_as_uint(s + 0.f);  // −0 becomes 0
    if (s != s) return 0xffffffffu;
    return u & 0x80000000u ? ~u : u | 0x80000000u;
}

// Inclusive sum over the block's threads; `warps`: 32 words of shared memory.
__device__ __forceinline__ uint32_t block_scan(uint32_t x, uint32_t *warps) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const uint32_t other = __shfl_up_sync(0xffffffffu, x, o);
        if (lane >= o) x += other;
    }
    __syncthreads();  // the words are free
    if (lane == 31) warps[warp] = x;
    __syncthreads();
    uint32_t before = lane < warp ? warps[lane] : 0u;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) before += __shfl_xor_sync(0xffffffffu, before, o);
    return x + before;
}

template <bool kHeld>
__global__ void __launch_bounds__(kEvictThreads) kv_evict_select_kernel(const KvEvictParams p) {
    __shared__ uint32_t bins[3][kEvictBins];
    __shared__ uint32_t warps[32], found[2], counts[2];
    griddep_launch_dependents();
    const int tid = threadIdx.x;
    const uint32_t rank = cluster_ctarank(), ranks = cluster_nctarank();
    for (int i = tid; i < 3 * kEvictBins; i += kEvictThreads) (&bins[0][0])[i] = 0;
    if (tid < 2) counts[tid] = 0;
    griddep_wait();
    const int64_t row = cluster_id_x();  // sequence · kv_heads + key head
    const int64_t b = row / p.cache.kv_heads;
    const int64_t table_tokens = p.cache.table_width * p.cache.page_size, wide = p.to_width * p.cache.page_size;
    int64_t n = p.seq_lens[b];
    if (n < 0 || n > table_tokens) {
        if (tid == 0) atomicOr(p.status, kKvErrLength);
        n = n < 0 ? 0 : table_tokens;
    }
    const int64_t stay = n < p.keep ? n : p.keep;
    // The last ones (all, where they fit) keep their order; `want` of the first m are chosen.
    const int64_t want = n > p.keep ? p.keep - p.recent : 0, m = n > p.keep ? n - p.recent : 0;
    const int64_t span = ((m + ranks - 1) / ranks + kEvictPer - 1) / kEvictPer * kEvictPer;
    const int64_t low = span * rank < m ? span * rank : m, high = low + span < m ? low + span : m;
    const float *in = p.scores + row * p.score_tokens;
    float held[kHeld ? kEvictHeld : 1][kEvictPer];
    if (kHeld && want > 0) {
#pragma unroll
        for (int k = 0; k < kEvictHeld; ++k)
#pragma unroll
            for (int j = 0; j < kEvictPer; ++j) {
                const int64_t i = low + k * kEvictSlab + tid * kEvictPer + j;
                held[k][j] = i < high ? in[i] : 0.f;
            }
    }
    float *out = p.scores_out + row * wide;
    int32_t *kept = p.kept + row * p.keep;
    const int64_t step = int64_t(ranks) * kEvictThreads, mine = int64_t(rank) * kEvictThreads + tid;
    if (rank == 0 && tid == 0 && row % p.cache.kv_heads == 0) p.lens_out[b] = static_cast<int32_t>(stay);
    for (int64_t i = stay + mine; i < wide; i += step) out[i] = 0.f;
    for (int64_t i = stay + mine; i < p.keep; i += step) kept[i] = -1;
    for (int64_t i = m + mine; i < n; i += step) {
        kept[want + i - m] = static_cast<int32_t>(i);
        out[want + i - m] = in[i];
    }
    if (want == 0) return;  // (every CTA of the cluster)

    // f(first place, scores) for each of this thread's runs of kEvictPer scores; every thread of
    // the block comes to each, with places at or past `high` where it has none.
    auto each_run = [&](auto f) {
        if constexpr (kHeld) {
#pragma unroll
            for (int k = 0; k < kEvictHeld; ++k)
                if (low + k * kEvictSlab < high) f(low + k * kEvictSlab + tid * kEvictPer, held[k]);
        } else {
            for (int64_t base = low; base < high; base += kEvictSlab) {
                float s[kEvictPer];
#pragma unroll
                for (int j = 0; j < kEvictPer; ++j) s[j] = base + tid * kEvictPer + j < high ? in[base + tid * kEvictPer + j] : 0.f;
                f(base + tid * kEvictPer, s);
            }
        }
    };
    // The whole row's CTAs have come here.
    auto all_here = [&]() {
        if (ranks > 1) {
            cluster_arrive();
            cluster_wait();
        } else {
            __syncthreads();
        }
    };
    __syncthreads();
    uint32_t border = 0, rest = static_cast<uint32_t>(want);
#pragma unroll
    for (int pass = 0; pass < 3; ++pass) {
        const int shift = pass == 0 ? 21 : pass == 1 ? 10 : 0;
        const uint32_t digits = pass == 2 ? 1023u : 2047u;
        each_run([&](int64_t i0, const float(&s)[kEvictPer]) {
#pragma unroll
            for (int j = 0; j < kEvictPer; ++j) {
                const uint32_t key = score_key(s[j]);
                const bool counted = i0 + j < high && (pass == 0 || (key >> (shift + (pass == 2 ? 10 : 11))) == border);
                const uint32_t digit = (key >> shift) & digits;
                // One addition for a warp whose digits are all alike (scores that are all zero).
                const uint32_t who = __ballot_sync(0xffffffffu, counted);
                if (who == 0) continue;
                const int lead = __ffs(who) - 1;
                const uint32_t first = __shfl_sync(0xffffffffu, digit, lead);
                if (__all_sync(0xffffffffu, !counted || digit == first)) {
                    if ((tid & 31) == lead) atomicAdd(&bins[pass][first], __popc(who));
                } else if (counted) {
                    atomicAdd(&bins[pass][digit], 1u);
                }
            }
        });
        all_here();
        // Two digits a thread, the highest first, over all CTAs of the cluster.
        const uint32_t d1 = kEvictBins - 1 - 2 * tid, d0 = d1 - 1;
        uint32_t c1 = bins[pass][d1], c0 = bins[pass][d0];
        for (uint32_t o = 1; o < ranks; ++o) {
            const uint32_t at = map_to_rank(smem_u32(&bins[pass][0]), rank + o < ranks ? rank + o : rank + o - ranks);
            c1 += ld_cluster_u32(at + d1 * 4);
            c0 += ld_cluster_u32(at + d0 * 4);
        }
        const uint32_t upto = block_scan(c1 + c0, warps), before = upto - c1 - c0;
        if (before < rest && rest <= upto) {
            const bool upper = rest <= before + c1;
            found[0] = upper ? d1 : d0;
            found[1] = rest - before - (upper ? 0 : c1);
        }
        __syncthreads();
        border = pass == 0 ? found[0] : (border << (pass == 2 ? 10 : 11)) | found[0];
        rest = found[1];
    }

    // Keys above the border and at it in the CTAs before this one.
    uint32_t above = 0, equal = 0;
    if (ranks > 1) {
        uint32_t a = 0, e = 0;
        each_run([&](int64_t i0, const float(&s)[kEvictPer]) {
#pragma unroll
            for (int j = 0; j < kEvictPer; ++j) {
                const uint32_t key = score_key(s[j]);
                a += i0 + j < high && key > border;
                e += i0 + j < high && key == border;
            }
        });
        a = __reduce_add_sync(0xffffffffu, a), e = __reduce_add_sync(0xffffffffu, e);
        if ((tid & 31) == 0) {
            if (a) atomicAdd(&counts[0], a);
            if (e) atomicAdd(&counts[1], e);
        }
        all_here();
        for (uint32_t r = 0; r < rank; ++r) {
            const uint32_t at = map_to_rank(smem_u32(&counts[0]), r);
            above += ld_cluster_u32(at);
            equal += ld_cluster_u32(at + 4);
        }
        cluster_arrive();  // no CTA leaves while another reads its counts
    }
    each_run([&](int64_t i0, const float(&s)[kEvictPer]) {
        uint32_t key[kEvictPer], mine_of = 0;  // (above << 16) + equal: kEvictSlab at most of each
#pragma unroll
        for (int j = 0; j < kEvictPer; ++j) {
            key[j] = score_key(s[j]);
            if (i0 + j < high) mine_of += key[j] > border ? 0x10000u : key[j] == border ? 1u : 0u;
        }
        const uint32_t upto = block_scan(mine_of, warps);
        uint32_t a = above + ((upto - mine_of) >> 16), e = equal + ((upto - mine_of) & 0xffffu);
#pragma unroll
        for (int j = 0; j < kEvictPer; ++j) {
            if (i0 + j >= high) break;
            const bool up = key[j] > border, at = key[j] == border;
            if (up || (at && e < rest)) {
                const int64_t to = static_cast<int64_t>(a) + (e < rest ? e : rest);
                kept[to] = static_cast<int32_t>(i0 + j);
                out[to] = s[j];
            }
            a += up, e += at;
        }
        if (tid == kEvictThreads - 1) found[0] = upto;
        __syncthreads();
        above += found[0] >> 16, equal += found[0] & 0xffffu;
    });
    if (ranks > 1) cluster_wait();
}

// The copy: 16 bytes of a token's key and value a thread, four tokens at a time so
// that eight loads are on their way.  Bytes bound it: each kept row is read and
// written once.
constexpr int kEvictCopyThreads = 256;
constexpr int kEvictAhead = 4;

__global__ void __launch_bounds__(kEvictCopyThreads) kv_evict_copy_kernel(const KvEvictParams p, const int blocks_of_row) {
    griddep_launch_dependents();
    griddep_wait();
    const KvCacheView &c = p.cache;
    const int64_t row = blockIdx.x / blocks_of_row, part = blockIdx.x % blocks_of_row;
    const int64_t b = row / c.kv_heads, head = row % c.kv_heads;
    const int stay = p.lens_out[b];
    const int chunks = c.head_dim * p.elem / 16, tokens = kEvictCopyThreads / chunks;  // of a block at a time
    const int chunk = threadIdx.x % chunks, first = threadIdx.x / chunks;
    if (first >= tokens) return;
    const int32_t *kept = p.kept + row * p.keep;
    const int32_t *from_table = c.table + b * c.table_width, *to_table = p.to_table + b * p.to_width;
    const uint32_t page_size = static_cast<uint32_t>(c.page_size);
    auto offset = [&](const int32_t *table, uint32_t token) -> int64_t {  // in bytes, −1 for a bad page
        const uint32_t page = token / page_size;
        const int64_t at = table[page];
        if (at < 0 || at >= c.num_pages) {
            atomicOr(p.status, kKvErrPage);
            return -1;
        }
        return (at * c.page_stride + (token - page * page_size) * c.token_stride + head * c.head_stride) * p.elem + chunk * 16;
    };
    uint8_t *k = static_cast<uint8_t *>(p.k_cache), *v = static_cast<uint8_t *>(p.v_cache);
    for (int64_t base = int64_t(part) * tokens * kEvictAhead + first; base < stay; base += int64_t(blocks_of_row) * tokens * kEvictAhead) {
        int64_t from[kEvictAhead], to[kEvictAhead];
        uint4 kx[kEvictAhead], vx[kEvictAhead];
#pragma unroll
        for (int i = 0; i < kEvictAhead; ++i) {
            const int64_t o = base + i * tokens;
            from[i] = o < stay ? kept[o] : -1;
        }
#pragma unroll
        for (int i = 0; i < kEvictAhead; ++i) {
            if (from[i] < 0) continue;
            to[i] = offset(to_table, static_cast<uint32_t>(base + i * tokens));
            from[i] = offset(from_table, static_cast<uint32_t>(from[i]));
            if (to[i] < 0) from[i] = -1;
        }
#pragma unroll
        for (int i = 0; i < kEvictAhead; ++i) {
            if (from[i] < 0) continue;
            kx[i] = *reinterpret_cast<const uint4 *>(k + from[i]);
            vx[i] = *reinterpret_cast<const uint4 *>(v + from[i]);
        }
#pragma unroll
        for (int i = 0; i < kEvictAhead; ++i) {
            if (from[i] < 0) continue;
            *reinterpret_cast<uint4 *>(k + to[i]) = kx[i];
            *reinterpret_cast<uint4 *>(v + to[i]) = vx[i];
        }
    }
}

}  // namespace dev
}  // namespace projgb
