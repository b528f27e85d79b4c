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
// memory once and stay in shared memory (kHeld; rows of more than 16384 a CTA
// are read again by every pass), and the passes are loops of little code: unrolled
// over scores held in registers they waited for instructions.  A cluster shares a long
// row and does the same search on the sums of its CTAs' counts, in each of them: of the
// first digit, of which few values occur, a CTA adds its own to everyone's sums; of the
// others everyone reads all counts.
constexpr int kEvictThreads = 512, kEvictWarps = kEvictThreads / 32;
constexpr int kEvictBins = 2048;
constexpr int kEvictSpan = 8192;    // scores of a CTA, where a cluster of at most kEvictCluster gives that
constexpr int kEvictCluster = 8;    // (16, with half the scores each: 61 us instead of 57 for one row of 131071)
constexpr int kEvictRun = 128;      // scores of a warp at a time, four a lane
constexpr int kEvictSlab = 16384;   // scores of a CTA at a time: places within them take 16 bits

__device__ __forceinline__ uint32_t score_key(float s) {
    const uint32_t u = __float_as_uint(s + 0.f);  // −0 becomes 0
    if (s != s) return 0xffffffffu;
    return u & 0x80000000u ? ~u : u | 0x80000000u;
}

// Inclusive sum over the block's threads; `warps`: a word a warp of shared memory.
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
    return x + __reduce_add_sync(0xffffffffu, lane < warp ? warps[lane] : 0u);
}
__device__ __forceinline__ uint4 ld_cluster_u4(uint32_t addr) {
    uint4 v;
    asm volatile("ld.shared::cluster.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(addr));
    return v;
}
__device__ __forceinline__ void add_cluster(uint32_t cluster_addr, uint32_t x) {
    asm volatile("red.relaxed.cluster.shared::cluster.add.u32 [%0], %1;" ::"r"(cluster_addr), "r"(x) : "memory");
}

template <bool kHeld>
__global__ void __launch_bounds__(kEvictThreads) kv_evict_select_kernel(const KvEvictParams p) {
    __shared__ __align__(16) uint32_t bins[3][kEvictBins], sums[kEvictBins];  // of this CTA's keys; of the row's first digits
    __shared__ uint32_t warps[kEvictWarps], found[2], totals[2];
    extern __shared__ __align__(16) float held[];  // this CTA's scores
    griddep_launch_dependents();
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const uint32_t rank = cluster_ctarank(), ranks = cluster_nctarank();
    static_assert(kEvictBins == 4 * kEvictThreads, "four digits a thread");
    for (int i = 0; i < 3; ++i) reinterpret_cast<uint4 *>(bins[i])[tid] = make_uint4(0u, 0u, 0u, 0u);
    reinterpret_cast<uint4 *>(sums)[tid] = make_uint4(0u, 0u, 0u, 0u);
    if (tid < 2) totals[tid] = 0;
    if (ranks > 1) cluster_arrive();  // the sums are clear
    const uint32_t row_of = cluster_id_x(), kv_heads = p.cache.kv_heads;  // sequence · kv_heads + key head
    const int64_t row = row_of, b = row_of / kv_heads;
    griddep_wait();
    const int64_t table_tokens = p.cache.table_width * p.cache.page_size, wide = p.to_width * p.cache.page_size;
    int64_t n = p.seq_lens[b];
    if (n < 0 || n > table_tokens) {
        if (tid == 0) atomicOr(p.status, kKvErrLength);
        n = n < 0 ? 0 : table_tokens;
    }
    const int64_t stay = n < p.keep ? n : p.keep;
    // The last ones (all, where they fit) keep their order; `want` of the first m are chosen.
    const int64_t want = n > p.keep ? p.keep - p.recent : 0, m = n > p.keep ? n - p.recent : 0;
    const int64_t span = ((static_cast<uint32_t>(m) + ranks - 1) / ranks + 3) / 4 * 4;  // (a row's tokens fit 31 bits)
    const int64_t low = span * rank < m ? span * rank : m;
    const int mine = static_cast<int>(low + span < m ? span : m - low);  // scores low, low + 1 ... of this CTA
    const float *row_scores = p.scores + row * p.score_tokens, *in = row_scores + low;
    const bool vec = (reinterpret_cast<uintptr_t>(in) & 15u) == 0;
    if (kHeld && want > 0) {
        const int whole = vec ? mine / 4 : 0;
        for (int i = tid; i < whole; i += kEvictThreads) cp_async16(smem_u32(held + 4 * i), in + 4 * i);
#pragma unroll 4
        for (int i = 4 * whole + tid; i < mine; i += kEvictThreads) held[i] = in[i];
    }
    float *out = p.scores_out + row * wide;
    int32_t *kept = p.kept + row * p.keep;
    const int64_t step = int64_t(ranks) * kEvictThreads, at = int64_t(rank) * kEvictThreads + tid;
    if (rank == 0 && tid == 0 && row_of - static_cast<uint32_t>(b) * kv_heads == 0) p.lens_out[b] = static_cast<int32_t>(stay);
    for (int64_t i = stay + at; i < wide; i += step) out[i] = 0.f;
    for (int64_t i = stay + at; i < p.keep; i += step) kept[i] = -1;
#pragma unroll 4
    for (int64_t i = m + at; i < n; i += step) {
        kept[want + i - m] = static_cast<int32_t>(i);
        out[want + i - m] = row_scores[i];
    }
    if (ranks > 1) cluster_wait();
    if (want == 0) return;  // (every CTA of the cluster)

    // Scores i .. i + 3 of this CTA, i a multiple of four below `mine`; what is at and past `mine` is not used.
    auto four = [&](int i, float(&x)[4]) {
        if (kHeld || (vec && i + 4 <= mine)) {
            const float4 v = kHeld ? *reinterpret_cast<const float4 *>(held + i) : *reinterpret_cast<const float4 *>(in + i);
            x[0] = v.x, x[1] = v.y, x[2] = v.z, x[3] = v.w;
        } else {
#pragma unroll
            for (int j = 0; j < 4; ++j) x[j] = i + j < mine ? in[i + j] : 0.f;
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
    asm volatile("cp.async.wait_all;" ::: "memory");
    __syncthreads();
    uint32_t border = 0, rest = static_cast<uint32_t>(want);
    uint32_t more = 0, level_here = 0;  // this thread's digits' keys of this CTA above the border; at it
#pragma unroll 1
    for (int pass = 0; pass < 3; ++pass) {
        const int shift = pass == 0 ? 21 : pass == 1 ? 10 : 0, known = pass == 1 ? 21 : 10;
        const uint32_t digits = pass == 2 ? 1023u : 2047u;
#pragma unroll 2
        for (int i = 4 * tid; i < mine; i += 4 * kEvictThreads) {
            float x[4];
            four(i, x);
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const uint32_t key = score_key(x[j]);
                if (i + j < mine && (pass == 0 || key >> known == border)) atomicAdd(&bins[pass][(key >> shift) & digits], 1u);
            }
        }
        __syncthreads();
        // Four digits a thread, the highest first.
        const uint32_t d0 = kEvictBins - 4 - 4 * tid;
        const uint4 local = *reinterpret_cast<const uint4 *>(&bins[pass][d0]);
        uint4 c = local;
        if (ranks > 1) {
            if (pass == 0) {
                const uint32_t has[4] = {local.x, local.y, local.z, local.w};
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    if (has[j])
                        for (uint32_t r = 0; r < ranks; ++r) add_cluster(map_to_rank(smem_u32(&sums[d0 + j]), r), has[j]);
                all_here();
                c = *reinterpret_cast<const uint4 *>(sums + d0);
            } else {
                all_here();
                uint4 other[kEvictCluster - 1];  // (asked for together)
#pragma unroll
                for (uint32_t o = 1; o < kEvictCluster; ++o) {
                    other[o - 1] = make_uint4(0u, 0u, 0u, 0u);
                    if (o < ranks) other[o - 1] = ld_cluster_u4(map_to_rank(smem_u32(&bins[pass][d0]), rank + o < ranks ? rank + o : rank + o - ranks));
                }
#pragma unroll
                for (int o = 0; o < kEvictCluster - 1; ++o) c.x += other[o].x, c.y += other[o].y, c.z += other[o].z, c.w += other[o].w;
            }
        }
        const uint32_t all = c.x + c.y + c.z + c.w;
        uint32_t before = block_scan(all, warps) - all;
        const uint32_t counts[4] = {c.w, c.z, c.y, c.x}, here[4] = {local.w, local.z, local.y, local.x};
        level_here = 0;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            if (before + counts[j] < rest) more += here[j];
            if (before < rest && rest <= before + counts[j]) {
                found[0] = d0 + 3 - j;
                found[1] = rest - before;
                level_here = here[j];
            }
            before += counts[j];
        }
        __syncthreads();
        border = pass == 0 ? found[0] : (border << (pass == 2 ? 10 : 11)) | found[0];
        rest = found[1];
    }

    // A slab's scores from `base` on, a warp's `runs` · kEvictRun of them in a row.
    auto runs_of = [&](int base) {
        const int left = mine - base < kEvictSlab ? mine - base : kEvictSlab;
        return (left + kEvictWarps * kEvictRun - 1) / (kEvictWarps * kEvictRun);
    };
    // Kept places and scores of a run, together: over the first two digits' counts, which the
    // other CTAs have read by the last one's.
    uint2 *stage = reinterpret_cast<uint2 *>(bins[0]) + warp * kEvictRun;
    static_assert(kEvictWarps * kEvictRun * sizeof(uint2) <= 2 * sizeof(bins[0]), "room");
    // (keys above the border << 16) + (keys at it), of four.
    auto weigh = [&](int i, const float(&x)[4]) {
        uint32_t sum = 0;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const uint32_t key = score_key(x[j]);
            if (i + j < mine) sum += key > border ? 0x10000u : key == border ? 1u : 0u;
        }
        return sum;
    };
    uint32_t above = 0, equal = 0;  // before the slab, first of the CTAs before this one
    if (ranks > 1) {
        const uint32_t a = __reduce_add_sync(0xffffffffu, more), e = __reduce_add_sync(0xffffffffu, level_here);
        if (lane == 0) {
            for (uint32_t r = rank + 1; r < ranks; ++r) {
                if (a) add_cluster(map_to_rank(smem_u32(&totals[0]), r), a);
                if (e) add_cluster(map_to_rank(smem_u32(&totals[1]), r), e);
            }
        }
        all_here();  // (and no CTA adds to another's memory after this)
        above = totals[0], equal = totals[1];
    }
#pragma unroll 1
    for (int base = 0; base < mine; base += kEvictSlab) {
        const int runs = runs_of(base);
        uint32_t of_warp = 0;
#pragma unroll 2
        for (int k = 0; k < runs; ++k) {
            const int i = base + (warp * runs + k) * kEvictRun + lane * 4;
            float x[4];
            if (i < mine) {
                four(i, x);
                of_warp += weigh(i, x);
            }
        }
        of_warp = __reduce_add_sync(0xffffffffu, of_warp);
        __syncthreads();
        if (lane == 0) warps[warp] = of_warp;
        __syncthreads();
        const uint32_t theirs = lane < kEvictWarps ? warps[lane] : 0u;
        const uint32_t earlier = __reduce_add_sync(0xffffffffu, lane < warp ? theirs : 0u);
        const uint32_t slab = __reduce_add_sync(0xffffffffu, theirs);
        uint32_t a0 = above + (earlier >> 16), e0 = equal + (earlier & 0xffffu);  // before the run
#pragma unroll 1
        for (int k = 0; k < runs; ++k) {
            const int i = base + (warp * runs + k) * kEvictRun + lane * 4;
            float x[4] = {0.f, 0.f, 0.f, 0.f};
            if (i < mine) four(i, x);
            const uint32_t sum = weigh(i, x);
            uint32_t upto = sum;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const uint32_t other = __shfl_up_sync(0xffffffffu, upto, o);
                if (lane >= o) upto += other;
            }
            uint32_t a = a0 + ((upto - sum) >> 16), e = e0 + ((upto - sum) & 0xffffu);
            // The kept ones are next to each other: gathered in shared memory, and then written
            // in whole rows of the warp (stores of the few of each lane took half the time).
            const uint32_t begin = a0 + (e0 < rest ? e0 : rest);
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const uint32_t key = score_key(x[j]);
                const bool there = i + j < mine, up = there && key > border, level = there && key == border;
                if (up || (level && e < rest))
                    stage[a + (e < rest ? e : rest) - begin] = make_uint2(static_cast<uint32_t>(low) + i + j, __float_as_uint(x[j]));
                a += up, e += level;
            }
            const uint32_t run = __shfl_sync(0xffffffffu, upto, 31);
            a0 += run >> 16, e0 += run & 0xffffu;
            __syncwarp();
            for (uint32_t o = lane; o < a0 + (e0 < rest ? e0 : rest) - begin; o += 32) {
                const uint2 v = stage[o];
                kept[begin + o] = static_cast<int32_t>(v.x);
                out[begin + o] = __uint_as_float(v.y);
            }
            __syncwarp();
        }
        above += slab >> 16, equal += slab & 0xffffu;
    }
}

// The copy.  A block first looks up where up to 256 kept tokens lie and go, a thread
// each, and then copies 16 bytes of a token's key and value a thread, four tokens at a
// time so that eight loads are on their way.  Bytes bound it: each kept row is read
// and written once.  (With the lookups in the copying threads, three loads one after
// another before every four tokens, 32 sequences took 86 us at 62 % of the DRAM rate.)
constexpr int kEvictCopyThreads = 256;
constexpr int kEvictAhead = 4;

__global__ void __launch_bounds__(kEvictCopyThreads) kv_evict_copy_kernel(const KvEvictParams p, const int blocks_of_row, const int tokens) {
    __shared__ int64_t from_of[kEvictCopyThreads], to_of[kEvictCopyThreads];  // bytes, of the token's row; −1: not copied
    griddep_launch_dependents();
    const KvCacheView &c = p.cache;
    const uint32_t row_of = blockIdx.x / static_cast<uint32_t>(blocks_of_row), kv_heads = c.kv_heads;
    const int64_t row = row_of, part = blockIdx.x % static_cast<uint32_t>(blocks_of_row);
    const int64_t b = row_of / kv_heads, head = row_of % kv_heads;
    const int chunks = c.head_dim * p.elem / 16, pass = kEvictCopyThreads / chunks;  // tokens of a pass of the block
    const int chunk = threadIdx.x % chunks, first = threadIdx.x / chunks;
    const uint32_t page_size = static_cast<uint32_t>(c.page_size);
    uint8_t *k = static_cast<uint8_t *>(p.k_cache) + chunk * 16, *v = static_cast<uint8_t *>(p.v_cache) + chunk * 16;
    griddep_wait();
    const int64_t stay = p.lens_out[b];
    const int32_t *kept = p.kept + row * p.keep;
    auto offset = [&](const int32_t *table, uint32_t token) -> int64_t {
        const uint32_t page = token / page_size;
        const int64_t at = table[page];
        if (at < 0 || at >= c.num_pages) {
            atomicOr(p.status, kKvErrPage);
            return -1;
        }
        return (at * c.page_stride + (token - page * page_size) * c.token_stride + head * c.head_stride) * p.elem;
    };
    for (int64_t base = part * tokens; base < stay; base += int64_t(blocks_of_row) * tokens) {
        const int count = stay - base < tokens ? static_cast<int>(stay - base) : tokens;
        __syncthreads();  // the places of the round before are read
        if (static_cast<int>(threadIdx.x) < count) {
            const int64_t o = base + threadIdx.x;
            const int64_t to = offset(p.to_table + b * p.to_width, static_cast<uint32_t>(o));
            const int64_t from = offset(c.table + b * c.table_width, static_cast<uint32_t>(kept[o]));
            from_of[threadIdx.x] = to < 0 ? -1 : from;
            to_of[threadIdx.x] = to;
        }
        __syncthreads();
        if (first >= pass) continue;  // (threads past the last whole token of a pass)
        for (int o = first; o < count; o += pass * kEvictAhead) {
            int64_t from[kEvictAhead];
            uint4 kx[kEvictAhead], vx[kEvictAhead];
#pragma unroll
            for (int i = 0; i < kEvictAhead; ++i) {
                from[i] = o + i * pass < count ? from_of[o + i * pass] : -1;
                if (from[i] < 0) continue;
                kx[i] = *reinterpret_cast<const uint4 *>(k + from[i]);
                vx[i] = *reinterpret_cast<const uint4 *>(v + from[i]);
            }
#pragma unroll
            for (int i = 0; i < kEvictAhead; ++i) {
                if (from[i] < 0) continue;
                const int64_t to = to_of[o + i * pass];
                *reinterpret_cast<uint4 *>(k + to) = kx[i];
                *reinterpret_cast<uint4 *>(v + to) = vx[i];
            }
        }
    }
}

}  // namespace dev
}  // namespace projgb
