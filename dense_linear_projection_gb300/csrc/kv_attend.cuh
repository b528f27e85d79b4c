// Device code of attention of one new token of each sequence over the paged
// key-value cache.
//
// Mathematics.  For one sequence and one key head, the G query heads that share
// it, and tokens t: x[t,h] = scale·log2(e)·q[h]·k[t];  with a running maximum m,
// l = Σ 2^(x − m) and o = Σ 2^(x − m)·v[t].  Two parts (m, l, o), (m', l', o')
// join with M = max(m, m'): l·2^(m − M) + l'·2^(m' − M), and o likewise; out =
// o / l, lse = ln 2·(M + log2 l).
//
// What bounds it: the bytes of K and V, each read once for all G heads.  So
//   * a warp works alone on 16 or 32 tokens at a time, with a ring of shared-memory
//     stages of its own filled by 16-byte asynchronous copies, and waits for no
//     other warp until its row ends;
//   * both products are swapped: X[tokens, heads] = K·Qᵀ and Oᵀ[dim, heads] =
//     Vᵀ·P, so K and V are the 16-row operand of the tensor-core step and the
//     heads its 8 columns: a group of up to 8 heads costs one step per 16 tokens
//     × 16 elements, and a wider group a second one on the same operand.
//   * the tokens of all sequences and key heads, in tiles of a CTA's step, form one
//     line that the CTAs share evenly: CTA c takes places [c·T/C, (c+1)·T/C).  A
//     row that several CTAs share is joined by the one that arrives last, in CTA
//     order, from fp32 partial results in scratch.
//
// Precision: fp32 logits, weights and sums.  The weights enter the second
// product as 16-bit parts that hold them as fp32 does (split): three of bf16, or
// over e4m3 two of fp16, to 2^-23 of a weight or 2^-52 of the largest.  An e4m3
// cache is converted to fp16 (exact); the queries then are fp16 too, scaled by a
// power of two per head: elements down to 2^-32 of the head's largest are exact,
// smaller ones are held to 2^-40 of it (a logit's fp32 sum holds no more beside
// the largest).
#pragma once

#include <cuda_fp16.h>

#include "kv_internal.h"
#include "proj_kernel.cuh"
#include "proj_warp.cuh"

namespace projgb {
namespace dev {

template <bool kE4m3, int kDim, int kNT, int kKeyHeads>
struct AttendShape {
    static constexpr int kElem = kE4m3 ? 1 : 2;
    static constexpr int kRow = kDim * kElem;         // bytes of a token's row in a stage
    static constexpr int kChunks = kRow / 16;         // 16-byte chunks of a row
    // Token blocks of 16 a step: two where a row is short, so that a step is
    // 8 KiB or more and its two chains of tensor-core steps and shuffles overlap
    // (an 8-bit cache of 128-wide heads ran at 66 % of the copy bandwidth with one).
    static constexpr int kBlocks = kRow <= 128 ? 2 : 1;
    static constexpr int kStep = 16 * kBlocks;        // tokens of a warp's step
    // A CTA's row is one key head with its warps on consecutive steps, or two key
    // heads with two warps each.
    static constexpr int kLanes = kKvWarps / kKeyHeads;
    static constexpr int kTile = kLanes * kStep;      // unit of the work shared between CTAs
    static constexpr int kStage = 2 * kStep * kRow;   // keys, then values
    static constexpr int kHeads = 8 * kNT;             // query heads of a warp
    static constexpr int kRowHeads = kHeads * kKeyHeads;
    static constexpr int kJoin = kKvWarps * kHeads * (kDim + 4) * 4;  // the warps' sums, fp32
    static constexpr int kSmall = kKvWarps * kHeads * 8 + 64;   // their maxima and sums of weights; flags
    // Two CTAs an SM (one for 256-wide heads): while one joins its warps, the
    // other streams.
    static constexpr int kPerSm = kDim > 128 ? 1 : 2;
    static constexpr int kBudget = (kPerSm == 2 ? 113 : 226) * 1024 - kJoin - kSmall;
    static constexpr int kFit = kBudget / (kKvWarps * kStage);
    static constexpr int kStages = kFit > 8 ? 8 : kFit;
    static constexpr int kSmem = kKvWarps * kStages * kStage + kJoin + kSmall;
    static_assert(kStages >= 2, "a stage to read and one to fill");
};

__device__ __forceinline__ uint32_t e4m3x2_to_half2(uint32_t two) {
    uint32_t h;
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"(static_cast<uint16_t>(two)));
    return h;
}
__device__ __forceinline__ float exp2_fast(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// fp16 has no exponent below -24, so the weights (1 at most) are taken 2^15 times
// as large, and what their high parts leave 2^12 times as large again, next to
// values 2^12 times smaller (e4m3 times 2^-12 is exact in fp16): a weight loses
// 2^-23 of itself or 2^-52, whichever is more.  (131071 tokens of 25 nats below one
// whose value is zero are still all of the output.)
constexpr float kHalfWeight = 32768.f, kHalfWeightBack = 1.f / 32768.f, kHalfRest = 4096.f;
constexpr uint32_t kHalfRestBack = 0x0C000C00u;  // 2^-12, twice

__device__ __forceinline__ uint32_t half2_mul(uint32_t a, uint32_t b) {
    uint32_t d;
    asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
    return d;
}

// Two weights as 16-bit parts, each of what the parts before it leave: three of
// bf16 (24 bits) or two of fp16 (22).  Measured against two bf16 parts: one sequence
// of 131071 tokens 92.0 us instead of 91.4, 64 ragged ones 161.8 and 162.0; against
// fp16 parts of unscaled weights: 16 ragged sequences in 8 bits 94 instead of 92.
template <bool kHalf>
struct WeightParts {
    static constexpr int kCount = kHalf ? 2 : 3;
    uint32_t part[kCount];
};
template <bool kHalf>
__device__ __forceinline__ WeightParts<kHalf> split(float a, float b) {
    WeightParts<kHalf> s;
    if constexpr (kHalf) {
        a *= kHalfWeight, b *= kHalfWeight;
        const __half2 h = __floats2half2_rn(a, b);
        const float2 f = __half22float2(h);
        const __half2 r = __floats2half2_rn((a - f.x) * kHalfRest, (b - f.y) * kHalfRest);
        s.part[0] = *reinterpret_cast<const uint32_t *>(&h);
        s.part[1] = *reinterpret_cast<const uint32_t *>(&r);
    } else {
        // A part is the upper half of the next float below, so that every part of
        // a positive weight is positive: an infinite value times 0, or times parts
        // of both signs, would be NaN.
        constexpr float kBelow = 0x1.fffffep-1f;
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const uint32_t ha = __float_as_uint(__fmul_rz(a, kBelow)), hb = __float_as_uint(__fmul_rz(b, kBelow));
            s.part[i] = __byte_perm(ha, hb, 0x7632);
            a -= __uint_as_float(ha & 0xffff0000u), b -= __uint_as_float(hb & 0xffff0000u);
        }
        s.part[2] = bf16_pair(a, b);
    }
    return s;
}

// Byte offset of chunk c of row r in an operand of a stage: the chunks of
// eight consecutive rows at one column fall in eight different 16-byte banks.
template <int kRow>
__device__ __forceinline__ uint32_t chunk_at(int r, int c) {
    if constexpr (kRow >= 128) return r * kRow + ((c ^ (r & 7)) << 4);
    return r * kRow + ((c ^ ((r >> 1) & 3)) << 4);  // 64-byte rows, two to a 128-byte line
}

// a·b / c and a / b for b < 512 and c < 512 in the first: 32-bit where they fit
// (a 64-bit division takes about 0.1 us, at the start of every row).
__device__ __forceinline__ int64_t share_of(int64_t a, uint32_t b, uint32_t c) {
    if (a < (int64_t(1) << 23)) return static_cast<uint32_t>(a) * b / c;
    return a * b / c;
}
__device__ __forceinline__ int64_t divide(int64_t a, int64_t b) {
    if (((a | b) >> 32) == 0) return static_cast<uint32_t>(a) / static_cast<uint32_t>(b);
    return a / b;
}

// A place on the line of work: sequence b, whose rows (one for each of the
// `units`: key head, chunk of query heads) begin at `base`.  A row is kKvRowCost
// places for its start and its join, which take about as long as a tile, and
// then a place for each of its `tiles`.
struct AttendCursor {
    int64_t base = 0, tiles = 0, span = 0;
    int b = 0;
    int low = 0, n = 0;  // the tokens attended are [low, n)
};

struct AttendSegment {
    int unit, first, last;  // tokens [first, last) of the cursor's sequence; last <= n
    int64_t row_begin;      // the row's first place on the line
    int64_t places;         // the segment's length on the line
    int64_t tiles;          // of the segment: 0 where it holds only the row's start
};

template <typename Shape>
__device__ __forceinline__ void read_length(const KvAttendParams &p, int b, AttendCursor &c) {
    const int64_t most = p.cache.table_width * p.cache.page_size;
    int n = p.seq_lens[b];
    if (n < 0 || n > most) {
        atomicOr(p.status, kKvErrLength);
        n = n < 0 ? 0 : static_cast<int>(most);
    }
    c.n = n;
    c.low = p.window > 0 && n > p.window ? n - static_cast<int>(p.window) : 0;
    c.tiles = (n - (c.low & ~(Shape::kStep - 1)) + Shape::kTile - 1) / Shape::kTile;
    c.span = c.tiles > 0 ? c.tiles + kKvRowCost : 0;
}

// Moves the cursor to the sequence that holds place `pos` (which exists).
template <typename Shape>
__device__ __forceinline__ void seek(const KvAttendParams &p, AttendCursor &c, int64_t pos) {
    while (pos >= c.base + c.span * p.units) {
        c.base += c.span * p.units;
        ++c.b;
        read_length<Shape>(p, c.b, c);
    }
}

// The part of places [pos, end) that lies in pos's row.
template <typename Shape>
__device__ __forceinline__ AttendSegment segment_at(const AttendCursor &c, int64_t pos, int64_t end) {
    constexpr int kTile = Shape::kTile;
    AttendSegment s;
    s.unit = static_cast<int>(divide(pos - c.base, c.span));
    s.row_begin = c.base + s.unit * c.span;
    const int64_t from = pos - s.row_begin, to = end - s.row_begin < c.span ? end - s.row_begin : c.span;
    const int64_t k0 = from > kKvRowCost ? from - kKvRowCost : 0, k1 = to > kKvRowCost ? to - kKvRowCost : 0;
    const int start = c.low & ~(Shape::kStep - 1);
    s.first = start + static_cast<int>(k0) * kTile;
    s.last = k1 == c.tiles ? c.n : start + static_cast<int>(k1) * kTile;
    s.places = to - from;
    s.tiles = k1 - k0;
    return s;
}

// What a thread holds of a row while it is joined: four elements of kPer heads.
template <int kHeads, int kDim>
struct JoinPart {
    static constexpr int kLanes = kDim / 4;                      // threads of a head
    static constexpr int kHeadStep = kKvThreads / kLanes;        // heads at a time
    static constexpr int kPer = kHeads / kHeadStep;
    static constexpr int kPitch = kDim + 4;                      // of a head in the warps' sums: conflict-free
    static constexpr int kFloats = kHeads * (kDim + 2);          // of a partial result: maxima, sums of weights, [head][dim]
    static_assert(kPer >= 1, "every thread has an element");
    float m[kPer], l[kPer];
    float4 o[kPer];

    __device__ __forceinline__ void clear() {
#pragma unroll
        for (int k = 0; k < kPer; ++k) {
            m[k] = -INFINITY;
            l[k] = 0.f;
            o[k] = make_float4(0.f, 0.f, 0.f, 0.f);
        }
    }
};

__device__ __forceinline__ float finite_or_zero(float top) { return top == -INFINITY ? 0.f : top; }

// One part, of maximum m, against the joint maximum: in the same operations
// wherever a part is joined.
template <int kHeads, int kDim>
__device__ __forceinline__ void add_part(JoinPart<kHeads, kDim> &r, int k, float m, float l, float4 o) {
    const float w = exp2_fast(m - finite_or_zero(r.m[k]));
    r.l[k] = __fmaf_rn(w, l, r.l[k]);
    r.o[k].x = __fmaf_rn(w, o.x, r.o[k].x), r.o[k].y = __fmaf_rn(w, o.y, r.o[k].y);
    r.o[k].z = __fmaf_rn(w, o.z, r.o[k].z), r.o[k].w = __fmaf_rn(w, o.w, r.o[k].w);
}

// Joins the partial results in slots slot(0) .. slot(count - 1), in that order,
// against the maximum of all; the loads of several are in flight at a time.  Heads
// past `heads` are unused.
template <int kHeads, int kDim, typename Slot>
__device__ __forceinline__ void join_parts(const float *partials, int count, Slot slot, int heads, JoinPart<kHeads, kDim> &r) {
    using Part = JoinPart<kHeads, kDim>;
    constexpr int kAtOnce = 8;
    const int h0 = threadIdx.x / Part::kLanes, d = threadIdx.x % Part::kLanes * 4;
    r.clear();
#pragma unroll
    for (int k = 0; k < Part::kPer; ++k) {
        const int h = h0 + k * Part::kHeadStep;
        if (h >= heads) break;
        for (int c = 0; c < count; c += kAtOnce) {
            float m[kAtOnce], l[kAtOnce];
            float4 o[kAtOnce];
#pragma unroll
            for (int i = 0; i < kAtOnce; ++i) {
                const float *from = partials + slot(c + i < count ? c + i : c) * Part::kFloats;
                m[i] = __ldcg(from + h);
                l[i] = __ldcg(from + kHeads + h);
                o[i] = __ldcg(reinterpret_cast<const float4 *>(from + 2 * kHeads + h * kDim + d));
            }
            if (c == 0) {
                for (int x = kAtOnce; x < count; x += kAtOnce)
#pragma unroll
                    for (int i = 0; i < kAtOnce; ++i)
                        r.m[k] = fmaxf(r.m[k], __ldcg(partials + slot(x + i < count ? x + i : x) * Part::kFloats + h));
#pragma unroll
                for (int i = 0; i < kAtOnce; ++i) r.m[k] = fmaxf(r.m[k], m[i]);
            }
#pragma unroll
            for (int i = 0; i < kAtOnce; ++i) {
                if (c + i >= count) break;
                add_part(r, k, m[i], l[i], o[i]);
            }
        }
    }
}

// The same, bit for bit, by way of `ring` (shared memory of `bytes` that no copy is
// under way to): one round trip for as many parts as it holds.
template <int kHeads, int kDim, typename Slot>
__device__ __forceinline__ void join_parts_in(uint8_t *ring, int bytes, const float *partials, int count, Slot slot, int heads,
                                              JoinPart<kHeads, kDim> &r) {
    using Part = JoinPart<kHeads, kDim>;
    const int h0 = threadIdx.x / Part::kLanes, d = threadIdx.x % Part::kLanes * 4;
    const int floats = 2 * kHeads + heads * kDim, at_once = bytes / (floats * 4);  // the heads in use come first
    const uint32_t to = smem_u32(ring);
    r.clear();
    for (int c = 0; c < count; c += at_once) {
        const int n = min(at_once, count - c);
        for (int i = 0; i < n; ++i) {
            const float *from = partials + slot(c + i) * Part::kFloats;
            for (int x = threadIdx.x * 4; x < floats; x += kKvThreads * 4) cp_async16(to + (i * floats + x) * 4, from + x);
        }
        cp_async_commit();
        if (c == 0) {  // the maxima of the parts that the ring does not hold yet
#pragma unroll
            for (int k = 0; k < Part::kPer; ++k) {
                const int h = h0 + k * Part::kHeadStep;
                if (h >= heads) break;
#pragma unroll 4
                for (int i = n; i < count; ++i) r.m[k] = fmaxf(r.m[k], __ldcg(partials + slot(i) * Part::kFloats + h));
            }
        }
        cp_async_wait<0>();
        __syncthreads();
        const float *part = reinterpret_cast<const float *>(ring);
#pragma unroll
        for (int k = 0; k < Part::kPer; ++k) {
            const int h = h0 + k * Part::kHeadStep;
            if (h >= heads) break;
            if (c == 0)
                for (int i = 0; i < n; ++i) r.m[k] = fmaxf(r.m[k], part[i * floats + h]);
#pragma unroll 4
            for (int i = 0; i < n; ++i)
                add_part(r, k, part[i * floats + h], part[i * floats + kHeads + h],
                         *reinterpret_cast<const float4 *>(part + i * floats + 2 * kHeads + h * kDim + d));
        }
        __syncthreads();
    }
}

// Writes this CTA's partial result to slot `at` and says so; true for the last
// of `expected` arrivals at `counter`, which then sees all of theirs.
template <int kHeads, int kDim>
__device__ __forceinline__ bool leave_part(float *partials, int64_t at, uint32_t *counter, int expected, int heads,
                                           const JoinPart<kHeads, kDim> &r, int *flag) {
    using Part = JoinPart<kHeads, kDim>;
    const int h0 = threadIdx.x / Part::kLanes, d = threadIdx.x % Part::kLanes * 4;
    float *part = partials + at * Part::kFloats;
#pragma unroll
    for (int k = 0; k < Part::kPer; ++k) {
        const int h = h0 + k * Part::kHeadStep;
        if (h >= heads) break;
        if (d == 0) {
            __stcg(part + h, r.m[k]);
            __stcg(part + kHeads + h, r.l[k]);
        }
        __stcg(reinterpret_cast<float4 *>(part + 2 * kHeads + h * kDim + d), r.o[k]);
    }
    __syncthreads();
    if (threadIdx.x == 0) {
        // Releases every thread's stores (they happened before the barrier) and
        // acquires those of the arrivals before it.
        uint32_t before;
        asm volatile("atom.add.acq_rel.gpu.global.u32 %0, [%1], 1;" : "=r"(before) : "l"(counter) : "memory");
        const bool last = before == static_cast<uint32_t>(expected - 1);
        if (last) *counter = 0;  // as every run finds it
        *flag = last;
    }
    __syncthreads();
    const bool last = *flag != 0;
    __syncthreads();  // the flag is free again
    return last;
}

template <bool kE4m3, int kDim, int kNT, int kKeyHeads>
__global__ void __launch_bounds__(kKvThreads, AttendShape<kE4m3, kDim, kNT, kKeyHeads>::kPerSm) kv_attend_kernel(KvAttendParams p) {
    using Shape = AttendShape<kE4m3, kDim, kNT, kKeyHeads>;
    constexpr int kHeads = Shape::kHeads, kStages = Shape::kStages, kRow = Shape::kRow;
    constexpr int kSteps = kDim / 16;  // 16-wide steps over a head
    constexpr int kStep = Shape::kStep, kBlocks = Shape::kBlocks;
    constexpr int kRowHeads = Shape::kRowHeads;  // head h of a row: query head h / kKeyHeads of its key head h % kKeyHeads
    extern __shared__ __align__(1024) uint8_t smem[];
    griddep_launch_dependents();
    const KvCacheView &cache = p.cache;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int g = lane >> 2, j = lane & 3;
    const int step_lane = warp / kKeyHeads, row_key = warp % kKeyHeads;  // which of a tile's steps, which key head
    // Key head `key` of a row, and the chunk of its query heads.  (Two key heads: one chunk.)
    auto key_head = [&](int unit, int key) { return kKeyHeads == 1 ? unit / p.chunks : unit * kKeyHeads + key; };
    auto chunk_of = [&](int unit) { return kKeyHeads == 1 ? unit % p.chunks : 0; };
    const uint32_t ring = smem_u32(smem) + warp * kStages * Shape::kStage;
    float *join = reinterpret_cast<float *>(smem + kKvWarps * kStages * Shape::kStage);  // [warp][head][dim + 4]
    float *join_m = join + kKvWarps * kHeads * (kDim + 4);                                    // [warp][head]
    float *join_l = join_m + kKvWarps * kHeads;
    int *flag = reinterpret_cast<int *>(join_l + kKvWarps * kHeads);

    // Chunks past head_dim stay zero: no copy ever writes them.
    if (cache.head_dim < kDim) {
        for (int at = tid * 16; at < kKvWarps * kStages * Shape::kStage; at += kKvThreads * 16)
            *reinterpret_cast<uint4 *>(smem + at) = make_uint4(0u, 0u, 0u, 0u);
        __syncthreads();
    }
    griddep_wait();

    // The line of work: every lane sums a run of sequences, and a scan over
    // the lanes (the same in every warp: no barrier) gives the total and where
    // this CTA's part of it begins.
    const int B = static_cast<int>(p.sequences);
    const int run = (B + 31) / 32;
    AttendCursor cur;  // the warp's place in computing
    int64_t pos, end, total;
    uint32_t ctas;
    {
        int64_t incl = 0;
        for (int b = lane * run; b < B && b < (lane + 1) * run; ++b) {
            AttendCursor c;
            read_length<Shape>(p, b, c);
            incl += c.span * p.units;
        }
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int64_t other = __shfl_up_sync(0xffffffffu, incl, o);
            if (lane >= o) incl += other;
        }
        total = __shfl_sync(0xffffffffu, incl, 31);
        // CTAs at work: each has kKvMinPlaces at least (but the first of few).
        const int64_t worth = (total + kKvMinPlaces - 1) / kKvMinPlaces;
        ctas = worth < gridDim.x ? static_cast<uint32_t>(worth) : gridDim.x;
        pos = blockIdx.x < ctas ? share_of(total, blockIdx.x, ctas) : total;
        end = blockIdx.x < ctas ? share_of(total, blockIdx.x + 1, ctas) : total;
        if (pos < end) {
            // First lane whose inclusive sum is past pos.
            const int from = __ffs(__ballot_sync(0xffffffffu, incl > pos)) - 1;
            const int64_t before = __shfl_sync(0xffffffffu, incl, from > 0 ? from - 1 : 0);
            cur.base = from > 0 ? before : 0;
            cur.b = from * run;
            read_length<Shape>(p, cur.b, cur);
            seek<Shape>(p, cur, pos);
        }
    }

    // ---- loading: a cursor of its own, up to kStages - 1 steps ahead.
    AttendCursor lcur = cur;
    int64_t lpos = pos;
    AttendSegment lseg{};
    bool lmore = pos < end;
    if (lmore) lseg = segment_at<Shape>(lcur, lpos, end);
    int ltok = lseg.first + step_lane * kStep;  // first token of the step to load next
    int64_t lhead = 0;  // the row's head in the cache
    int lpage = -1;     // page of token ltok + lane % kStep, -1: not attended
    int lplace = 0;
    auto settle = [&]() {  // moves to the next step that exists and asks for its pages
        while (ltok >= lseg.last) {
            lpos += lseg.places;
            if (lpos >= end) {
                lmore = false;
                return;
            }
            seek<Shape>(p, lcur, lpos);
            lseg = segment_at<Shape>(lcur, lpos, end);
            ltok = lseg.first + step_lane * kStep;
        }
        lhead = static_cast<int64_t>(key_head(lseg.unit, row_key)) * cache.head_stride;
        const int t = ltok + (lane & (kStep - 1));
        lpage = -1;
        if (t >= lcur.low && t < lseg.last) {
            const uint32_t q = static_cast<uint32_t>(t) / static_cast<uint32_t>(cache.page_size);
            lplace = t - static_cast<int>(q) * cache.page_size;
            lpage = cache.table[lcur.b * cache.table_width + q];
            if (lpage < 0 || lpage >= cache.num_pages) {
                atomicOr(p.status, kKvErrPage);
                lpage = -1;
            }
        }
    };
    if (lmore) settle();
    constexpr uint32_t kAll = kStep == 32 ? 0xffffffffu : 0xffffu;
    uint32_t valid[kStages];  // tokens of each stage that are attended, a bit each
#pragma unroll
    for (int s = 0; s < kStages; ++s) valid[s] = 0;
    const int row_chunks = cache.head_dim * Shape::kElem / 16;
    auto load = [&](int slot) {
        uint32_t bits = 0;
        if (lmore) {
            const bool ok = lpage >= 0;
            bits = __ballot_sync(0xffffffffu, ok) & kAll;
            const int64_t offset =
                ok ? lpage * cache.page_stride + lplace * cache.token_stride + lhead : 0;
            const uint32_t to = ring + slot * Shape::kStage;
            const uint8_t *kc = static_cast<const uint8_t *>(p.k_cache), *vc = static_cast<const uint8_t *>(p.v_cache);
            constexpr int kRowsAtOnce = 32 / (Shape::kChunks < 32 ? Shape::kChunks : 32);
#pragma unroll
            for (int i = 0; i < kStep / kRowsAtOnce; ++i) {
                const int r = i * kRowsAtOnce + lane / Shape::kChunks, c = lane % Shape::kChunks;
                const int64_t at = __shfl_sync(0xffffffffu, offset, r) * Shape::kElem + c * 16;
                const bool fill = (bits >> r) & 1u;
                if (c < row_chunks) {
                    const uint32_t d = to + chunk_at<kRow>(r, c);
                    cp_async16(d, kc + (fill ? at : 0), fill);
                    cp_async16(d + kStep * kRow, vc + (fill ? at : 0), fill);
                }
            }
            ltok += Shape::kTile;
            settle();
        }
#pragma unroll
        for (int s = 0; s < kStages; ++s)
            if (s == slot) valid[s] = bits;
        cp_async_commit();
    };
    int slot_in = 0, slot = 0;
#pragma unroll
    for (int s = 0; s < kStages - 1; ++s) load(slot_in++);

    // Sequences without tokens have no tiles: their rows are written here.
    for (int b = blockIdx.x; b < B; b += gridDim.x) {
        AttendCursor c;
        read_length<Shape>(p, b, c);
        if (c.n > 0) continue;
        for (int i = tid; i < p.q_heads * cache.head_dim; i += kKvThreads) p.out[b * p.out_stride + i] = 0;
        if (p.lse)
            for (int h = tid; h < p.q_heads; h += kKvThreads) p.lse[static_cast<int64_t>(b) * p.q_heads + h] = -INFINITY;
    }
    if (pos >= end) return;

    // ---- computing, row by row.  The queries of a row are asked for before
    // the row ahead of it is joined.
    // Second operand: column (head) g, rows (elements) of lane j.  From an 8-bit
    // cache the elements come 4j .. 4j + 3 of each 16 (below).
    uint2 raw[kNT][kSteps];
    float key_scale = 1.f;
    AttendSegment seg;
    auto ask = [&]() {
        for (; pos < end; pos += seg.places) {
            seek<Shape>(p, cur, pos);
            seg = segment_at<Shape>(cur, pos, end);
            if (seg.tiles > 0) break;
        }
        if (pos >= end) return;
        const int chunk = chunk_of(seg.unit), key = key_head(seg.unit, row_key);
        const int heads = min(p.chunk_heads, p.group - chunk * p.chunk_heads);
        const int64_t head0 = key * p.group + chunk * p.chunk_heads;
#pragma unroll
        for (int t = 0; t < kNT; ++t) {
            const uint16_t *q = p.q + cur.b * p.q_stride + (head0 + 8 * t + g) * cache.head_dim;
#pragma unroll
            for (int k = 0; k < kSteps; ++k) {
                const bool in = 8 * t + g < heads && 16 * k < cache.head_dim;
                if constexpr (kE4m3) {
                    raw[t][k] = in ? *reinterpret_cast<const uint2 *>(q + 16 * k + 4 * j) : make_uint2(0u, 0u);
                } else {
                    raw[t][k].x = in ? *reinterpret_cast<const uint32_t *>(q + 16 * k + 2 * j) : 0u;
                    raw[t][k].y = in ? *reinterpret_cast<const uint32_t *>(q + 16 * k + 8 + 2 * j) : 0u;
                }
            }
        }
        if (kE4m3 && p.k_scale) key_scale = p.k_scale[key];
    };
    ask();
    while (pos < end) {
        const int chunk = chunk_of(seg.unit);
        const int heads = kKeyHeads * min(p.chunk_heads, p.group - chunk * p.chunk_heads);  // of the row
        const int row_b = cur.b;
        const int64_t row_tiles = cur.tiles, seg_tiles = seg.tiles, row_begin = seg.row_begin;
        const int seg_unit = seg.unit;

        uint32_t qf[kNT][kSteps][2];
        float factor[kNT][2];  // logit to exponent of two, of this lane's heads 2j, 2j + 1
#pragma unroll
        for (int t = 0; t < kNT; ++t) {
            const float scale = p.scale * 1.4426950408889634f;
            if constexpr (!kE4m3) {
#pragma unroll
                for (int k = 0; k < kSteps; ++k) qf[t][k][0] = raw[t][k].x, qf[t][k][1] = raw[t][k].y;
                factor[t][0] = factor[t][1] = scale;
            } else {
                uint32_t top = 0;  // largest magnitude, as bf16 bits
#pragma unroll
                for (int k = 0; k < kSteps; ++k) {
                    top = max(max(top, raw[t][k].x & 0x7fffu), (raw[t][k].x >> 16) & 0x7fffu);
                    top = max(max(top, raw[t][k].y & 0x7fffu), (raw[t][k].y >> 16) & 0x7fffu);
                }
                top = max(top, __shfl_xor_sync(0xffffffffu, top, 1));
                top = max(top, __shfl_xor_sync(0xffffffffu, top, 2));
                // 2^-e brings the largest to [2^14, 2^15), so that fp16 holds elements
                // down to 2^-32 of it exactly; e within ±126 keeps both powers normal numbers.
                const int e = min(126, max(-126, static_cast<int>(top >> 7) - 127 - 14));
                const float down = __uint_as_float(static_cast<uint32_t>(127 - e) << 23);
#pragma unroll
                for (int k = 0; k < kSteps; ++k) {
                    const uint32_t w[2] = {raw[t][k].x, raw[t][k].y};
#pragma unroll
                    for (int i = 0; i < 2; ++i) {
                        const __half2 h = __floats2half2_rn(__uint_as_float(w[i] << 16) * down,
                                                            __uint_as_float(w[i] & 0xffff0000u) * down);
                        qf[t][k][i] = *reinterpret_cast<const uint32_t *>(&h);
                    }
                }
                const float up = scale * __uint_as_float(static_cast<uint32_t>(127 + e) << 23) * key_scale;
                factor[t][0] = __shfl_sync(0xffffffffu, up, 8 * j);
                factor[t][1] = __shfl_sync(0xffffffffu, up, 8 * j + 4);
            }
        }

        float m[kNT][2], l[kNT][2], o[kNT][kSteps][4];
#pragma unroll
        for (int t = 0; t < kNT; ++t) {
            m[t][0] = m[t][1] = -INFINITY;
            l[t][0] = l[t][1] = 0.f;
#pragma unroll
            for (int d = 0; d < kSteps; ++d) o[t][d][0] = o[t][d][1] = o[t][d][2] = o[t][d][3] = 0.f;
        }

        for (int tok = seg.first + step_lane * kStep; tok < seg.last; tok += Shape::kTile) {
            cp_async_wait<kStages - 2>();
            __syncwarp();
            uint32_t bits = 0;
#pragma unroll
            for (int s = 0; s < kStages; ++s)
                if (s == slot) bits = valid[s];
            load(slot_in == kStages ? 0 : slot_in);
            slot_in = slot_in == kStages ? 1 : slot_in + 1;
            const uint32_t ks = ring + slot * Shape::kStage, vs = ks + kStep * kRow;
            slot = slot + 1 == kStages ? 0 : slot + 1;

            float x[kBlocks][kNT][4];
#pragma unroll
            for (int n = 0; n < kBlocks; ++n)
#pragma unroll
                for (int t = 0; t < kNT; ++t) x[n][t][0] = x[n][t][1] = x[n][t][2] = x[n][t][3] = 0.f;
            if constexpr (!kE4m3) {
#pragma unroll
                for (int k = 0; k < kSteps; ++k)
#pragma unroll
                    for (int n = 0; n < kBlocks; ++n) {
                        uint32_t a[4];
                        ldsm_x4(a, ks + chunk_at<kRow>(16 * n + (lane & 15), 2 * k + (lane >> 4)));
#pragma unroll
                        for (int t = 0; t < kNT; ++t)
                            mma16816<false>(x[n][t], a[0], a[1], a[2], a[3], qf[t][k][0], qf[t][k][1]);
                    }
            } else {
                // A 16-byte chunk holds 16 elements: lane j of a row receives
                // elements 4j .. 4j + 3, so the first pair stands at the
                // step's rows 2j, 2j + 1 and the second at rows 2j + 8, + 9.
#pragma unroll
                for (int k = 0; k < kSteps; k += 2)
#pragma unroll
                    for (int n = 0; n < kBlocks; ++n) {
                        uint32_t a[4];
                        ldsm_x4(a, ks + chunk_at<kRow>(16 * n + (lane & 15), k + (lane >> 4)));
#pragma unroll
                        for (int i = 0; i < 2; ++i) {
                            const uint32_t up = a[2 * i], dn = a[2 * i + 1];
                            const uint32_t a0 = e4m3x2_to_half2(up), a2 = e4m3x2_to_half2(up >> 16);
                            const uint32_t a1 = e4m3x2_to_half2(dn), a3 = e4m3x2_to_half2(dn >> 16);
#pragma unroll
                            for (int t = 0; t < kNT; ++t)
                                mma16816<true>(x[n][t], a0, a1, a2, a3, qf[t][k + i][0], qf[t][k + i][1]);
                        }
                    }
            }

            // x: tokens g (0, 1) and g + 8 (2, 3) of each block, heads 2j and 2j + 1.
            constexpr int kParts = WeightParts<kE4m3>::kCount;
            uint32_t weight[kBlocks][kNT][2][kParts];
#pragma unroll
            for (int t = 0; t < kNT; ++t) {
#pragma unroll
                for (int n = 0; n < kBlocks; ++n)
#pragma unroll
                    for (int i = 0; i < 4; ++i) x[n][t][i] *= factor[t][i & 1];
                if (bits != kAll) {
#pragma unroll
                    for (int n = 0; n < kBlocks; ++n)
#pragma unroll
                        for (int i = 0; i < 4; ++i)
                            if (!((bits >> (16 * n + g + 8 * (i >> 1))) & 1u)) x[n][t][i] = -INFINITY;
                }
                float keep[2];
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    float top = fmaxf(x[0][t][h], x[0][t][2 + h]);
                    if constexpr (kBlocks == 2) top = fmaxf(top, fmaxf(x[1][t][h], x[1][t][2 + h]));
                    top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 4));
                    top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 8));
                    top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 16));
                    top = fmaxf(top, m[t][h]);
                    const float base = top == -INFINITY ? 0.f : top;  // no token yet: every weight is 0
                    keep[h] = exp2_fast(m[t][h] - base);
                    m[t][h] = top;
                    l[t][h] *= keep[h];
#pragma unroll
                    for (int n = 0; n < kBlocks; ++n) {
                        x[n][t][h] = exp2_fast(x[n][t][h] - base);
                        x[n][t][2 + h] = exp2_fast(x[n][t][2 + h] - base);
                        l[t][h] += x[n][t][h] + x[n][t][2 + h];
                    }
                }
                if (__any_sync(0xffffffffu, keep[0] != 1.f || keep[1] != 1.f)) {
#pragma unroll
                    for (int d = 0; d < kSteps; ++d) {
                        o[t][d][0] *= keep[0];
                        o[t][d][1] *= keep[1];
                        o[t][d][2] *= keep[0];
                        o[t][d][3] *= keep[1];
                    }
                }
#pragma unroll
                for (int n = 0; n < kBlocks; ++n)
#pragma unroll
                    for (int i = 0; i < 2; ++i) {
                        const WeightParts<kE4m3> s = split<kE4m3>(x[n][t][2 * i], x[n][t][2 * i + 1]);
#pragma unroll
                        for (int y = 0; y < kParts; ++y) weight[n][t][i][y] = transpose8x8(s.part[y]);
                    }
            }
            if constexpr (!kE4m3) {
#pragma unroll
                for (int n = 0; n < kBlocks; ++n)
#pragma unroll
                    for (int d = 0; d < kSteps; ++d) {
                        uint32_t a[4];
                        ldsm_x4_t(a, vs + chunk_at<kRow>(16 * n + (lane & 7) + ((lane >> 4) << 3), 2 * d + ((lane >> 3) & 1)));
#pragma unroll
                        for (int t = 0; t < kNT; ++t)
#pragma unroll
                            for (int y = 0; y < kParts; ++y)
                                mma16816<false>(o[t][d], a[0], a[1], a[2], a[3], weight[n][t][0][y], weight[n][t][1][y]);
                    }
            } else {
                // Transposed in pairs of elements: a lane receives elements
                // 2g, 2g + 1 of tokens 2j, 2j + 1.  Rows 0..7 of the step take
                // the even elements, rows 8..15 the odd ones.
#pragma unroll
                for (int n = 0; n < kBlocks; ++n)
#pragma unroll
                    for (int d = 0; d < kSteps; d += 2) {
                        uint32_t a[4];
                        ldsm_x4_t(a, vs + chunk_at<kRow>(16 * n + (lane & 7) + (((lane >> 3) & 1) << 3), d + (lane >> 4)));
#pragma unroll
                        for (int i = 0; i < 2; ++i) {
                            const uint32_t lo8 = __byte_perm(a[2 * i], 0, 0x3120), hi8 = __byte_perm(a[2 * i + 1], 0, 0x3120);
                            const uint32_t a0 = e4m3x2_to_half2(lo8), a1 = e4m3x2_to_half2(lo8 >> 16);
                            const uint32_t a2 = e4m3x2_to_half2(hi8), a3 = e4m3x2_to_half2(hi8 >> 16);
                            const uint32_t s0 = half2_mul(a0, kHalfRestBack), s1 = half2_mul(a1, kHalfRestBack);
                            const uint32_t s2 = half2_mul(a2, kHalfRestBack), s3 = half2_mul(a3, kHalfRestBack);
#pragma unroll
                            for (int t = 0; t < kNT; ++t) {
                                mma16816<true>(o[t][d + i], a0, a1, a2, a3, weight[n][t][0][0], weight[n][t][1][0]);
                                mma16816<true>(o[t][d + i], s0, s1, s2, s3, weight[n][t][0][1], weight[n][t][1][1]);
                            }
                        }
                    }
            }
        }

        pos += seg.places;
        ask();

        // Join the warps.
        using Part = JoinPart<kRowHeads, kDim>;
#pragma unroll
        for (int t = 0; t < kNT; ++t) {
#pragma unroll
            for (int h = 0; h < 2; ++h) {
#pragma unroll
                for (int s = 4; s < 32; s <<= 1) l[t][h] += __shfl_xor_sync(0xffffffffu, l[t][h], s);
                if (g == 0) {
                    join_m[warp * kHeads + 8 * t + 2 * j + h] = m[t][h];
                    join_l[warp * kHeads + 8 * t + 2 * j + h] = l[t][h];
                }
            }
#pragma unroll
            for (int d = 0; d < kSteps; ++d) {
                float *to = join + (warp * kHeads + 8 * t + 2 * j) * Part::kPitch + 16 * d;
                if constexpr (kE4m3) {
                    *reinterpret_cast<float2 *>(to + 2 * g) = make_float2(o[t][d][0], o[t][d][2]);
                    *reinterpret_cast<float2 *>(to + Part::kPitch + 2 * g) = make_float2(o[t][d][1], o[t][d][3]);
                } else {
                    to[g] = o[t][d][0];
                    to[Part::kPitch + g] = o[t][d][1];
                    to[g + 8] = o[t][d][2];
                    to[Part::kPitch + g + 8] = o[t][d][3];
                }
            }
        }
        __syncthreads();
        const int h0 = tid / Part::kLanes, d0 = tid % Part::kLanes * 4;
        Part r;
        r.clear();
#pragma unroll
        for (int k = 0; k < Part::kPer; ++k) {
            const int h = h0 + k * Part::kHeadStep;
            if (h >= heads) break;
            const int at = h % kKeyHeads * kHeads + h / kKeyHeads;  // in the first of its warps
            float warp_m[Shape::kLanes];
#pragma unroll
            for (int i = 0; i < Shape::kLanes; ++i) {
                warp_m[i] = join_m[i * kRowHeads + at];
                r.m[k] = fmaxf(r.m[k], warp_m[i]);
            }
            const float base = finite_or_zero(r.m[k]);
#pragma unroll
            for (int i = 0; i < Shape::kLanes; ++i) {
                const float w = exp2_fast(warp_m[i] - base);
                const float4 v = *reinterpret_cast<const float4 *>(join + (i * kRowHeads + at) * Part::kPitch + d0);
                r.l[k] += w * join_l[i * kRowHeads + at];
                r.o[k].x += w * v.x, r.o[k].y += w * v.y, r.o[k].z += w * v.z, r.o[k].w += w * v.w;
            }
        }

        bool write = true;
        if (seg_tiles != row_tiles) {
            // Other CTAs own the rest of the row: leave this part in scratch,
            // and join all parts if the others are there already.
            // First and last owner of its tiles.
            const int64_t row_first = row_begin + kKvRowCost, row_end = row_first + row_tiles;
            const int c0 = static_cast<int>(divide((row_first + 1) * ctas - 1, total));
            const int c1 = static_cast<int>(divide(row_end * ctas - 1, total));
            const int parts = c1 - c0 + 1, mine = static_cast<int>(blockIdx.x) - c0;
            // A CTA's scratch: slot 0 for a row begun by another, slot 1 for the row that it begins last.
            auto slot = [&](int part) { return int64_t(2) * (c0 + part) + (part == 0 ? 1 : 0); };
            uint32_t *counter = p.counters + static_cast<int64_t>(row_b) * p.units + seg_unit;
            // A CTA that has no more to load joins by way of its ring.
            auto join_all = [&](int count, auto at) {
                if (pos >= end)
                    join_parts_in<kRowHeads, kDim>(smem, kKvWarps * kStages * Shape::kStage, p.partials, count, at, heads, r);
                else
                    join_parts<kRowHeads, kDim>(p.partials, count, at, heads, r);
            };
            if (parts <= kKvJoinOnce) {
                write = leave_part<kRowHeads, kDim>(p.partials, slot(mine), counter, parts, heads, r, flag);
                if (write) join_all(parts, slot);
            } else {
                // Many parts: in groups, each joined into its first part's
                // slot by its own last arrival, and then the groups.
                const int size = parts <= kKvJoinMany ? kKvJoinGroup : 2 * kKvJoinGroup;
                const int g0 = mine / size * size, in_group = min(size, parts - g0);
                write = leave_part<kRowHeads, kDim>(p.partials, slot(mine), p.group_counters + slot(g0), in_group, heads, r, flag);
                if (write) {
                    join_all(in_group, [&](int i) { return slot(g0 + i); });
                    __syncthreads();  // every thread has read the slot that is written next
                    const int groups = (parts + size - 1) / size;
                    write = leave_part<kRowHeads, kDim>(p.partials, slot(g0), counter, groups, heads, r, flag);
                    if (write) join_all(groups, [&](int i) { return slot(i * size); });
                }
            }
        }
        if (write) {
#pragma unroll
            for (int k = 0; k < Part::kPer; ++k) {
                const int h = h0 + k * Part::kHeadStep;
                if (h >= heads) break;
                const int key = key_head(seg_unit, h % kKeyHeads);
                const int64_t head = static_cast<int64_t>(key) * p.group + chunk * p.chunk_heads + h / kKeyHeads;
                const float by = kE4m3 ? (p.v_scale ? p.v_scale[key] : 1.f) * kHalfWeightBack : 1.f;
                const float inv = r.l[k] == 0.f ? 0.f : by / r.l[k];  // (a NaN stays one)
                if (d0 < cache.head_dim)
                    *reinterpret_cast<uint2 *>(p.out + row_b * p.out_stride + head * cache.head_dim + d0) =
                        make_uint2(bf16_pair(r.o[k].x * inv, r.o[k].y * inv), bf16_pair(r.o[k].z * inv, r.o[k].w * inv));
                if (p.lse && d0 == 0)
                    p.lse[static_cast<int64_t>(row_b) * p.q_heads + head] =
                        r.l[k] == 0.f ? -INFINITY : (r.m[k] + log2f(r.l[k])) * 0.6931471805599453f;
            }
        }
        __syncthreads();  // the join buffer is free again
    }
    cp_async_wait<0>();
}

}  // namespace dev
}  // namespace projgb
