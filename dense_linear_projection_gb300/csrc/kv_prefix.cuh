// Device code of attention over a prefix that a whole batch shares, and of its join
// with each sequence's own tokens.
//
// Mathematics.  The R = sequences · group query rows of one key head against the
// prefix's tokens: X[row, t] = scale·log2(e)·q[row]·k[t], and for a stretch of tokens
// m = max X, l = Σ 2^(X − m), o = Σ 2^(X − m)·v[t] (a part).  Parts join as in
// kv_attend.cuh: against the largest m.
//
// What bounds it: with 128 rows a tile the products, 2 · 128 · 128 · head_dim
// operations a 128 tokens for X and, with a weight in three bf16 parts (24 bits, as
// kv_attend.cuh holds it), three times that for o; so up to 128 rows the bytes of K
// and V (each read once for the whole batch) take about as long, and past them the
// tensor core alone counts.  So
//   * X = Q·Kᵀ and o += P·V are tcgen05 products of 128 rows, accumulated in tensor
//     memory: X of two token tiles, so that the one's softmax overlaps the other's
//     products, and o.  P stays in tensor memory too, written over X.
//   * warps 0..15 turn X into P, in two groups that take every other tile, so that the one's
//     waits lie under the other's arithmetic (splitting a weight takes 12 of the 20
//     instructions for two of them).  A thread has one row (tensor-memory lane) and half of
//     a tile's tokens.
//   * weights are relative to the maximum of the first tile of a CTA's stretch, so that a
//     later tile's X is read once and nothing is handed on: fp32 sums and bf16 parts are as
//     exact at 2^60 as at 1.  Where a tile's sum comes to 2^64, or o is not finite, the
//     stretch is done again with running maxima, o rescaled where they grow by more than
//     2^8 (kLazy).  (With running maxima throughout, 128 sequences behind 32768 tokens took
//     237 us.  Nearly every stretch done again, with keys that rise so far or infinite values
//     everywhere: 226 -> 415 us; 64 sequences behind 8192 73.5 -> 107; over 8 bits 74 -> 128.)
//   * warps 16..19 fill a ring of token tiles: pages of whole multiples of 8 tokens by TMA
//     boxes of up to 32 tokens, others, and the prefix's end, by 16-byte asynchronous copies
//     (which any page size and strides allow); warp 20 issues the products.
//   * (key head, row tile, token tile) in this order are one line that the CTAs share
//     evenly; each stretch of one row tile leaves a part in the workspace.
//
// Measured: 1024 rows a key head, 8 key heads, 32768 tokens: 193 us, 712 TFLOP/s of the
// formula's operations and 1424 of those carried out, 74 % of what a library product
// reaches; 512 rows, 8192 tokens: 36 us (a quarter of it the start and end of the 13
// tiles that a CTA has).  Of a tile's 3000 cycles the products take 2100.  Tiles of 64 tokens in
// four buffers, a group of warps each: 294 us for the first where two of 128 took 258
// (every change between the two products costs about 300 cycles); the products issued from
// a branch of one lane: 418; X held in registers by 16 warps: spills.
//
// Every wait is bounded (wait_limit_ns); one that runs out records itself, and the CTA drains its
// products and copies, frees its tensor memory and returns; the rows whose parts it had not
// computed then come out as NaN.
#pragma once

#include "kv_attend.cuh"

namespace projgb {
namespace dev {

constexpr int kPrefixRows = 128;          // query rows of a tile
constexpr int kPrefixGroups = 2;          // of softmax warps, for every other tile each
constexpr int kPrefixPieces = 2;          // of a tile's tokens, a softmax thread's each
constexpr int kPrefixSums = kPrefixGroups * kPrefixPieces;  // threads of a row
constexpr int kPrefixSoftmaxWarps = 4 * kPrefixSums, kPrefixLoadWarps = 4;
constexpr int kPrefixLoaders = 32 * kPrefixLoadWarps;
constexpr int kPrefixThreads = 32 * (kPrefixSoftmaxWarps + kPrefixLoadWarps + 1);
constexpr float kLazy = 8.f;
constexpr float kMostSum = 0x1p64f;  // of a tile's weights, relative to the first tile's maximum
constexpr int64_t kPrefixWaitNs = 1000000000;
constexpr int64_t kPrefixFaultNs = 100000;   // instead, where one is to run out
constexpr uint64_t kPrefixLandNs = 2000000;  // for copies on their way

template <bool kE4m3, int kDim>
struct PrefixShape {
    static constexpr int kTokens = kDim > 128 ? 64 : 128;  // of a tile
    static constexpr int kTile = kTokens * kDim * 2;        // bytes of a tile of keys or values, bf16
    static constexpr int kRaw = kE4m3 ? kTile / 2 : 0;      // as they are in an 8-bit cache
    static constexpr int kSlots = kDim <= 64 ? 6 : kE4m3 ? 3 : kDim <= 128 ? 5 : 4;  // (three: keys of two tiles, values of one)
    static constexpr int kRaws = kE4m3 ? (kDim > 128 ? 2 : 4) : 0;
    static constexpr int kQ = kPrefixRows * kDim * 2;
    static constexpr int kCtl = 9216;
    static constexpr int kSmem = kQ + kSlots * kTile + kRaws * kRaw + kCtl;
    // Tensor memory: o, then two buffers of X, each with room for P's three parts: of 16 tokens
    // the first two lie over their X, the third after X.  (A thread so overwrites only what it
    // has read itself.)
    static constexpr int kBuffer = kTokens / 2 * 3;
    static constexpr int kColumns = kDim + 2 * kBuffer;
    // A part: [maximum of a row][its threads' sums][kDim/4][row] float4.
    static constexpr int kPart = (1 + kPrefixSums) * kPrefixRows + kPrefixRows * kDim;
    static_assert(kColumns <= 512 && kSmem <= 227 * 1024, "tensor memory and shared memory of an SM");
};

struct PrefixCtl {
    uint64_t full[8], empty[8], raw_full[4][kPrefixLoadWarps], q_full, q_empty, x_full[2], p_full[2][2], o_done[2], drain;
    uint64_t base_full[2][4];  // [quarter of the rows]: a base has been left
    uint32_t tmem;
    int abort_flag;
    uint32_t valid[8][4];     // tokens of the last tiles that exist, a bit each
    uint4 row[kPrefixLoadWarps][2][32];  // [tile & 1]: where a token lies in the cache (bytes), how many bytes of it to copy
    float top[2][kPrefixPieces][kPrefixRows];  // [tile & 1]: a row's maximum
    float base[2][kPrefixRows];                // what weights are relative to, the last two left
    uint32_t redo[2];                          // stretches to be done again, a bit each (the last for all from it on)
};
static_assert(sizeof(PrefixCtl) <= 9216, "PrefixShape::kCtl");

// D[tmem] (+)= A[tmem] · B[smem], bf16, fp32 accumulators.
__device__ __forceinline__ void tc_mma_ts(uint32_t d_tmem, uint32_t a_tmem, uint64_t b_desc, uint32_t idesc, uint32_t accumulate) {
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d_tmem),
        "r"(a_tmem), "l"(b_desc), "r"(idesc), "r"(accumulate)
        : "memory");
}
__device__ __forceinline__ void tma_load_4d(uint32_t dst, const void *map, uint32_t bar, int32_t x, int32_t y, int32_t z, int32_t w) {
    asm volatile(
        "cp.async.bulk.tensor.4d.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4, %5}], [%6];" ::"r"(dst),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(z), "r"(w), "r"(bar)
        : "memory");
}
__device__ __forceinline__ void tmem_store8(uint32_t at, const uint32_t (&r)[8]) {
    asm volatile("tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"r"(at), "r"(r[0]),
                 "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7])
                 : "memory");
}
__device__ __forceinline__ void tmem_store16(uint32_t at, const float (&v)[16]) {
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, "
        "%16};" ::"r"(at),
        "f"(v[0]), "f"(v[1]), "f"(v[2]), "f"(v[3]), "f"(v[4]), "f"(v[5]), "f"(v[6]), "f"(v[7]), "f"(v[8]), "f"(v[9]), "f"(v[10]),
        "f"(v[11]), "f"(v[12]), "f"(v[13]), "f"(v[14]), "f"(v[15])
        : "memory");
}
// Columns of the thread's lane, as they are.
__device__ __forceinline__ void tmem_load(uint32_t at, uint32_t (&r)[16]) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x16.b32 "
        "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, [%16];\n\t"
        "tcgen05.wait::ld.sync.aligned;"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
        : "r"(at)
        : "memory");
}
__device__ __forceinline__ void tmem_load(uint32_t at, uint32_t (&r)[32]) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x32.b32 "
        "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, %16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31}, [%32];\n\t"
        "tcgen05.wait::ld.sync.aligned;"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]), "=r"(r[16]), "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]), "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
        : "r"(at)
        : "memory");
}
__device__ __forceinline__ void tmem_store(uint32_t at, const uint32_t (&r)[16]) {
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, "
        "%16};" ::"r"(at),
        "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]), "r"(r[10]),
        "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
        : "memory");
}
__device__ __forceinline__ void tmem_store_wait() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }
__device__ __forceinline__ void async_proxy_fence() { asm volatile("fence.proxy.async.shared::cta;" ::: "memory"); }
// 16 bytes, of which `from` has the first `bytes` (16 or 0: then zeros).
__device__ __forceinline__ void cp_async16n(uint32_t to, const void *from, uint32_t bytes) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(to), "l"(from), "r"(bytes) : "memory");
}
// Arrives on `bar` once the thread's copies so far are in shared memory.
__device__ __forceinline__ void cp_async_arrive(uint32_t bar) {
    asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(bar) : "memory");
}
// One lane of a converged warp, the same one every time.
__device__ __forceinline__ bool elect_one() {
    uint32_t yes;
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "elect.sync _|p, 0xffffffff;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(yes));
    return yes != 0;
}
__device__ __forceinline__ void named_barrier(int id, int threads) {
    asm volatile("bar.sync %0, %1;" ::"r"(id), "r"(threads) : "memory");
}

// Two weights as three bf16 parts, the same as split<false>'s: each but the last the upper half of
// the next float below, so that every part of a positive weight is positive.
__device__ __forceinline__ void split3(uint64_t w, uint32_t &hi, uint32_t &mid, uint32_t &lo) {
    const uint64_t below = pair_of(0x1.fffffep-1f, 0x1.fffffep-1f), minus = pair_of(-1.f, -1.f);
    uint32_t *to[2] = {&hi, &mid};
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const float2 h = pair_to(mul2_rz(w, below));
        const uint32_t a = __float_as_uint(h.x), b = __float_as_uint(h.y);
        *to[i] = __byte_perm(a, b, 0x7632);
        w = fma2(pair_of(__uint_as_float(a & 0xffff0000u), __uint_as_float(b & 0xffff0000u)), minus, w);
    }
    const float2 r = pair_to(w);
    lo = bf16_pair(r.x, r.y);
}

// kind::f16 instruction descriptor: fp32 accumulators, bf16 operands, M = 128.
__device__ constexpr uint32_t prefix_idesc(int n, bool b_mn_major) {
    return (1u << 4) | (1u << 7) | (1u << 10) | (b_mn_major ? 1u << 16 : 0u) | (static_cast<uint32_t>(n >> 3) << 17) | (8u << 24);
}

// 16 values of an 8-bit cache as bf16 (exact), by way of fp16 (which keeps NaN).
__device__ __forceinline__ void e4m3_to_bf16(uint4 raw, uint4 &lo, uint4 &hi) {
    const uint32_t w[4] = {raw.x, raw.y, raw.z, raw.w};
    uint32_t o[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const uint32_t h = e4m3x2_to_half2(w[i / 2] >> (16 * (i & 1)));
        const float2 f = __half22float2(*reinterpret_cast<const __half2 *>(&h));
        o[i] = bf16_pair(f.x, f.y);
    }
    lo = make_uint4(o[0], o[1], o[2], o[3]);
    hi = make_uint4(o[4], o[5], o[6], o[7]);
}

// The stretch of the line that is CTA c's, and its part of one (key head, row tile).
struct PrefixWork {
    int64_t pos, end, tiles, unit;  // places; token tiles of a unit; unit of place `pos`
    __device__ __forceinline__ PrefixWork(const KvPrefixParams &p) {
        const int64_t total = p.cache.kv_heads * p.row_tiles * p.tiles;
        pos = total * blockIdx.x / gridDim.x;
        end = total * (blockIdx.x + 1) / gridDim.x;
        tiles = p.tiles;
        unit = pos / tiles;
    }
};

// The part of a CTA that has not computed it: NaN in the sums of thread t of the sums' kPrefixSums ·
// kPrefixRows, so that the rows' outputs and log sums are NaN and not what the memory held before.
template <class Shape>
__device__ __forceinline__ void leave_nan(const KvPrefixParams &p, int64_t unit, int t) {
    if (t < kPrefixSums * kPrefixRows) p.partials[(unit + blockIdx.x) * Shape::kPart + kPrefixRows + t] = NAN;
}

template <bool kE4m3, int kDim>
__global__ void __launch_bounds__(kPrefixThreads, 1)
    kv_prefix_kernel(const __grid_constant__ KvPrefixParams p, const __grid_constant__ CUtensorMap k_map,
                     const __grid_constant__ CUtensorMap v_map) {
    using Shape = PrefixShape<kE4m3, kDim>;
    constexpr int kTokens = Shape::kTokens, kTile = Shape::kTile, kSlots = Shape::kSlots;
    constexpr int kPiece = kTokens / kPrefixPieces;        // tokens of a softmax thread
    constexpr int kMine = kTokens / kPrefixLoadWarps;       // of a loading warp
    constexpr int kOwn = kDim / kPrefixSums;                // elements of its row that a softmax thread writes
    static_assert(kPiece == 2 * kMine, "a piece's tokens are two loading warps'");
    constexpr uint32_t kAll = kMine == 32 ? 0xffffffffu : 0xffffu;
    extern __shared__ __align__(1024) uint8_t smem[];
    uint8_t *ring = smem + Shape::kQ, *raws = ring + kSlots * kTile;
    PrefixCtl *ctl = reinterpret_cast<PrefixCtl *>(raws + Shape::kRaws * Shape::kRaw);
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    volatile int *abort_flag = &ctl->abort_flag;
    if (smem_u32(smem) & 1023u) {  // (128-byte swizzled tiles; the same in every thread)
        griddep_wait();  // (the next kernel counts on what came before this one)
        if (tid == 0) atomicOr(p.status, kKvErrWait);
        const PrefixWork work(p);
        for (int64_t unit = work.unit; unit * work.tiles < work.end; ++unit) leave_nan<Shape>(p, unit, tid);
        return;
    }
    if (warp == kPrefixSoftmaxWarps + kPrefixLoadWarps) {
        tmem_alloc<false>(smem_u32(&ctl->tmem), 512);
        tmem_relinquish<false>();
    }
    if (tid == 0) {
        static_assert(Shape::kRaws <= 4 && (!kE4m3 || kSlots >= 3), "barriers");
        for (int i = 0; i < 8; ++i) {
            // (A copying loader arrives when its copies do; its warp once more, for `valid`.)
            mbar_init(smem_u32(&ctl->full[i]), kE4m3 ? kPrefixLoaders : kPrefixLoaders + kPrefixLoadWarps);
            mbar_init(smem_u32(&ctl->empty[i]), 1);
            if (kE4m3 && i < Shape::kRaws)
                for (int w = 0; w < kPrefixLoadWarps; ++w) mbar_init(smem_u32(&ctl->raw_full[i][w]), 33);
        }
        mbar_init(smem_u32(&ctl->q_full), kPrefixLoaders);
        mbar_init(smem_u32(&ctl->q_empty), 1);
        for (int i = 0; i < 2; ++i) {
            mbar_init(smem_u32(&ctl->x_full[i]), 1);
            for (int h = 0; h < 2; ++h) mbar_init(smem_u32(&ctl->p_full[i][h]), 32 * kPrefixSoftmaxWarps / kPrefixGroups);
            mbar_init(smem_u32(&ctl->o_done[i]), 1);
            for (int q = 0; q < 4; ++q) mbar_init(smem_u32(&ctl->base_full[i][q]), 32 * kPrefixPieces);
        }
        mbar_init(smem_u32(&ctl->drain), 1);
        ctl->abort_flag = 0;
        ctl->redo[0] = ctl->redo[1] = 0;
        fence_barrier_init();
    }
    // Elements past head_dim stay zero: no copy ever writes them.
    if (p.cache.head_dim < kDim)
        for (int at = tid * 16; at < Shape::kQ + kSlots * kTile; at += kPrefixThreads * 16)
            *reinterpret_cast<uint4 *>(smem + at) = make_uint4(0u, 0u, 0u, 0u);
    async_proxy_fence();
    tc_fence_before_sync();
    __syncthreads();
    tc_fence_after_sync();
    const uint32_t tmem = ctl->tmem;
    const PrefixWork work(p);
    griddep_wait();
    // Only now: the own tokens' attention, launched after this kernel, does not wait for its results
    // and reads what the kernels before this one wrote (64 CTAs of a small call leave 88 SMs to it; on an
    // SM with a CTA of this kernel there is no room for one of it, so that with a CTA on every SM it
    // follows, as these end).
    griddep_launch_dependents();

    auto waited = [&](uint64_t *bar, uint32_t parity) {
        return wait_phase(smem_u32(bar), parity, abort_flag, p.status, kKvErrWait, p.wait_limit_ns);
    };
    // The same for a whole warp, whose lanes go on or stop together.
    auto warp_waited = [&](uint64_t *bar, uint32_t parity) { return __all_sync(0xffffffffu, waited(bar, parity)) != 0; };
    // Places [pos, end) in stretches of one unit each, which is counted on (a 64-bit division
    // takes a third of a microsecond, and each role would have several before its first tile).
    auto stretch_end = [&](int64_t unit) {
        const int64_t unit_end = (unit + 1) * work.tiles;
        return unit_end < work.end ? unit_end : work.end;
    };
    const uint32_t row_tiles = static_cast<uint32_t>(p.row_tiles);  // (units stay below 2^31)
    const int rows = static_cast<int>(p.sequences) * p.group;  // of a key head
    // What each role does: all stretches with weights relative to their first tile's maxima; then,
    // once every role is there, the stretches in which that did not do, one by one, with maxima kept
    // tile by tile.  `begin`, its unit and `end`: what is done now; false once there is no more.
    auto flag_of = [&](int64_t unit) {
        const int64_t at = unit - work.unit;
        return at < 63 ? static_cast<int>(at) : 63;
    };
    auto more_work = [&](int64_t &begin, int64_t &unit, int64_t &end, bool &kept) {
        if (!kept) {
            named_barrier(10, kPrefixThreads);
            if (!(ctl->redo[0] | ctl->redo[1])) return false;
            kept = true;
            end = work.pos;
            unit = work.unit - 1;
        }
        while (end < work.end) {
            begin = end;
            end = stretch_end(++unit);
            const int at = flag_of(unit);
            if ((ctl->redo[at >> 5] >> (at & 31)) & 1u) return true;
        }
        return false;
    };

    if (warp >= kPrefixSoftmaxWarps && warp < kPrefixSoftmaxWarps + kPrefixLoadWarps) {
        // ------------------------------------------------------------ loaders
        const int loader = warp - kPrefixSoftmaxWarps;
        constexpr int kElem = kE4m3 ? 1 : 2;
        constexpr int kRowChunks = kDim * kElem / 16;            // 16-byte chunks of a token in the cache
        constexpr int kAtOnce = 32 / kRowChunks < 1 ? 1 : 32 / kRowChunks;  // of them a pass of the warp takes
        static_assert(kRowChunks <= 32, "a lane has one chunk of a row");
        constexpr int kBatch = 4;  // rows whose places are read together (a copy is not moved past such a read)
        const int c = lane % kRowChunks, r_of = lane / kRowChunks;
        const bool mine = c < p.cache.head_dim * kElem / 16;  // a chunk that the cache has
        const uint8_t *k_from = static_cast<const uint8_t *>(p.k_cache) + c * 16, *v_from = static_cast<const uint8_t *>(p.v_cache) + c * 16;
        // Where this lane's token of a tile lies.  Its page is asked for a tile ahead, and the
        // page's number and the place in it go on by additions (a 64-bit division takes a third
        // of a microsecond: with three of them a tile the loaders were what the rest waited for).
        const uint32_t page_size = static_cast<uint32_t>(p.cache.page_size);
        const uint32_t step_pages = kTokens / page_size, step_places = kTokens % page_size;
        int64_t look_tile = 0, look_left = 0;
        uint32_t look_unit = 0;
        uint32_t look_page = 0, look_place = 0;  // of the lane's token of tile look_tile
        auto look_at = [&]() {
            const uint32_t t = static_cast<uint32_t>(look_tile) * kTokens + loader * kMine + lane;
            look_page = t / page_size;
            look_place = t - look_page * page_size;
        };
        int32_t page = -1;          // asked for, of the tile before look_tile
        uint32_t place_of = 0;
        bool inside = false;
        int32_t look_head = 0, head_index = 0;
        auto ask_page = [&]() {
            inside = look_left > 0 && lane < kMine && look_tile * kTokens + loader * kMine + lane < p.prefix;
            page = inside ? p.cache.table[look_page] : -1;
            place_of = look_place;
            head_index = look_head;
            --look_left;
            look_page += step_pages;
            look_place += step_places;
            if (look_place >= page_size) look_place -= page_size, ++look_page;
            if (++look_tile == work.tiles) {
                look_tile = 0;
                look_head = static_cast<int32_t>(++look_unit / row_tiles);
                look_at();
            }
        };
        // The first of places [begin, end), which begin in `unit`.
        auto look_from = [&](int64_t begin, int64_t unit, int64_t end) {
            look_tile = begin - unit * work.tiles, look_unit = static_cast<uint32_t>(unit), look_left = end - begin;
            look_head = static_cast<int32_t>(look_unit / row_tiles);
            look_at();
            ask_page();
        };
        int32_t box_page = 0, box_place = 0, box_head = 0;
        // Leaves what was asked for to the warp, for the tile of number `n`, and asks for the next;
        // returns which tokens exist.
        auto take_page = [&](int64_t n) {
            const bool there = page >= 0 && page < p.cache.num_pages;
            if (inside && !there) atomicOr(p.status, kKvErrPage);
            const int64_t at = there ? (page * p.cache.page_stride + place_of * p.cache.token_stride + head_index * p.cache.head_stride) * kElem : 0;
            const uint32_t bits = __ballot_sync(0xffffffffu, there);
            box_page = page, box_place = static_cast<int32_t>(place_of), box_head = head_index;
            if (p.box == 0 || bits != kAll)
                ctl->row[loader][n & 1][lane] =
                    make_uint4(static_cast<uint32_t>(at), static_cast<uint32_t>(at >> 32), there ? 16u : 0u, 0u);
            ask_page();
            __syncwarp();
            return bits;
        };
        // Where a 16-byte chunk of a row lies in a tile of 64-element blocks, swizzled.
        auto chunk_to = [&](int rows_of, int r, int chunk) {
            return static_cast<uint32_t>((chunk >> 3) * rows_of * 128 + r * 128 + (((chunk & 7) ^ (r & 7)) << 4));
        };
        // This thread's copies are in shared memory, where the tensor core reads them (what TMA
        // brings needs no fence).
        auto copies_done = []() {
            asm volatile("cp.async.wait_all;" ::: "memory");
            async_proxy_fence();
        };
        int64_t n = 0;  // tiles loaded
        int slot = 0;                   // of the ring
        uint32_t phase = 0;
        int segment = 0;
        bool ok = true;
        // 8-bit: raw tiles are on their way kRaws - 1 ahead of the one that is converted.
        int64_t raw_in = 0;
        uint32_t raw_bits = 0;
        uint32_t raw_valid[kE4m3 ? Shape::kRaws / 2 : 1];
        int64_t raw_tiles = 0;
        // This warp's tokens by TMA, a box from each lane that has a box's first token; `block` bytes
        // of a token go to each of `blocks` places `apart` bytes from one another.
        auto load_boxes = [&](const CUtensorMap *map, uint32_t to, uint32_t bar, int blocks, int elements, uint32_t block, uint32_t apart) {
            if (lane == 0) mbar_arrive_expect_tx(bar, static_cast<uint32_t>(blocks) * kMine * block);
            __syncwarp();
            if (lane < kMine && (lane & (p.box - 1)) == 0)
                for (int j = 0; j < blocks; ++j)
                    tma_load_4d(to + j * apart + static_cast<uint32_t>(lane) * block, map, bar, j * elements, box_place, box_head, box_page);
        };
        auto row_offset = [](uint4 row) { return static_cast<int64_t>(static_cast<uint64_t>(row.y) << 32 | row.x); };
        auto ask_raw = [&]() {  // the next raw tile: keys, then values
            if constexpr (kE4m3) {
                if (raw_in >= raw_tiles) return;
                const int which = static_cast<int>(raw_in & 1), at = static_cast<int>(raw_in % Shape::kRaws);
                if (which == 0) {
                    raw_bits = take_page(raw_in >> 1);
#pragma unroll
                    for (int s = 0; s < Shape::kRaws / 2; ++s)
                        if (at / 2 == s) raw_valid[s] = raw_bits;
                }
                const uint32_t to = smem_u32(raws) + static_cast<uint32_t>(at * Shape::kRaw + loader * kMine * kDim);
                const uint32_t bar = smem_u32(&ctl->raw_full[at][loader]);
                if (p.box > 0 && raw_bits == kAll) {
                    load_boxes(which ? &v_map : &k_map, to, bar, 1, 0, kDim, 0);
                    mbar_arrive(bar);
                } else {
                    const uint8_t *from = which ? v_from : k_from;
                    const uint4 *rows_of = ctl->row[loader][(raw_in >> 1) & 1] + r_of;
#pragma unroll
                    for (int i = 0; i < kMine / kAtOnce; i += kBatch) {
                        uint4 row[kBatch];
#pragma unroll
                        for (int j = 0; j < kBatch; ++j) row[j] = rows_of[(i + j) * kAtOnce];
#pragma unroll
                        for (int j = 0; j < kBatch; ++j)
                            if (mine) cp_async16n(to + ((i + j) * kAtOnce + r_of) * kDim + c * 16, from + row_offset(row[j]), row[j].z);
                    }
                    cp_async_arrive(bar);
                    if (lane == 0) mbar_arrive(bar);
                }
                ++raw_in;
            }
        };
        int64_t begin = work.pos, first_unit = work.unit, end = work.end;
        bool kept = false;
        do {
        look_from(begin, first_unit, end);
        raw_tiles += 2 * (end - begin);
        if constexpr (kE4m3)
            for (int i = 0; ok && i < Shape::kRaws - 1; ++i) ask_raw();
        for (int64_t pos = begin, unit = first_unit; ok && pos < end; ++unit) {
            // A row tile's queries, once its predecessor's products are done with the buffer.
            const int64_t seg_end = stretch_end(unit);
            if (segment > 0 && !warp_waited(&ctl->q_empty, static_cast<uint32_t>(segment - 1) & 1u)) {
                ok = false;
                break;
            }
            {
                constexpr int kQChunks = kDim / 8, kStep = kPrefixLoaders / kQChunks;  // chunks of a row; rows between a thread's
                const uint32_t head = static_cast<uint32_t>(unit) / row_tiles, group = p.group;
                const int qc = (tid - 32 * kPrefixSoftmaxWarps) % kQChunks, r0 = (tid - 32 * kPrefixSoftmaxWarps) / kQChunks;
                uint32_t row = (static_cast<uint32_t>(unit) - head * row_tiles) * kPrefixRows + r0, b = row / group, g = row - b * group;
                const uint32_t step_b = kStep / group, step_g = kStep - step_b * group;
                if (qc * 8 < p.cache.head_dim)
#pragma unroll 4
                    for (int r = r0; r < kPrefixRows; r += kStep) {
                        const bool fill = row < static_cast<uint32_t>(rows);
                        cp_async16(smem_u32(smem) + chunk_to(kPrefixRows, r, qc),
                                   p.q + (fill ? b * p.q_stride + (static_cast<int64_t>(head) * group + g) * p.cache.head_dim + qc * 8 : 0), fill);
                        row += kStep, b += step_b, g += step_g;
                        if (g >= group) g -= group, ++b;
                    }
            }
            ++segment;
            bool asked = true;  // the queries are on their way
            for (; ok && pos < seg_end; ++pos, ++n) {
                uint32_t bits = 0;
                if constexpr (!kE4m3) bits = take_page(n);
                for (int which = 0; which < 2; ++which) {
                    if (!warp_waited(&ctl->empty[slot], phase ^ 1u)) {
                        ok = false;
                        break;
                    }
                    const uint32_t to = smem_u32(ring) + slot * kTile;
                    if constexpr (!kE4m3) {
                        const uint32_t bar = smem_u32(&ctl->full[slot]);
                        if (lane == 0 && which == 0) ctl->valid[n & 7][loader] = bits;
                        if (p.box > 0 && bits == kAll) {
                            load_boxes(which ? &v_map : &k_map, to + loader * kMine * 128, bar, (p.cache.head_dim + 63) / 64, 64, 128,
                                       kTokens * 128);
                            mbar_arrive(bar);
                        } else {
                            const uint8_t *from = which ? v_from : k_from;
                            const uint4 *rows_of = ctl->row[loader][n & 1] + r_of;
#pragma unroll
                            for (int i = 0; i < kMine / kAtOnce; i += kBatch) {
                                uint4 row[kBatch];
#pragma unroll
                                for (int j = 0; j < kBatch; ++j) row[j] = rows_of[(i + j) * kAtOnce];
#pragma unroll
                                for (int j = 0; j < kBatch; ++j)
                                    if (mine)
                                        cp_async16n(to + chunk_to(kTokens, loader * kMine + (i + j) * kAtOnce + r_of, c), from + row_offset(row[j]),
                                                    row[j].z);
                            }
                            copies_done();
                            mbar_arrive(bar);
                            if (lane == 0) mbar_arrive(bar);
                        }
                    } else {
                        ask_raw();
                        const int at = static_cast<int>((2 * n + which) % Shape::kRaws);
                        if (!warp_waited(&ctl->raw_full[at][loader], static_cast<uint32_t>((2 * n + which) / Shape::kRaws) & 1u)) {
                            ok = false;
                            break;
                        }
                        if (which == 0) {
#pragma unroll
                            for (int s = 0; s < Shape::kRaws / 2; ++s)
                                if (static_cast<int>(n % (Shape::kRaws / 2)) == s) bits = raw_valid[s];
                            if (lane == 0) ctl->valid[n & 7][loader] = bits;
                        }
                        const uint8_t *from = raws + at * Shape::kRaw;
#pragma unroll
                        for (int i = 0; i < kMine / kAtOnce; ++i) {
                            const int r = loader * kMine + i * kAtOnce + r_of;
                            if (!mine) continue;
                            uint4 lo, hi;
                            e4m3_to_bf16(*reinterpret_cast<const uint4 *>(from + r * kDim + c * 16), lo, hi);
                            *reinterpret_cast<uint4 *>(ring + slot * kTile + chunk_to(kTokens, r, 2 * c)) = lo;
                            *reinterpret_cast<uint4 *>(ring + slot * kTile + chunk_to(kTokens, r, 2 * c + 1)) = hi;
                        }
                        async_proxy_fence();
                        mbar_arrive(smem_u32(&ctl->full[slot]));
                    }
                    // (Only now: the first keys are asked for before the queries are waited for.  Their
                    // slot is freed by products before this stretch's, which no queries hold up.)
                    if (asked) {
                        copies_done();
                        mbar_arrive(smem_u32(&ctl->q_full));
                        asked = false;
                    }
                    if (++slot == kSlots) slot = 0, phase ^= 1u;
                }
            }
        }
        } while (more_work(begin, first_unit, end, kept));
        asm volatile("cp.async.wait_all;" ::: "memory");
    } else if (warp == kPrefixSoftmaxWarps + kPrefixLoadWarps) {
        // ------------------------------------------------------------ products
        // The whole warp runs the loop, so that descriptors and addresses are the same in every
        // lane and stay in uniform registers; one elected lane issues.  (From a branch of one lane
        // each product took about 100 cycles to issue, whatever its width.)
        {
            constexpr uint32_t kIdX = prefix_idesc(kTokens, false), kIdO = prefix_idesc(kDim, true);
            // (The address field of a descriptor, in 16-byte units, holds every offset without a carry.)
            const uint64_t q_desc = smem_desc_sw128(smem_u32(smem), 16, 1024), k_desc = smem_desc_sw128(smem_u32(ring), 16, 1024),
                           v_desc = smem_desc_sw128(smem_u32(ring), kTokens * 128, 1024);
            int64_t begin = work.pos, first_unit = work.unit, end = work.end, xpos = 0, x_seg_end = 0, x_unit = 0;
            bool kept = false;
            int segment = 0, xslot = 0;  // the ring goes keys, values, keys, values ...
            uint32_t xphase = 0;
            auto next = [&](int &slot, uint32_t &phase) {
                if ((slot += 2) >= kSlots) {
                    slot -= kSlots;
                    phase ^= 1u;
                }
            };
            // X of the next place; false once a wait ran out.
            auto issue_x = [&](int64_t n) {
                // (Fault injection: nobody arrives on that barrier.  As any wait that runs out, wherever.)
                if (n == p.fault_place && !warp_waited(&ctl->drain, 0)) return false;
                if (xpos == x_seg_end) {
                    if (!warp_waited(&ctl->q_full, static_cast<uint32_t>(segment) & 1u)) return false;
                    ++segment;
                    x_seg_end = stretch_end(x_unit++);
                }
                if (!warp_waited(&ctl->full[xslot], xphase)) return false;
                tc_fence_after_sync();
                const uint64_t kd = k_desc + static_cast<uint64_t>(xslot) * (kTile >> 4);
                const uint32_t d = tmem + kDim + static_cast<uint32_t>(n & 1) * Shape::kBuffer;
                ++xpos;
                if (elect_one()) {
#pragma unroll
                    for (int k = 0; k < kDim / 16; ++k) {
                        const uint64_t block = static_cast<uint64_t>(k / 4), in = static_cast<uint64_t>(k % 4) * 32;
                        tc_mma<false>(d, q_desc + ((block * kPrefixRows * 128 + in) >> 4), kd + ((block * kTokens * 128 + in) >> 4), kIdX,
                                      k > 0);
                    }
                    tc_commit<false>(smem_u32(&ctl->empty[xslot]));
                    tc_commit<false>(smem_u32(&ctl->x_full[n & 1]));
                    if (xpos == x_seg_end) tc_commit<false>(smem_u32(&ctl->q_empty));
                }
                __syncwarp();
                next(xslot, xphase);
                return true;
            };
            int vslot = 1;
            uint32_t vphase = 0;
            int64_t n = 0;
            bool ok = true;
            do {
            int64_t unit = first_unit, seg_begin = begin, seg_end = stretch_end(unit);
            xpos = x_seg_end = begin;
            x_unit = first_unit;
            ok = ok && issue_x(n);
            for (int64_t pos = begin; ok && pos < end; ++pos, ++n) {
                if (pos == seg_end) {
                    seg_begin = pos;
                    seg_end = stretch_end(++unit);
                }
                if (xpos < end) ok = issue_x(n + 1);
                ok = ok && warp_waited(&ctl->full[vslot], vphase);
                const uint64_t vd = v_desc + static_cast<uint64_t>(vslot) * (kTile >> 4);
                const uint32_t a = tmem + kDim + static_cast<uint32_t>(n & 1) * Shape::kBuffer;
                const uint32_t more = pos > seg_begin;
                // The first half of each piece's tokens, then the second, as P of them is there: the
                // tensor core works on the one while the other is made.
#pragma unroll
                for (int h = 0; ok && h < 2; ++h) {
                    ok = warp_waited(&ctl->p_full[n & 1][h], static_cast<uint32_t>(n >> 1) & 1u);
                    if (!ok) break;
                    tc_fence_after_sync();
                    if (elect_one()) {
#pragma unroll
                        for (int y = 0; y < 3; ++y)
#pragma unroll
                            for (int i = 0; i < kTokens / 32; ++i) {
                                constexpr int kSteps = kPiece / 32;  // 16-token steps of a half
                                const int k = i / kSteps * 2 * kSteps + h * kSteps + i % kSteps;
                                tc_mma_ts(tmem, y < 2 ? a + 16 * k + 8 * y : a + kTokens + 8 * k, vd + k * (2048 >> 4), kIdO,
                                          h > 0 || y > 0 || i > 0 ? 1u : more);
                            }
                        if (h == 1) {
                            tc_commit<false>(smem_u32(&ctl->empty[vslot]));
                            tc_commit<false>(smem_u32(&ctl->o_done[n & 1]));
                        }
                    }
                    __syncwarp();
                }
                next(vslot, vphase);
            }
            } while (more_work(begin, first_unit, end, kept));
            // Every product is done before the tensor memory is given back, whatever happened.
            if (elect_one()) {
                tc_commit<false>(smem_u32(&ctl->drain));
                const uint64_t t0 = globaltimer_ns();
                while (!mbar_try_wait(smem_u32(&ctl->drain), 0) && static_cast<int64_t>(globaltimer_ns() - t0) < kPrefixWaitNs) {
                }
            }
        }
        __syncwarp();
    } else {
        // ------------------------------------------------------------ softmax
        const int quarter = warp & 3, piece = (warp >> 2) % kPrefixPieces, group = warp / (4 * kPrefixPieces);
        const int r = quarter * 32 + lane, share = group * kPrefixPieces + piece;
        const uint32_t at_lane = tmem + (static_cast<uint32_t>(quarter * 32) << 16);
        const uint32_t buffer = at_lane + kDim + group * Shape::kBuffer, x0 = buffer + piece * kPiece;  // of the group's tiles
        // Named barriers: the pieces of a group's rows; all softmax warps.  Every warp comes to the
        // one for every tile of its group and to the other for every stretch, whatever ran out.
        // (The hand-over between the groups is not one: they are not in step, and a barrier that
        // one group had passed twice would take that for the other's arrival.)
        const int own_barrier = 1 + group * 4 + quarter, all_barrier = 9;
        int64_t n = 0, left = 0;  // tiles; bases left before the stretch
        bool ok = true, kept = false;
        int64_t begin = work.pos, first_unit = work.unit, end = work.end;
        do {
        for (int64_t pos = begin, unit = first_unit; pos < end; ++unit) {
            const int64_t seg_first = n, seg_begin = pos, seg_end = stretch_end(unit);
            const uint32_t head = static_cast<uint32_t>(unit) / row_tiles, row = (static_cast<uint32_t>(unit) - head * row_tiles) * kPrefixRows + r;
            const float factor = p.scale * 1.4426950408889634f * (kE4m3 && p.k_scale ? p.k_scale[head] : 1.f);
            const float none = factor < 0.f ? INFINITY : -INFINITY;
            float m = -INFINITY, l = 0.f;  // what this thread's sum is relative to
            bool bad = false;
            for (; pos < seg_end; ++pos, ++n) {
                if (static_cast<int>(n & 1) != group) continue;
                ok = ok && warp_waited(&ctl->x_full[group], static_cast<uint32_t>(n >> 1) & 1u);
                tc_fence_after_sync();
                uint32_t bits[2] = {kAll, kAll};  // tokens of the piece that exist, a loading warp's each
                if (ok) bits[0] = ctl->valid[n & 7][2 * piece], bits[1] = ctl->valid[n & 7][2 * piece + 1];
                if (kept || pos == seg_begin) {
                    // The tile's maxima: of the first tile, or of each where they are kept.
                    float top = none;
                    if (ok) {
#pragma unroll
                        for (int w = 0; w < 2; ++w) {
                            uint32_t x[kMine];
                            tmem_load(x0 + w * kMine, x);
                            if (bits[w] != kAll) {
#pragma unroll
                                for (int i = 0; i < kMine; ++i)
                                    if (!((bits[w] >> i) & 1u)) x[i] = __float_as_uint(none);
                            }
                            if (factor < 0.f) {
#pragma unroll
                                for (int i = 0; i < kMine; i += 2) top = fminf(fminf(__uint_as_float(x[i]), __uint_as_float(x[i + 1])), top);
                            } else {
#pragma unroll
                                for (int i = 0; i < kMine; i += 2) top = fmaxf(fmaxf(__uint_as_float(x[i]), __uint_as_float(x[i + 1])), top);
                            }
                        }
                        top *= factor;
                        ctl->top[group][piece][r] = top;
                    }
                    named_barrier(own_barrier, 32 * kPrefixPieces);
                    const int64_t at = left + (n - seg_first);  // of the bases left
                    if (pos > seg_begin)
                        ok = ok && warp_waited(&ctl->base_full[(at - 1) & 1][quarter], static_cast<uint32_t>((at - 1) >> 1) & 1u);
                    const float before = pos > seg_begin ? ctl->base[(at - 1) & 1][r] : -INFINITY;
                    top = fmaxf(top, ctl->top[group][piece ^ 1][r]);
                    const bool grown = top > before + kLazy || (before == -INFINITY && top > before);
                    const float base_now = grown ? top : before;
                    if (piece == 0) ctl->base[at & 1][r] = base_now;
                    mbar_arrive(smem_u32(&ctl->base_full[at & 1][quarter]));
                    if (!ok) continue;
                    if (base_now != m) {
                        l *= exp2_fast(m - base_now);
                        m = base_now;
                    }
                    bad = bad || m == -INFINITY;  // (no token in the first tile: nothing to be relative to)
                    if (pos > seg_begin && __any_sync(0xffffffffu, grown)) {
                        // o of the tiles before is complete once the last one's product is.  (The
                        // barrier's phase before that ended before X of this tile was there.)
                        ok = warp_waited(&ctl->o_done[(n - 1) & 1], static_cast<uint32_t>((n - 1) >> 1) & 1u);
                        if (!ok) continue;
                        tc_fence_after_sync();
                        const float keep = grown ? exp2_fast(before - m) : 1.f;
#pragma unroll 1
                        for (int d = 0; d < kDim / kPrefixPieces; d += 16) {
                            float o[16];
                            tmem_load16(at_lane + piece * (kDim / kPrefixPieces) + d, o);
#pragma unroll
                            for (int i = 0; i < 16; ++i) o[i] *= keep;
                            tmem_store16(at_lane + piece * (kDim / kPrefixPieces) + d, o);
                        }
                    }
                } else if (n == seg_first + 1) {  // the other group's first tile of the stretch
                    ok = ok && warp_waited(&ctl->base_full[left & 1][quarter], static_cast<uint32_t>(left >> 1) & 1u);
                    if (ok) m = ctl->base[left & 1][r];
                }
                if (!ok) continue;
                const float base = finite_or_zero(m);
                const uint64_t factors = pair_of(factor, factor), bases = pair_of(-base, -base);
                uint64_t sum = pair_of(0.f, 0.f);  // of the tile: no long chain of additions
                // X is read again, 16 tokens at a time in a loop: held in registers it would leave
                // room for half as many warps, and unrolled over the tile the code of the three
                // roles does not stay in the instruction cache (6600 cycles a tile).
#pragma unroll 1
                for (int i = 0; i < kPiece / 16; ++i) {
                    uint32_t x[16], hi_mid[16], lo[8];
                    tmem_load(x0 + 16 * i, x);
                    const uint32_t there = (16 * i < kMine ? bits[0] : bits[1]) >> (16 * i % kMine);
                    float w[16];
#pragma unroll
                    for (int j = 0; j < 8; ++j) {
                        const float2 v = pair_to(fma2(pair_of(__uint_as_float(x[2 * j]), __uint_as_float(x[2 * j + 1])), factors, bases));
                        w[2 * j] = exp2_fast(v.x), w[2 * j + 1] = exp2_fast(v.y);
                    }
                    if ((there & 0xffffu) != 0xffffu) {
#pragma unroll
                        for (int j = 0; j < 16; ++j)
                            if (!((there >> j) & 1u)) w[j] = 0.f;
                    }
#pragma unroll
                    for (int j = 0; j < 8; ++j) {
                        const uint64_t both = pair_of(w[2 * j], w[2 * j + 1]);
                        sum = add2(sum, both);
                        split3(both, hi_mid[j], hi_mid[8 + j], lo[j]);
                    }
                    tmem_store(x0 + 16 * i, hi_mid);
                    tmem_store8(buffer + kTokens + piece * (kPiece / 2) + 8 * i, lo);
                    if (i % (kPiece / 32) == kPiece / 32 - 1) {
                        tmem_store_wait();
                        tc_fence_before_sync();
                        mbar_arrive(smem_u32(&ctl->p_full[group][i / (kPiece / 32)]));
                    }
                }
                const float2 sums = pair_to(sum);
                bad = bad || !(sums.x + sums.y < kMostSum);
                l += sums.x + sums.y;
            }
            // The part: o of every tile of the stretch, relative to the last base, from both groups.
            left += kept ? n - seg_first : 1;
            named_barrier(all_barrier, 32 * kPrefixSoftmaxWarps);
            const float last = ctl->base[(left - 1) & 1][r];
            ok = ok && warp_waited(&ctl->o_done[(n - 1) & 1], static_cast<uint32_t>((n - 1) >> 1) & 1u);
            tc_fence_after_sync();
            if (ok) {
                float *part = p.partials + (unit + blockIdx.x) * Shape::kPart;
                const bool mine = row < static_cast<uint32_t>(rows);
                float none_of = 0.f;  // 0 · o: NaN where o is not finite
                if (mine) {
                    if (share == 0) part[r] = last;
                    part[(1 + share) * kPrefixRows + r] = last != m ? l * exp2_fast(m - last) : l;
                }
                const float by = kE4m3 && p.v_scale ? p.v_scale[head] : 1.f;
                float4 *to = reinterpret_cast<float4 *>(part + (1 + kPrefixSums) * kPrefixRows);
#pragma unroll 1
                for (int d = 0; d < kOwn; d += 16) {
                    const int at = share * kOwn + d;
                    float o[16];
                    tmem_load16(at_lane + at, o);
#pragma unroll
                    for (int i = 0; i < 16; ++i) none_of = __fmaf_rn(0.f, o[i], none_of);
                    if (mine)
#pragma unroll
                        for (int i = 0; i < 4; ++i)
                            to[(at / 4 + i) * kPrefixRows + r] =
                                make_float4(o[4 * i] * by, o[4 * i + 1] * by, o[4 * i + 2] * by, o[4 * i + 3] * by);
                }
                // Weights that come to 2^64 relative to the first tile's maximum, or none to be relative
                // to, or a sum that is not finite, as it may then be of large values: once more, with
                // maxima kept.
                if (!kept && __any_sync(0xffffffffu, mine && (bad || none_of != 0.f)) && lane == 0) {
                    const int at = flag_of(unit);
                    atomicOr(&ctl->redo[at >> 5], 1u << (at & 31));
                }
            } else {
                leave_nan<Shape>(p, unit, share * kPrefixRows + r);
            }
            // No product of the next stretch begins before all of o is read.
            tc_fence_before_sync();
            named_barrier(all_barrier, 32 * kPrefixSoftmaxWarps);
        }
        } while (more_work(begin, first_unit, end, kept));
    }
    tc_fence_before_sync();
    __syncthreads();
    if (warp == kPrefixSoftmaxWarps + kPrefixLoadWarps) {
        if (*abort_flag) {
            // A wait ran out, in whichever role: TMA copies that nobody has waited for may be on their
            // way to this block's memory, those of loaders that came to their end among them.  They
            // land within microseconds; a barrier that not everyone came to does not tell.
            const uint64_t t0 = globaltimer_ns();
            while (globaltimer_ns() - t0 < kPrefixLandNs) {
            }
        }
        tc_fence_after_sync();
        tmem_dealloc<false>(tmem, 512);
    }
}

// The join: eight rows of a key head a block, 128 threads on every kGroups-th part each; then
// the sequences' own part.  Bytes bound it (the parts), and the few loads one after another:
// with a few parts a unit one group of threads has them all on their way, and eight blocks an
// SM (128 sequences behind 32768 tokens, up to four parts a unit, whole call: 224 us and 236
// with four groups; 64 behind 8192, up to six: 81 and 78; the
// prefix's kernel has since become 4 us shorter).
constexpr int kCombineRows = 8, kCombineLanes = 16, kCombineMost = 4;
constexpr int kCombineThreads = kCombineRows * kCombineLanes;  // of a group
constexpr int kCombineFew = 4;  // parts of a unit, at most, for one group

template <int kDim, int kGroups>
__global__ void __launch_bounds__(kCombineThreads *kGroups) kv_combine_kernel(const KvCombineParams p) {
    constexpr int kPart = PrefixShape<false, kDim>::kPart;
    constexpr int kPer = kDim / 4 / kCombineLanes;  // float4s of a thread
    __shared__ float tops[kGroups][kCombineRows], sums[kGroups][kCombineRows];
    __shared__ float4 values[kGroups > 1 ? kGroups - 1 : 1][kDim / 4][kCombineRows];
    griddep_launch_dependents();
    const int tid = threadIdx.x;
    const int i = tid % kCombineRows, c = tid / kCombineRows % kCombineLanes, group = tid / (kCombineRows * kCombineLanes);
    const int rows = static_cast<int>(p.sequences) * p.group;
    const int blocks = (rows + kCombineRows - 1) / kCombineRows;
    const int64_t head = blockIdx.x / blocks;
    const int row0 = static_cast<int>(blockIdx.x % blocks) * kCombineRows, row = row0 + i;
    const int64_t unit = head * p.row_tiles + row0 / kPrefixRows;
    const int r = row % kPrefixRows;
    const bool in = row < rows;
    // CTA of the first and of the last place of the unit: the one whose share holds it.
    const int64_t total = p.kv_heads * p.row_tiles * p.tiles;
    const int64_t c0 = ((unit * p.tiles + 1) * p.ctas - 1) / total, c1 = ((unit + 1) * p.tiles * p.ctas - 1) / total;
    const float *first = p.partials + (unit + c0) * kPart;
    const int parts = static_cast<int>(c1 - c0) + 1;
    // The own tokens' part, asked for beside the prefix's.
    const uint32_t b = in ? static_cast<uint32_t>(row) / p.group : 0u, g = in ? static_cast<uint32_t>(row) % p.group : 0u;
    const int64_t q_head = head * p.group + g, at = static_cast<int64_t>(b) * p.kv_heads * p.group + q_head;
    float2 own = make_float2(-INFINITY, 0.f);
    float4 own_values[kPer];
#pragma unroll
    for (int k = 0; k < kPer; ++k) own_values[k] = make_float4(0.f, 0.f, 0.f, 0.f);
    griddep_wait();
    if (in && group == 0) {
        own = p.top[at];
#pragma unroll
        for (int k = 0; k < kPer; ++k) {
            const int d = 4 * (c + k * kCombineLanes);
            if (d < p.head_dim) own_values[k] = *reinterpret_cast<const float4 *>(p.out32 + at * p.head_dim + d);
        }
    }
    float m = -INFINITY, l = 0.f;
    float4 o[kPer];
#pragma unroll
    for (int k = 0; k < kPer; ++k) o[k] = make_float4(0.f, 0.f, 0.f, 0.f);
    auto add = [&](float top, float sum, const float4 *v) {
        const float all = fmaxf(m, top), base = finite_or_zero(all);
        const float keep = exp2_fast(m - base), w = exp2_fast(top - base);
        m = all;
        l = l * keep + sum * w;
#pragma unroll
        for (int k = 0; k < kPer; ++k) {
            o[k].x = o[k].x * keep + v[k].x * w, o[k].y = o[k].y * keep + v[k].y * w;
            o[k].z = o[k].z * keep + v[k].z * w, o[k].w = o[k].w * keep + v[k].w * w;
        }
    };
    if (in) {
#pragma unroll 4
        for (int x = group; x < parts; x += kGroups) {
            const float *part = first + static_cast<int64_t>(x) * kPart;
            const float4 *from = reinterpret_cast<const float4 *>(part + (1 + kPrefixSums) * kPrefixRows);
            float4 v[kPer];
#pragma unroll
            for (int k = 0; k < kPer; ++k) v[k] = __ldcg(from + (c + k * kCombineLanes) * kPrefixRows + r);
            float sum = 0.f;
#pragma unroll
            for (int k = 1; k <= kPrefixSums; ++k) sum += __ldcg(part + k * kPrefixRows + r);
            add(__ldcg(part + r), sum, v);
        }
    }
    if (group > 0) {
        if (c == 0) tops[group][i] = m, sums[group][i] = l;
#pragma unroll
        for (int k = 0; k < kPer; ++k) values[group - 1][c + k * kCombineLanes][i] = o[k];
    }
    __syncthreads();
    if (group > 0 || !in) return;
#pragma unroll
    for (int x = 1; x < kGroups; ++x) {
        float4 v[kPer];
#pragma unroll
        for (int k = 0; k < kPer; ++k) v[k] = values[x - 1][c + k * kCombineLanes][i];
        add(tops[x][i], sums[x][i], v);
    }
    if (own.y != 0.f) {  // (the own tokens' values are divided by their sum; without tokens they are not written)
#pragma unroll
        for (int k = 0; k < kPer; ++k)
            own_values[k].x *= own.y, own_values[k].y *= own.y, own_values[k].z *= own.y, own_values[k].w *= own.y;
        add(own.x, own.y, own_values);
    }
    const float inv = l == 0.f ? 0.f : 1.f / l;
#pragma unroll
    for (int k = 0; k < kPer; ++k) {
        const int d = 4 * (c + k * kCombineLanes);
        if (d < p.head_dim)
            *reinterpret_cast<uint2 *>(p.out + b * p.out_stride + q_head * p.head_dim + d) =
                make_uint2(bf16_pair(o[k].x * inv, o[k].y * inv), bf16_pair(o[k].z * inv, o[k].w * inv));
    }
    if (p.lse && c == 0) p.lse[at] = l == 0.f ? -INFINITY : (m + log2f(l)) * 0.6931471805599453f;
}

}  // namespace dev
}  // namespace projgb
