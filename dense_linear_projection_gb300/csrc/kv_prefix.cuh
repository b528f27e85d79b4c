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
//   * warps 0..7 turn X into P: a thread has one row (tensor-memory lane) and half
//     of a tile's tokens; two threads of a row meet over its maximum.
//   * o is rescaled only where the maximum grows by more than 2^8 (kLazy): a
//     weight then is at most 2^8, which costs fp32 sums nothing.
//   * warps 8..11 fill a ring of token tiles (16-byte asynchronous copies: a page may
//     have any number of tokens and any strides), warp 12 issues the products.
//   * (key head, row tile, token tile) in this order are one line that the CTAs share
//     evenly; each stretch of one row tile leaves a part in the workspace.
//
// Every wait is bounded; one that runs out records itself, and the CTA drains its
// copies, frees its tensor memory and returns.
#pragma once

#include "kv_attend.cuh"

namespace projgb {
namespace dev {

constexpr int kPrefixRows = 128;          // query rows of a tile
constexpr int kPrefixSoftmaxWarps = 8, kPrefixLoadWarps = 4;
constexpr int kPrefixLoaders = 32 * kPrefixLoadWarps;
constexpr int kPrefixThreads = 32 * (kPrefixSoftmaxWarps + kPrefixLoadWarps + 1);
constexpr float kLazy = 8.f;
constexpr int64_t kPrefixWaitNs = 1000000000;

template <bool kE4m3, int kDim>
struct PrefixShape {
    static constexpr int kTokens = kDim > 128 ? 64 : 128;  // of a tile
    static constexpr int kTile = kTokens * kDim * 2;        // bytes of a tile of keys or values, bf16
    static constexpr int kRaw = kE4m3 ? kTile / 2 : 0;      // as they are in an 8-bit cache
    static constexpr int kSlots = kE4m3 ? 4 : kDim > 128 ? 5 : 6;
    static constexpr int kRaws = kE4m3 ? (kDim > 128 ? 2 : 4) : 0;
    static constexpr int kQ = kPrefixRows * kDim * 2;
    static constexpr int kCtl = 2048;
    static constexpr int kSmem = kQ + kSlots * kTile + kRaws * kRaw + kCtl;
    // Tensor memory: o, then two buffers of X, each with room for P's three parts.
    static constexpr int kBuffer = kTokens / 2 * 3;
    static constexpr int kColumns = kDim + 2 * kBuffer;
    // A part: [maximum of a row][sum of either half of its tokens][kDim/4][row] float4.
    static constexpr int kPart = 3 * kPrefixRows + kPrefixRows * kDim;
    static_assert(kColumns <= 512 && kSmem <= 227 * 1024, "tensor memory and shared memory of an SM");
};

struct PrefixCtl {
    uint64_t full[8], empty[8], q_full, q_empty, x_full[2], p_full[2], o_done[2], drain;
    uint32_t tmem;
    int abort_flag;
    uint32_t valid[8][4];     // tokens of the last tiles that exist, a bit each
    float top[2][kPrefixRows];  // a row's maximum over the other half of the tile, and of the next one
};
static_assert(sizeof(PrefixCtl) <= 2048, "PrefixShape::kCtl");

// D[tmem] (+)= A[tmem] · B[smem], bf16, fp32 accumulators.
__device__ __forceinline__ void tc_mma_ts(uint32_t d_tmem, uint32_t a_tmem, uint64_t b_desc, uint32_t idesc, uint32_t accumulate) {
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d_tmem),
        "r"(a_tmem), "l"(b_desc), "r"(idesc), "r"(accumulate)
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
__device__ __forceinline__ void tmem_store_wait() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }
__device__ __forceinline__ void async_proxy_fence() { asm volatile("fence.proxy.async.shared::cta;" ::: "memory"); }
// Arrives on `bar` once the thread's copies so far are in shared memory.
__device__ __forceinline__ void cp_async_arrive(uint32_t bar) {
    asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(bar) : "memory");
}
__device__ __forceinline__ void named_barrier(int id, int threads) {
    asm volatile("bar.sync %0, %1;" ::"r"(id), "r"(threads) : "memory");
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
    int64_t pos, end, tiles;  // places; token tiles of a unit
    __device__ __forceinline__ PrefixWork(const KvPrefixParams &p) {
        const int64_t total = p.cache.kv_heads * p.row_tiles * p.tiles;
        pos = total * blockIdx.x / gridDim.x;
        end = total * (blockIdx.x + 1) / gridDim.x;
        tiles = p.tiles;
    }
};

template <bool kE4m3, int kDim>
__global__ void __launch_bounds__(kPrefixThreads, 1) kv_prefix_kernel(const KvPrefixParams p) {
    using Shape = PrefixShape<kE4m3, kDim>;
    constexpr int kTokens = Shape::kTokens, kTile = Shape::kTile, kSlots = Shape::kSlots;
    constexpr int kHalf = kTokens / 2;  // tokens of a softmax thread
    extern __shared__ __align__(1024) uint8_t smem[];
    uint8_t *ring = smem + Shape::kQ, *raws = ring + kSlots * kTile;
    PrefixCtl *ctl = reinterpret_cast<PrefixCtl *>(raws + Shape::kRaws * Shape::kRaw);
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    volatile int *abort_flag = &ctl->abort_flag;
    if (smem_u32(smem) & 1023u) {  // (128-byte swizzled tiles; the same in every thread)
        if (tid == 0) atomicOr(p.status, kKvErrWait);
        return;
    }
    griddep_launch_dependents();
    if (warp == kPrefixSoftmaxWarps + kPrefixLoadWarps) {
        tmem_alloc<false>(smem_u32(&ctl->tmem), 512);
        tmem_relinquish<false>();
    }
    if (tid == 0) {
        for (int i = 0; i < kSlots; ++i) {
            // (A copying loader arrives when its copies do; its warp once more, for `valid`.)
            mbar_init(smem_u32(&ctl->full[i]), kE4m3 ? kPrefixLoaders : kPrefixLoaders + kPrefixLoadWarps);
            mbar_init(smem_u32(&ctl->empty[i]), 1);
        }
        mbar_init(smem_u32(&ctl->q_full), kPrefixLoaders);
        mbar_init(smem_u32(&ctl->q_empty), 1);
        for (int i = 0; i < 2; ++i) {
            mbar_init(smem_u32(&ctl->x_full[i]), 1);
            mbar_init(smem_u32(&ctl->p_full[i]), 32 * kPrefixSoftmaxWarps);
            mbar_init(smem_u32(&ctl->o_done[i]), 1);
        }
        mbar_init(smem_u32(&ctl->drain), 1);
        ctl->abort_flag = 0;
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
    griddep_wait();

    const PrefixWork work(p);
    auto waited = [&](uint64_t *bar, uint32_t parity) {
        return wait_phase(smem_u32(bar), parity, abort_flag, p.status, kKvErrWait, kPrefixWaitNs);
    };
    // The same for a whole warp, whose lanes go on or stop together.
    auto warp_waited = [&](uint64_t *bar, uint32_t parity) { return __all_sync(0xffffffffu, waited(bar, parity)) != 0; };
    // Places [pos, end) in stretches of one unit.
    auto stretch_end = [&](int64_t pos) {
        const int64_t unit_end = (pos / work.tiles + 1) * work.tiles;
        return unit_end < work.end ? unit_end : work.end;
    };
    const int rows = static_cast<int>(p.sequences) * p.group;  // of a key head

    if (warp >= kPrefixSoftmaxWarps && warp < kPrefixSoftmaxWarps + kPrefixLoadWarps) {
        // ------------------------------------------------------------ loaders
        const int loader = warp - kPrefixSoftmaxWarps;
        constexpr int kElem = kE4m3 ? 1 : 2;
        constexpr int kRowChunks = kDim * kElem / 16;            // 16-byte chunks of a token in the cache
        constexpr int kMine = kTokens / kPrefixLoadWarps;        // tokens of a warp
        constexpr int kAtOnce = 32 / kRowChunks < 1 ? 1 : 32 / kRowChunks;  // of them a pass of the warp takes
        static_assert(kRowChunks <= 32, "a lane has one chunk of a row");
        const int chunks = p.cache.head_dim * kElem / 16;
        const int c = lane % kRowChunks, r_of = lane / kRowChunks;
        const uint8_t *caches[2] = {static_cast<const uint8_t *>(p.k_cache), static_cast<const uint8_t *>(p.v_cache)};
        // The places of this warp's tokens of a tile, asked for a tile ahead.
        int64_t place = 0;
        bool there = false;
        auto look_up = [&](int64_t pos) {
            there = false;
            if (pos >= work.end) return;
            const int64_t tile = pos % work.tiles, unit = pos / work.tiles;
            const int64_t t = tile * kTokens + loader * kMine + lane;
            if (lane < kMine && t < p.prefix) {
                const uint32_t at = static_cast<uint32_t>(t), page_size = static_cast<uint32_t>(p.cache.page_size);
                const int32_t page = p.cache.table[at / page_size];
                there = page >= 0 && page < p.cache.num_pages;
                if (!there) atomicOr(p.status, kKvErrPage);
                place = page * p.cache.page_stride + (at % page_size) * p.cache.token_stride +
                        unit / p.row_tiles * p.cache.head_stride;
            }
        };
        look_up(work.pos);
        // Where a 16-byte chunk of a row lies in a tile of 64-element blocks, swizzled.
        auto chunk_to = [&](int rows_of, int r, int chunk) {
            return static_cast<uint32_t>((chunk >> 3) * rows_of * 128 + r * 128 + (((chunk & 7) ^ (r & 7)) << 4));
        };
        int64_t n = 0, pos = work.pos;  // tiles loaded; their line
        int slot = 0;                   // of the ring
        uint32_t phase = 0;
        int segment = 0;
        bool ok = true;
        // 8-bit: raw tiles are on their way kRaws - 1 ahead of the one that is converted.
        int64_t raw_in = 0, raw_pos = work.pos;
        uint32_t raw_valid[kE4m3 ? Shape::kRaws / 2 : 1];
        const int64_t raw_tiles = 2 * (work.end - work.pos);
        auto ask_raw = [&]() {  // the next raw tile: keys, then values, of raw_pos
            if constexpr (kE4m3) {
                if (raw_in < raw_tiles) {
                    const int which = static_cast<int>(raw_in & 1);
                    const uint32_t bits = __ballot_sync(0xffffffffu, there);
                    const uint32_t to = smem_u32(raws) + static_cast<uint32_t>(raw_in % Shape::kRaws) * Shape::kRaw;
#pragma unroll
                    for (int i = 0; i < kMine / kAtOnce; ++i) {
                        const int r = i * kAtOnce + r_of;
                        const int64_t at = __shfl_sync(0xffffffffu, place, r) + c * 16;
                        const bool fill = (bits >> r) & 1u;
                        cp_async16(to + (loader * kMine + r) * kDim + c * 16, caches[which] + (fill && c < chunks ? at : 0), fill && c < chunks);
                    }
                    if (which == 0) {
#pragma unroll
                        for (int s = 0; s < Shape::kRaws / 2; ++s)
                            if (static_cast<int>((raw_in / 2) % (Shape::kRaws / 2)) == s) raw_valid[s] = bits;
                    } else {
                        look_up(++raw_pos);
                    }
                    ++raw_in;
                }
                cp_async_commit();
            }
        };
        if constexpr (kE4m3)
            for (int i = 0; i < Shape::kRaws - 1; ++i) ask_raw();

        while (ok && pos < work.end) {
            // A row tile's queries, once its predecessor's products are done with the buffer.
            const int64_t unit = pos / work.tiles, seg_end = stretch_end(pos);
            if (segment > 0 && !warp_waited(&ctl->q_empty, static_cast<uint32_t>(segment - 1) & 1u)) break;
            {
                const int64_t head = unit / p.row_tiles, row0 = unit % p.row_tiles * kPrefixRows;
                constexpr int kQChunks = kDim / 8;
                for (int i = tid - 32 * kPrefixSoftmaxWarps; i < kPrefixRows * kQChunks; i += kPrefixLoaders) {
                    const int r = i / kQChunks, qc = i % kQChunks;
                    const int64_t row = row0 + r;
                    if (qc * 8 >= p.cache.head_dim) continue;
                    const bool fill = row < rows;
                    const uint32_t b = static_cast<uint32_t>(row) / p.group, g = static_cast<uint32_t>(row) % p.group;
                    cp_async16(smem_u32(smem) + chunk_to(kPrefixRows, r, qc),
                               p.q + (fill ? b * p.q_stride + (head * p.group + g) * p.cache.head_dim + qc * 8 : 0), fill);
                }
                cp_async_arrive(smem_u32(&ctl->q_full));
                if constexpr (kE4m3) cp_async_commit();
            }
            ++segment;
            for (; ok && pos < seg_end; ++pos, ++n) {
                uint32_t bits = 0;
                for (int which = 0; which < 2; ++which) {
                    if (!warp_waited(&ctl->empty[slot], phase ^ 1u)) {
                        ok = false;
                        break;
                    }
                    const uint32_t to = smem_u32(ring) + slot * kTile;
                    if constexpr (!kE4m3) {
                        bits = __ballot_sync(0xffffffffu, there);
#pragma unroll
                        for (int i = 0; i < kMine / kAtOnce; ++i) {
                            const int r = i * kAtOnce + r_of;
                            const int64_t at = __shfl_sync(0xffffffffu, place, r) * 2 + c * 16;
                            const bool fill = (bits >> r) & 1u;
                            if (c < chunks)
                                cp_async16(to + chunk_to(kTokens, loader * kMine + r, c), caches[which] + (fill ? at : 0), fill);
                        }
                        cp_async_arrive(smem_u32(&ctl->full[slot]));
                        if (lane == 0) {
                            if (which == 0) ctl->valid[n & 7][loader] = bits;
                            mbar_arrive(smem_u32(&ctl->full[slot]));
                        }
                        if (which == 1) look_up(pos + 1);
                    } else {
                        // This lane's own chunks of the raw tile are in: every copy but the
                        // kRaws - 1 asked for after it (a row tile's queries count as one more).
                        ask_raw();
                        cp_async_wait<Shape::kRaws - 1>();
                        if (which == 0) {
#pragma unroll
                            for (int s = 0; s < Shape::kRaws / 2; ++s)
                                if (static_cast<int>(n % (Shape::kRaws / 2)) == s) bits = raw_valid[s];
                            if (lane == 0) ctl->valid[n & 7][loader] = bits;
                        }
                        const uint8_t *from = raws + (2 * n + which) % Shape::kRaws * Shape::kRaw;
#pragma unroll
                        for (int i = 0; i < kMine / kAtOnce; ++i) {
                            const int r = loader * kMine + i * kAtOnce + r_of;
                            if (c >= chunks) continue;
                            uint4 lo, hi;
                            e4m3_to_bf16(*reinterpret_cast<const uint4 *>(from + r * kDim + c * 16), lo, hi);
                            *reinterpret_cast<uint4 *>(ring + slot * kTile + chunk_to(kTokens, r, 2 * c)) = lo;
                            *reinterpret_cast<uint4 *>(ring + slot * kTile + chunk_to(kTokens, r, 2 * c + 1)) = hi;
                        }
                        async_proxy_fence();
                        mbar_arrive(smem_u32(&ctl->full[slot]));
                    }
                    if (++slot == kSlots) slot = 0, phase ^= 1u;
                }
            }
        }
        cp_async_wait<0>();
        asm volatile("cp.async.wait_all;" ::: "memory");
    } else if (warp == kPrefixSoftmaxWarps + kPrefixLoadWarps) {
        // ------------------------------------------------------------ products
        if (lane == 0) {
            constexpr uint32_t kIdX = prefix_idesc(kTokens, false), kIdO = prefix_idesc(kDim, true);
            const uint32_t q0 = smem_u32(smem), ring0 = smem_u32(ring);
            int64_t pos = work.pos, seg_end = pos < work.end ? stretch_end(pos) : pos;
            int segment = 0, xslot = 0;  // the ring goes keys, values, keys, values ...
            uint32_t xphase = 0;
            auto next = [&](int &slot, uint32_t &phase) {
                if ((slot += 2) >= kSlots) {
                    slot -= kSlots;
                    phase ^= 1u;
                }
            };
            int64_t xpos = pos;
            int64_t x_seg_end = seg_end;
            bool x_first = true;
            // X of the next place; false once a wait ran out.
            auto issue_x = [&](int64_t n) {
                if (x_first) {
                    if (!waited(&ctl->q_full, static_cast<uint32_t>(segment) & 1u)) return false;
                    ++segment;
                    x_first = false;
                }
                if (!waited(&ctl->full[xslot], xphase)) return false;
                async_proxy_fence();
                tc_fence_after_sync();
                const uint32_t k0 = ring0 + xslot * kTile;
                const uint32_t d = tmem + kDim + static_cast<uint32_t>(n & 1) * Shape::kBuffer;
#pragma unroll
                for (int k = 0; k < kDim / 16; ++k) {
                    const uint32_t block = static_cast<uint32_t>(k / 4), in = static_cast<uint32_t>(k % 4) * 32;
                    tc_mma<false>(d, smem_desc_sw128(q0 + block * kPrefixRows * 128 + in, 16, 1024),
                                  smem_desc_sw128(k0 + block * kTokens * 128 + in, 16, 1024), kIdX, k > 0);
                }
                tc_commit<false>(smem_u32(&ctl->empty[xslot]));
                tc_commit<false>(smem_u32(&ctl->x_full[n & 1]));
                next(xslot, xphase);
                if (++xpos == x_seg_end && xpos < work.end) {
                    tc_commit<false>(smem_u32(&ctl->q_empty));
                    x_seg_end = stretch_end(xpos);
                    x_first = true;
                }
                return true;
            };
            int vslot = 1;
            uint32_t vphase = 0;
            int64_t n = 0, seg_begin = pos;
            bool ok = pos < work.end && issue_x(0);
            for (; ok && pos < work.end; ++pos, ++n) {
                if (pos == seg_end) {
                    seg_begin = pos;
                    seg_end = stretch_end(pos);
                }
                if (xpos < work.end && !issue_x(n + 1)) break;
                if (!waited(&ctl->p_full[n & 1], static_cast<uint32_t>(n >> 1) & 1u)) break;
                if (!waited(&ctl->full[vslot], vphase)) break;
                async_proxy_fence();
                tc_fence_after_sync();
                const uint32_t v0 = ring0 + vslot * kTile;
                const uint32_t a = tmem + kDim + static_cast<uint32_t>(n & 1) * Shape::kBuffer;
#pragma unroll
                for (int y = 0; y < 3; ++y)
#pragma unroll
                    for (int k = 0; k < kTokens / 16; ++k)
                        tc_mma_ts(tmem, a + y * (kTokens / 2) + k * 8, smem_desc_sw128(v0 + k * 2048, kTokens * 128, 1024), kIdO,
                                  pos > seg_begin || y > 0 || k > 0);
                tc_commit<false>(smem_u32(&ctl->empty[vslot]));
                tc_commit<false>(smem_u32(&ctl->o_done[n & 1]));
                next(vslot, vphase);
            }
            // Every product is done before the tensor memory is given back, whatever happened.
            tc_commit<false>(smem_u32(&ctl->drain));
            const uint64_t t0 = globaltimer_ns();
            while (!mbar_try_wait(smem_u32(&ctl->drain), 0) && static_cast<int64_t>(globaltimer_ns() - t0) < kPrefixWaitNs) {
            }
        }
        __syncwarp();
    } else {
        // ------------------------------------------------------------ softmax
        const int quarter = warp & 3, half = warp >> 2;
        const int r = quarter * 32 + lane;
        const uint32_t at_lane = tmem + (static_cast<uint32_t>(quarter * 32) << 16);
        int64_t n = 0;
        bool ok = true;
        for (int64_t pos = work.pos; pos < work.end;) {
            const int64_t unit = pos / work.tiles, seg_begin = pos, seg_end = stretch_end(pos);
            const int64_t head = unit / p.row_tiles, row = unit % p.row_tiles * kPrefixRows + r;
            const float factor = p.scale * 1.4426950408889634f * (kE4m3 && p.k_scale ? p.k_scale[head] : 1.f);
            float m = -INFINITY, l = 0.f;
            for (; pos < seg_end; ++pos, ++n) {
                const int buf = static_cast<int>(n & 1);
                const uint32_t x0 = at_lane + kDim + buf * Shape::kBuffer;
                ok = ok && warp_waited(&ctl->x_full[buf], static_cast<uint32_t>(n >> 1) & 1u);
                tc_fence_after_sync();
                float x[kHalf], top = -INFINITY;
                if (ok) {
                    if constexpr (kHalf == 64) {
                        tmem_load64(x0 + half * kHalf, x);
                    } else {
#pragma unroll
                        for (int i = 0; i < kHalf / 16; ++i)
                            tmem_load16(x0 + half * kHalf + 16 * i, *reinterpret_cast<float(*)[16]>(x + 16 * i));
                    }
#pragma unroll
                    for (int i = 0; i < kHalf; ++i) x[i] *= factor;
                    // Tokens of the half, in two words (of a loader warp's tokens each).
#pragma unroll
                    for (int w = 0; w < 2; ++w) {
                        constexpr int kBits = kTokens / kPrefixLoadWarps;
                        const uint32_t bits = ctl->valid[n & 7][half * 2 + w];
                        if (bits != (kBits == 32 ? 0xffffffffu : 0xffffu)) {
#pragma unroll
                            for (int i = 0; i < kBits; ++i)
                                if (!((bits >> i) & 1u)) x[w * kBits + i] = -INFINITY;
                        }
                    }
                    top = x[0];
#pragma unroll
                    for (int i = 1; i < kHalf; ++i) top = fmaxf(top, x[i]);
                    ctl->top[half][r] = top;
                }
                // Both halves of a row have read X, which P overwrites, and left their
                // maxima.  (Every warp comes here for every tile, whatever ran out.)
                tc_fence_before_sync();
                named_barrier(1 + quarter, 64);
                tc_fence_after_sync();
                top = fmaxf(top, ctl->top[half ^ 1][r]);
                named_barrier(1 + quarter, 64);
                if (!ok) continue;
                const bool grown = top > m + kLazy || (m == -INFINITY && top > m);
                const float before = m;
                if (grown) m = top;
                if (__any_sync(0xffffffffu, grown)) {
                    const float keep = grown ? exp2_fast(before - m) : 1.f;
                    l *= keep;
                    if (pos > seg_begin) {
                        // o of the tiles before is complete once the last one's product is.  (The
                        // barrier's phase before that ended two tiles ago, before X that was read then.)
                        ok = warp_waited(&ctl->o_done[(n - 1) & 1], static_cast<uint32_t>((n - 1) >> 1) & 1u);
                        if (!ok) continue;
                        tc_fence_after_sync();
#pragma unroll 1
                        for (int d = 0; d < kDim / 2; d += 16) {
                            float o[16];
                            tmem_load16(at_lane + half * (kDim / 2) + d, o);
#pragma unroll
                            for (int i = 0; i < 16; ++i) o[i] *= keep;
                            tmem_store16(at_lane + half * (kDim / 2) + d, o);
                        }
                    }
                }
                const float base = finite_or_zero(m);
                float sum[2] = {0.f, 0.f};  // of the tile: no long chain of additions
#pragma unroll
                for (int i = 0; i < kHalf; i += 16) {
                    uint32_t part[3][8];
#pragma unroll
                    for (int j = 0; j < 8; ++j) {
                        const float a = exp2_fast(x[i + 2 * j] - base), b = exp2_fast(x[i + 2 * j + 1] - base);
                        sum[0] += a;
                        sum[1] += b;
                        const WeightParts<false> s = split<false>(a, b);
#pragma unroll
                        for (int y = 0; y < 3; ++y) part[y][j] = s.part[y];
                    }
#pragma unroll
                    for (int y = 0; y < 3; ++y) tmem_store8(x0 + y * (kTokens / 2) + half * (kHalf / 2) + i / 2, part[y]);
                }
                l += sum[0] + sum[1];
                tmem_store_wait();
                tc_fence_before_sync();
                mbar_arrive(smem_u32(&ctl->p_full[buf]));
            }
            // The part: o of every tile of the stretch.
            ok = ok && warp_waited(&ctl->o_done[(n - 1) & 1], static_cast<uint32_t>((n - 1) >> 1) & 1u);
            if (!ok) continue;
            tc_fence_after_sync();
            float *part = p.partials + (unit + blockIdx.x) * Shape::kPart;
            const bool mine = row < rows;
            if (mine) {
                if (half == 0) part[r] = m;
                part[(1 + half) * kPrefixRows + r] = l;
            }
            const float by = kE4m3 && p.v_scale ? p.v_scale[head] : 1.f;
            float4 *to = reinterpret_cast<float4 *>(part + 3 * kPrefixRows);
#pragma unroll 1
            for (int d = 0; d < kDim / 2; d += 16) {
                const int at = half * (kDim / 2) + d;
                float o[16];
                tmem_load16(at_lane + at, o);
                if (mine)
#pragma unroll
                    for (int i = 0; i < 4; ++i)
                        to[(at / 4 + i) * kPrefixRows + r] =
                            make_float4(o[4 * i] * by, o[4 * i + 1] * by, o[4 * i + 2] * by, o[4 * i + 3] * by);
            }
            tc_fence_before_sync();
        }
    }
    tc_fence_before_sync();
    __syncthreads();
    if (warp == kPrefixSoftmaxWarps + kPrefixLoadWarps) {
        tc_fence_after_sync();
        tmem_dealloc<false>(tmem, 512);
    }
}

// The join: eight rows of a key head a block, its four groups of threads on every
// fourth part each; then the sequences' own part.  Bytes bound it (the parts).
constexpr int kCombineRows = 8, kCombineLanes = 16, kCombineGroups = 4;
constexpr int kCombineThreads = kCombineRows * kCombineLanes * kCombineGroups;

template <int kDim>
__global__ void __launch_bounds__(kCombineThreads) kv_combine_kernel(const KvCombineParams p) {
    constexpr int kPart = PrefixShape<false, kDim>::kPart;
    constexpr int kPer = kDim / 4 / kCombineLanes;  // float4s of a thread
    __shared__ float tops[kCombineGroups][kCombineRows], sums[kCombineGroups][kCombineRows];
    __shared__ float4 values[kCombineGroups - 1][kDim / 4][kCombineRows];
    griddep_launch_dependents();
    griddep_wait();
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
        for (int x = group; x < parts; x += kCombineGroups) {
            const float *part = first + static_cast<int64_t>(x) * kPart;
            const float4 *from = reinterpret_cast<const float4 *>(part + 3 * kPrefixRows);
            float4 v[kPer];
#pragma unroll
            for (int k = 0; k < kPer; ++k) v[k] = __ldcg(from + (c + k * kCombineLanes) * kPrefixRows + r);
            add(__ldcg(part + r), __ldcg(part + kPrefixRows + r) + __ldcg(part + 2 * kPrefixRows + r), v);
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
    for (int x = 1; x < kCombineGroups; ++x) {
        float4 v[kPer];
#pragma unroll
        for (int k = 0; k < kPer; ++k) v[k] = values[x - 1][c + k * kCombineLanes][i];
        add(tops[x][i], sums[x][i], v);
    }
    const uint32_t b = static_cast<uint32_t>(row) / p.group, g = static_cast<uint32_t>(row) % p.group;
    const int64_t q_head = head * p.group + g, at = static_cast<int64_t>(b) * p.kv_heads * p.group + q_head;
    const float2 own = p.top[at];
    if (own.y != 0.f) {  // (the own tokens' values are divided by their sum)
        float4 v[kPer];
#pragma unroll
        for (int k = 0; k < kPer; ++k) {
            const int d = 4 * (c + k * kCombineLanes);
            v[k] = make_float4(0.f, 0.f, 0.f, 0.f);
            if (d < p.head_dim) v[k] = *reinterpret_cast<const float4 *>(p.out32 + at * p.head_dim + d);
            v[k].x *= own.y, v[k].y *= own.y, v[k].z *= own.y, v[k].w *= own.y;
        }
        add(own.x, own.y, v);
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
