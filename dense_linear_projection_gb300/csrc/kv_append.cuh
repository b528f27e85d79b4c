// Device code of the paged key-value cache's append: rotary position and write.
#pragma once

#include <cuda_fp8.h>

#include "kv_internal.h"
#include "proj_kernel.cuh"
#include "proj_warp.cuh"

namespace projgb {
namespace dev {

// Append.  A unit is 16 elements of one head of one token: eight rotary pairs
// (kVec: two 16-byte loads, either 8 + 8 elements of the two halves or 16 in a
// row), or 16 elements that are only copied.  A thread takes the same unit of
// several heads, so its cosines and sines are read once.  Blocks of 128 threads:
// 8191 tokens of 96 heads took 67.6 us (89 % of the copy bandwidth), with 256
// threads 73.6 and 512 101; asking for two or more heads ahead was slower.  The rotation uses
// separate fp32 products and sums (no fused multiply-add): the value rounded to
// the cache's type is the formula's own.  Bytes bound it: each row is read and
// written once.
constexpr int kAppendThreads = 128;

__device__ __forceinline__ void unpack8(uint4 v, float *x) {
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        x[2 * i] = __uint_as_float(w[i] << 16);
        x[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
    }
}

__device__ __forceinline__ uint8_t to_e4m3(float x, float scale) {
    const float y = fminf(fmaxf(__fdiv_rn(x, scale), -448.f), 448.f);
    // fmaxf and fminf drop a NaN; the cache keeps it.
    return __nv_cvt_float_to_fp8(x != x ? x : y, __NV_SATFINITE, __NV_E4M3);
}

// Elements [at, at + 8) of a head, as bf16 or e4m3.
template <bool kE4m3>
__device__ __forceinline__ void store8(void *to, int64_t at, const float *x, float scale) {
    if constexpr (kE4m3) {
        uint32_t w[2] = {0, 0};
#pragma unroll
        for (int i = 0; i < 8; ++i) w[i / 4] |= static_cast<uint32_t>(to_e4m3(x[i], scale)) << (8 * (i % 4));
        *reinterpret_cast<uint2 *>(static_cast<uint8_t *>(to) + at) = make_uint2(w[0], w[1]);
    } else {
        *reinterpret_cast<uint4 *>(static_cast<uint16_t *>(to) + at) =
            make_uint4(bf16_pair(x[0], x[1]), bf16_pair(x[2], x[3]), bf16_pair(x[4], x[5]), bf16_pair(x[6], x[7]));
    }
}

template <bool kE4m3>
__device__ __forceinline__ void store1(void *to, int64_t at, float x, float scale) {
    if constexpr (kE4m3)
        static_cast<uint8_t *>(to)[at] = to_e4m3(x, scale);
    else
        static_cast<__nv_bfloat16 *>(to)[at] = __float2bfloat16_rn(x);
}

__device__ __forceinline__ void rotate(float &a, float &b, float cos, float sin) {
    const float u = __fsub_rn(__fmul_rn(a, cos), __fmul_rn(b, sin));
    b = __fadd_rn(__fmul_rn(b, cos), __fmul_rn(a, sin));
    a = u;
}

template <bool kE4m3, bool kInterleaved, bool kVec>
__global__ void __launch_bounds__(kAppendThreads) kv_append_kernel(const KvAppendParams p) {
    griddep_launch_dependents();
    griddep_wait();
    const KvCacheView &c = p.cache;
    const int64_t token = blockIdx.x;
    const int half = p.rot_dim / 2;
    const int pair_units = (half + 7) / 8, units = pair_units + (c.head_dim - p.rot_dim + 15) / 16;
    const int slots = kAppendThreads / units;  // heads a block takes at a time
    const int unit = threadIdx.x % units, slot = threadIdx.x / units;
    if (slot >= slots) return;
    const int64_t pos = p.positions[token];
    const int64_t seq = p.seq_ids ? p.seq_ids[token] : token;

    const bool rotary = unit < pair_units;
    const int j0 = 8 * unit;                              // first rotary pair
    const int d0 = p.rot_dim + 16 * (unit - pair_units);  // first copied element
    // First elements of the unit's two runs of eight.
    const int r0 = !rotary ? d0 : kInterleaved ? 2 * j0 : j0;
    const int r1 = rotary && !kInterleaved ? half + j0 : r0 + 8;
    const int heads = p.q_heads + 2 * c.kv_heads, stride = slots * gridDim.y;
    auto source = [&](int h) {
        const bool is_q = h < p.q_heads, is_v = h >= p.q_heads + c.kv_heads;
        const int head = is_q ? h : h - p.q_heads - (is_v ? c.kv_heads : 0);
        return (is_q ? p.q + token * p.q_stride : (is_v ? p.v : p.k) + token * p.kv_stride) + static_cast<int64_t>(head) * c.head_dim;
    };
    // The first head's elements are asked for beside the position.
    uint4 ahead[2] = {};
    auto ask = [&](int h) {
        if constexpr (kVec) {
            const uint16_t *from = source(h);
            ahead[0] = *reinterpret_cast<const uint4 *>(from + r0);
            ahead[1] = *reinterpret_cast<const uint4 *>(from + r1);
        }
    };
    const int first = slot + blockIdx.y * slots;
    if (first >= heads) return;
    ask(first);

    if (pos < 0) return;
    int bad = 0;
    if (pos >= c.table_width * c.page_size || (p.rope && pos >= p.rope_positions)) bad |= kKvErrPosition;
    if (seq < 0 || seq >= p.sequences) bad |= kKvErrSequence;
    int64_t page = 0;
    if (!bad) {
        page = c.table[seq * c.table_width + pos / c.page_size];
        if (page < 0 || page >= c.num_pages) bad |= kKvErrPage;
    }
    float cos[8], sin[8];
    if (rotary && !bad) {
        const float *r = p.rope + pos * p.rot_dim;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            cos[i] = j0 + i < half ? r[j0 + i] : 1.f;
            sin[i] = j0 + i < half ? r[half + j0 + i] : 0.f;
        }
    }
    if (bad) {
        if (unit == 0 && slot == 0 && blockIdx.y == 0) atomicOr(p.status, bad);
        return;
    }
    const int64_t place = page * c.page_stride + (pos % c.page_size) * c.token_stride;
    for (int h = first; h < heads; h += stride) {
        if (h != first) ask(h);
        const bool is_q = h < p.q_heads, is_v = h >= p.q_heads + c.kv_heads;
        const int head = is_q ? h : h - p.q_heads - (is_v ? c.kv_heads : 0);
        void *to = is_q ? p.q_out : is_v ? p.v_cache : p.k_cache;
        const int64_t at = is_q ? token * p.q_out_stride + static_cast<int64_t>(head) * c.head_dim : place + head * c.head_stride;
        const float *scales = is_v ? p.v_scale : p.k_scale;
        const float scale = kE4m3 && !is_q && scales ? scales[head] : 1.f;
        if constexpr (kVec) {
            float a[8], b[8];
            unpack8(ahead[0], a);
            unpack8(ahead[1], b);
            if (rotary && !is_v) {
#pragma unroll
                for (int x = 0; x < 8; ++x) {
                    if constexpr (kInterleaved) {
                        float *y = x < 4 ? a + 2 * x : b + 2 * (x - 4);
                        rotate(y[0], y[1], cos[x], sin[x]);
                    } else {
                        rotate(a[x], b[x], cos[x], sin[x]);
                    }
                }
            }
            if (is_q) {
                store8<false>(to, at + r0, a, 1.f);
                store8<false>(to, at + r1, b, 1.f);
            } else {
                store8<kE4m3>(to, at + r0, a, scale);
                store8<kE4m3>(to, at + r1, b, scale);
            }
        } else {
            const uint16_t *from = source(h);
#pragma unroll
            for (int x = 0; x < 8; ++x) {
                const int e0 = !rotary ? d0 + 2 * x : kInterleaved ? 2 * (j0 + x) : j0 + x;
                const int e1 = rotary && !kInterleaved ? half + j0 + x : e0 + 1;
                if (rotary ? j0 + x >= half : e0 >= c.head_dim) break;
                float a = bf16_bits_to_float(from[e0]), b = bf16_bits_to_float(from[e1]);
                if (rotary && !is_v) rotate(a, b, cos[x], sin[x]);
                if (is_q) {
                    store1<false>(to, at + e0, a, 1.f);
                    store1<false>(to, at + e1, b, 1.f);
                } else {
                    store1<kE4m3>(to, at + e0, a, scale);
                    store1<kE4m3>(to, at + e1, b, scale);
                }
            }
        }
    }
}

// Append with the norm of each head of q and k before the rotation, and a rotary
// row of the token's own:
//   y = x · w / sqrt(Σ x² / head_dim + eps),  then rotated at rope[rope_rows[token]].
// The squares are summed in fp32 by the lanes that hold a head's units (a power of
// two of them, idle ones past the last unit), so a head is read once and meets in
// log2(lanes) shuffles, while its next head is on the way; bytes bound it as they
// bound the append alone.  8191 tokens of 96 heads: 80 us (75 % of the copy
// bandwidth) with six blocks an SM, 85 with five (over 8 bits, 256 tokens of 64 + 16
// heads: 6.9 and 6.3; 8191 of 96: 86 and 88.5), 92 without the next head, 114 with the weights held in
// registers, which leave room for fewer warps than reading them from the L1 cache.
// The norm of one head: Σ x² below 2^120, and above 2^-90 where eps is too small to
// hide what squares below 2^-126 lose, is taken as it is; else the head is scaled by
// a power of two of its largest element first, so that every bf16 head has its norm.
__device__ __forceinline__ float group_sum(float x, int lanes, uint32_t mask) {
    for (int o = lanes / 2; o > 0; o >>= 1) x += __shfl_xor_sync(mask, x, o);
    return x;
}
// 1 / sqrt(Σ x² / head_dim + eps) of elements a, b, which it scales where it has to.
__device__ __forceinline__ float head_norm(float *a, float *b, float of_dim, float eps, int lanes, uint32_t mask) {
    uint64_t squares = pair_of(0.f, 0.f);
#pragma unroll
    for (int i = 0; i < 8; i += 2) {
        const uint64_t x = pair_of(a[i], a[i + 1]), y = pair_of(b[i], b[i + 1]);
        squares = fma2(x, x, fma2(y, y, squares));
    }
    const float2 both = pair_to(squares);
    float sum = group_sum(both.x + both.y, lanes, mask);
    if (sum < 0x1p120f && (sum >= 0x1p-90f || eps >= 0x1p-60f)) return rsqrtf(__fmaf_rn(sum, of_dim, eps));
    float top = 0.f;
#pragma unroll
    for (int i = 0; i < 8; ++i) top = fmaxf(top, fmaxf(fabsf(a[i]), fabsf(b[i])));
    for (int o = lanes / 2; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(mask, top, o));
    // 2^-e, e the exponent of the largest element, within ±126 (zeros and subnormals: -126).
    const int e = min(126, max(-126, static_cast<int>(__float_as_uint(top) >> 23) - 127));
    const float down = __uint_as_float(static_cast<uint32_t>(127 - e) << 23);
    sum = 0.f;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        a[i] *= down, b[i] *= down;
        sum = __fmaf_rn(a[i], a[i], __fmaf_rn(b[i], b[i], sum));
    }
    sum = group_sum(sum, lanes, mask) * of_dim;
    // (Its square may be out of range, and then is all there is.  `top` does not know of a NaN; the sum does.)
    const float root = sqrtf(eps) * down;
    return 1.f / (root > 0x1p60f && sum == sum ? root : sqrtf(__fmaf_rn(root, root, sum)));
}

// Elements [at, at + 8) of a head in 8 bits, x / scale, by products with a number below and one above
// 1 / scale (within[0] and within[1]).  Rounding is monotonic: the quotient, rounded to fp32 and then to
// e4m3, is between the two products' e4m3 numbers, and where these are one it is that one.  Else, near the
// middle between two e4m3 numbers, the division (a few values in a million; more where scales have few
// bits, whose quotients come to the very middle).  8191 tokens of 96 heads: 88.5 us, 106 with divisions
// alone; 103 where every scale is 3.
__device__ __forceinline__ void store8_between(void *to, int64_t at, const float *x, float scale, const float (&within)[2]) {
    uint32_t w[2][2];  // [product][word]
#pragma unroll
    for (int y = 0; y < 2; ++y) {
        const uint64_t by = pair_of(within[y], within[y]);
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const uint32_t lo = __nv_cvt_float2_to_fp8x2(pair_to(mul2(pair_of(x[4 * i], x[4 * i + 1]), by)), __NV_SATFINITE, __NV_E4M3);
            const uint32_t hi = __nv_cvt_float2_to_fp8x2(pair_to(mul2(pair_of(x[4 * i + 2], x[4 * i + 3]), by)), __NV_SATFINITE, __NV_E4M3);
            w[y][i] = lo | hi << 16;
        }
    }
    if (w[0][0] != w[1][0] || w[0][1] != w[1][1])
        store8<true>(to, at, x, scale);
    else
        *reinterpret_cast<uint2 *>(static_cast<uint8_t *>(to) + at) = make_uint2(w[0][0], w[0][1]);
}

// Eight weights from `at` on (aligned to 16 bytes).
__device__ __forceinline__ void load_weights(const void *w, int32_t f32, int at, float *x) {
    if (f32) {
        const float4 *from = reinterpret_cast<const float4 *>(static_cast<const float *>(w) + at);
        const float4 lo = from[0], hi = from[1];
        x[0] = lo.x, x[1] = lo.y, x[2] = lo.z, x[3] = lo.w, x[4] = hi.x, x[5] = hi.y, x[6] = hi.z, x[7] = hi.w;
    } else {
        unpack8(*reinterpret_cast<const uint4 *>(static_cast<const uint16_t *>(w) + at), x);
    }
}
__device__ __forceinline__ float load_weight(const void *w, int32_t f32, int at) {
    return f32 ? static_cast<const float *>(w)[at] : bf16_bits_to_float(static_cast<const uint16_t *>(w)[at]);
}

// lanes: threads of a head, the power of two at or above its units (32 at most).
template <bool kE4m3, bool kInterleaved, bool kVec>
__global__ void __launch_bounds__(kAppendThreads, kE4m3 ? 5 : 6) kv_append_norm_kernel(const KvAppendParams p, const int lanes) {
    griddep_launch_dependents();
    griddep_wait();
    const KvCacheView &c = p.cache;
    const int64_t token = blockIdx.x;
    const int half = p.rot_dim / 2;
    const int pair_units = (half + 7) / 8, units = pair_units + (c.head_dim - p.rot_dim + 15) / 16;
    const int slots = kAppendThreads / lanes;
    const int unit = threadIdx.x & (lanes - 1), slot = threadIdx.x / lanes;
    // The lanes of this head: every branch around a shuffle is theirs together.
    const uint32_t mask = lanes == 32 ? 0xffffffffu : ((1u << lanes) - 1u) << (threadIdx.x & 31 & ~(lanes - 1));
    const int heads = p.q_heads + 2 * c.kv_heads, stride = slots * gridDim.y;
    const int first = slot + blockIdx.y * slots;
    if (first >= heads) return;

    const bool rotary = unit < pair_units;
    const int j0 = 8 * unit;                              // first rotary pair
    const int d0 = p.rot_dim + 16 * (unit - pair_units);  // first copied element
    const int r0 = !rotary ? d0 : kInterleaved ? 2 * j0 : j0;  // first elements of the unit's two runs of eight
    const int r1 = rotary && !kInterleaved ? half + j0 : r0 + 8;
    // Pairs of this unit, and the elements of pair x.
    const int pairs = unit >= units ? 0 : min(8, rotary ? half - j0 : (c.head_dim - d0) / 2);
    auto e0 = [&](int x) { return !rotary ? d0 + 2 * x : kInterleaved ? 2 * (j0 + x) : j0 + x; };
    auto e1 = [&](int x) { return rotary && !kInterleaved ? half + j0 + x : e0(x) + 1; };

    const uint16_t *q_row = p.q + token * p.q_stride, *k_row = p.k + token * p.kv_stride, *v_row = p.v + token * p.kv_stride;
    const int keys = p.q_heads, values = p.q_heads + c.kv_heads;  // the first head of either
    auto source = [&](int h) {
        return (h < keys ? q_row : h < values ? k_row : v_row) + (h < keys ? h : h < values ? h - keys : h - values) * c.head_dim;
    };
    // The first head's elements are asked for beside the position.
    uint4 ahead[2] = {};
    auto ask = [&](int h) {
        if constexpr (kVec)
            if (pairs > 0) {
                const uint16_t *from = source(h);
                ahead[0] = *reinterpret_cast<const uint4 *>(from + r0);
                ahead[1] = *reinterpret_cast<const uint4 *>(from + r1);
            }
    };
    ask(first);

    const int64_t pos = p.positions[token];
    if (pos < 0) return;
    const int64_t seq = p.seq_ids ? p.seq_ids[token] : token;
    const int64_t row = p.rope_rows ? p.rope_rows[token] : pos;
    int bad = 0;
    if (pos >= c.table_width * c.page_size) bad |= kKvErrPosition;
    if (p.rope && (row < 0 || row >= p.rope_positions)) bad |= kKvErrRopeRow;
    if (seq < 0 || seq >= p.sequences) bad |= kKvErrSequence;
    // The cosines are asked for beside the page.
    float cos[8], sin[8];
    if (rotary && !(bad & kKvErrRopeRow)) {
        const float *r = p.rope + row * p.rot_dim;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            cos[i] = j0 + i < half ? r[j0 + i] : 1.f;
            sin[i] = j0 + i < half ? r[half + j0 + i] : 0.f;
        }
    }
    int64_t page = 0;
    const uint32_t page_of = static_cast<uint32_t>(pos) / static_cast<uint32_t>(c.page_size);
    if (!(bad & (kKvErrPosition | kKvErrSequence))) {
        page = c.table[seq * c.table_width + page_of];
        if (page < 0 || page >= c.num_pages) bad |= kKvErrPage;
    }
    if (bad) {
        if (threadIdx.x == 0 && blockIdx.y == 0) atomicOr(p.status, bad);
        return;
    }
    const int64_t place = page * c.page_stride + (static_cast<uint32_t>(pos) - page_of * static_cast<uint32_t>(c.page_size)) * c.token_stride;
    const float of_dim = 1.f / static_cast<float>(c.head_dim);
    for (int h = first; h < heads; h += stride) {
        const bool is_q = h < keys, is_v = h >= values;
        const int head = is_q ? h : is_v ? h - values : h - keys;
        void *to = is_q ? p.q_out : is_v ? p.v_cache : p.k_cache;
        const int64_t at = is_q ? token * p.q_out_stride + head * c.head_dim : place + head * c.head_stride;
        const float *scales = is_v ? p.v_scale : p.k_scale;
        const float scale = kE4m3 && !is_q && scales ? scales[head] : 1.f;
        const void *weight = is_q ? p.q_weight : is_v ? nullptr : p.k_weight;
        float a[8], b[8], wa[8], wb[8];
        if constexpr (kVec) {
            if (weight && pairs > 0) {
                load_weights(weight, p.weight_f32, r0, wa);
                load_weights(weight, p.weight_f32, r1, wb);
            }
            unpack8(ahead[0], a);
            unpack8(ahead[1], b);
        } else {
            const uint16_t *from = source(h);
#pragma unroll
            for (int x = 0; x < 8; ++x) {
                const bool in = x < pairs;
                a[x] = in ? bf16_bits_to_float(from[e0(x)]) : 0.f;
                b[x] = in ? bf16_bits_to_float(from[e1(x)]) : 0.f;
                wa[x] = in && weight ? load_weight(weight, p.weight_f32, e0(x)) : 0.f;
                wb[x] = in && weight ? load_weight(weight, p.weight_f32, e1(x)) : 0.f;
            }
        }
        if (h + stride < heads) ask(h + stride);
        if (weight) {
            const float by = head_norm(a, b, of_dim, p.eps, lanes, mask);
#pragma unroll
            for (int x = 0; x < 8; x += 2) {
                const uint64_t scale2 = pair_of(by, by);
                const float2 u = pair_to(mul2(mul2(pair_of(a[x], a[x + 1]), scale2), pair_of(wa[x], wa[x + 1])));
                const float2 v = pair_to(mul2(mul2(pair_of(b[x], b[x + 1]), scale2), pair_of(wb[x], wb[x + 1])));
                a[x] = u.x, a[x + 1] = u.y, b[x] = v.x, b[x + 1] = v.y;
            }
        }
        if (pairs == 0) continue;
        if (rotary && !is_v) {
            // (rotate()'s separate operations: as packed products and sums the compiler fused them, and a call
            // without norms had other bits than the append.)
#pragma unroll
            for (int x = 0; x < 8; ++x) {
                if constexpr (kVec && kInterleaved) {
                    float *y = x < 4 ? a + 2 * x : b + 2 * (x - 4);
                    rotate(y[0], y[1], cos[x], sin[x]);
                } else {
                    rotate(a[x], b[x], cos[x], sin[x]);
                }
            }
        }
        if constexpr (kVec) {
            if (is_q) {
                store8<false>(to, at + r0, a, 1.f);
                store8<false>(to, at + r1, b, 1.f);
            } else if (kE4m3 && scale >= 0x1p-100f && scale <= 0x1p100f) {
                // (The quotient with 1 is off by 2^-24, and the products by as much: 2^-22 is more than both.
                // Of a power of two the product is the quotient.)
                const float by = 1.f / scale;
                const bool exact = (__float_as_uint(scale) & 0x7fffffu) == 0;
                const float within[2] = {exact ? by : by * 0x1.fffff8p-1f, exact ? by : by * 0x1.000004p+0f};
                store8_between(to, at + r0, a, scale, within);
                store8_between(to, at + r1, b, scale, within);
            } else {
                store8<kE4m3>(to, at + r0, a, scale);
                store8<kE4m3>(to, at + r1, b, scale);
            }
        } else {
#pragma unroll
            for (int x = 0; x < 8; ++x) {
                if (x >= pairs) break;
                if (is_q) {
                    store1<false>(to, at + e0(x), a[x], 1.f);
                    store1<false>(to, at + e1(x), b[x], 1.f);
                } else {
                    store1<kE4m3>(to, at + e0(x), a[x], scale);
                    store1<kE4m3>(to, at + e1(x), b[x], scale);
                }
            }
        }
    }
}

}  // namespace dev
}  // namespace projgb
