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

}  // namespace dev
}  // namespace projgb
