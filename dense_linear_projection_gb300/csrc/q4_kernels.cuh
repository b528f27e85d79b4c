// Device code of the 4-bit projection Y = X·(s·(q − z))ᵀ (+ bias).
#pragma once

#include "proj_kernel.cuh"
#include "q4_internal.h"

namespace projgb {
namespace dev {

// Weight packing (preparation).  One thread writes the 16 bytes that one lane
// of a warp takes of a block of 16 weight rows × 64 K (see q4_internal.h).
__global__ void q4_pack_codes_kernel(const uint8_t *codes, uint4 *P, int64_t N, int64_t K, int64_t k_blocks,
                                     int64_t items) {
    for (int64_t e = blockIdx.x * static_cast<int64_t>(blockDim.x) + threadIdx.x; e < items;
         e += static_cast<int64_t>(gridDim.x) * blockDim.x) {
        const int lane = static_cast<int>(e & 31);
        const int64_t blk = e >> 5;  // (row tile · k_blocks + k-block) · 4 + row block of the tile
        const int64_t tk = blk >> 2;
        const int64_t n0 = (tk / k_blocks) * kQ4TileRows + (blk & 3) * 16 + (lane >> 2);
        uint32_t w[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int64_t k0 = (tk % k_blocks) * 64 + q4_k_of(lane & 3, i);
            uint32_t raw = 0;
#pragma unroll
            for (int half = 0; half < 2; ++half) {  // rows n0, n0 + 8
                const int64_t n = n0 + 8 * half;
                uint32_t four = 0x8888u;
                if (n < N && k0 < K)  // K is a multiple of 32: the four codes are all in range
                    four = codes[n * (K / 2) + k0 / 2] | (static_cast<uint32_t>(codes[n * (K / 2) + k0 / 2 + 1]) << 8);
                // Nibbles t and t + 4 become the low and high halves of operand register t.
                raw |= (four & 15u) << (4 * half);
                raw |= ((four >> 4) & 15u) << (4 * half + 16);
                raw |= ((four >> 8) & 15u) << (4 * half + 8);
                raw |= ((four >> 12) & 15u) << (4 * half + 24);
            }
            w[i] = __funnelshift_l(raw, raw, 3);
        }
        P[e] = make_uint4(w[0], w[1], w[2], w[3]);
    }
}

// Scales (pairs of rows r and r + 8 of a row block) and zero points (the same
// pairs, four bits each); zero scales past N and K.
__global__ void q4_pack_scales_kernel(const uint16_t *scales, const uint8_t *zeros, uint32_t *S, uint8_t *Z, int64_t N,
                                      int64_t groups, int64_t groups_padded, int64_t items) {
    for (int64_t e = blockIdx.x * static_cast<int64_t>(blockDim.x) + threadIdx.x; e < items;
         e += static_cast<int64_t>(gridDim.x) * blockDim.x) {
        const int64_t tg = e >> 5;
        const int64_t n = (tg / groups_padded) * kQ4TileRows + ((e >> 3) & 3) * 16 + (e & 7);
        const int64_t g = tg % groups_padded;
        uint32_t s = 0, z = 0x88u;
        if (g < groups) {
            if (n < N) s = scales[n * groups + g];
            if (n + 8 < N) s |= static_cast<uint32_t>(scales[(n + 8) * groups + g]) << 16;
            if (zeros) z = (n < N ? zeros[n * groups + g] & 15u : 8u) | ((n + 8 < N ? zeros[(n + 8) * groups + g] & 15u : 8u) << 4);
        }
        S[e] = s;
        if (Z) Z[e] = static_cast<uint8_t>(z);
    }
}

// One warp per weight row and token.
__global__ void q4_kernel(Q4Params p) {
    griddep_launch_dependents();
    griddep_wait();
    const int lane = threadIdx.x & 31;
    const int64_t n = blockIdx.x * static_cast<int64_t>(blockDim.x / 32) + threadIdx.x / 32;
    if (n >= p.N) return;
    const int64_t tile = n / kQ4TileRows;
    const int rb = static_cast<int>(n % kQ4TileRows) / 16, half = static_cast<int>(n % 16) / 8, r = static_cast<int>(n % 8);
    for (int64_t m = blockIdx.y; m < p.M; m += gridDim.y) {
        float acc = 0.f;
        for (int64_t kb = lane; kb < p.k_blocks; kb += 32) {
            for (int j = 0; j < 4; ++j) {
                const uint4 v = p.codes[((tile * p.k_blocks + kb) * 4 + rb) * 32 + r * 4 + j];
                const uint32_t w[4] = {v.x, v.y, v.z, v.w};
                for (int i = 0; i < 4; ++i) {
                    const int64_t k0 = kb * 64 + q4_k_of(j, i);
                    if (k0 >= p.K) continue;
                    const int64_t at = ((tile * p.groups_padded + k0 / p.group) * 4 + rb) * 8 + r;
                    const float s = bf16_bits_to_float(static_cast<uint16_t>(p.scales[at] >> (16 * half)));
                    const float z = p.zeros ? static_cast<float>((p.zeros[at] >> (4 * half)) & 15) : 8.f;
                    const uint32_t raw = __funnelshift_r(w[i], w[i], 3) >> (4 * half);
                    const uint16_t *x = p.X + m * p.K + k0;
                    acc += s * (bf16_bits_to_float(x[0]) * (static_cast<float>(raw & 15) - z) +
                                bf16_bits_to_float(x[1]) * (static_cast<float>((raw >> 16) & 15) - z) +
                                bf16_bits_to_float(x[2]) * (static_cast<float>((raw >> 8) & 15) - z) +
                                bf16_bits_to_float(x[3]) * (static_cast<float>((raw >> 24) & 15) - z));
                }
            }
        }
        for (int o = 16; o > 0; o >>= 1) acc += __shfl_xor_sync(0xffffffffu, acc, o);
        if (lane == 0) {
            if (p.bias) acc += bf16_bits_to_float(p.bias[n]);
            if (p.y_f32)
                static_cast<float *>(p.Y)[m * p.N + n] = acc;
            else
                static_cast<__nv_bfloat16 *>(p.Y)[m * p.N + n] = __float2bfloat16_rn(acc);
        }
    }
}

}  // namespace dev
}  // namespace projgb
