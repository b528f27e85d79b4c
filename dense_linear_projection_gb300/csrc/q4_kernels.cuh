// Device code of the 4-bit projection Y = X·(s·(q − z))ᵀ (+ bias).
#pragma once

#include "proj_kernel.cuh"
#include "proj_warp.cuh"
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
                raw |= (four & 15u) << (8 * half);
                raw |= ((four >> 4) & 15u) << (8 * half + 16);
                raw |= ((four >> 8) & 15u) << (8 * half + 4);
                raw |= ((four >> 12) & 15u) << (8 * half + 20);
            }
            w[i] = raw;
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

// ---- the projection
//
// Mathematics: Y[m,n] = Σ_g s[n,g]·(Σ_{k in g} q[n,k]·x[m,k] − z[n,g]·Σ_{k in g} x[m,k]).
//
// Codes as operands.  A bf16 number with exponent field 0 and mantissa q is
// q·2^-133 (a subnormal), and the scale goes on evenly into exponent field 1:
// the 16 bits 0000'0000'qqqq'0000 are q·2^-129 for every q of four bits.  So one
// AND makes a pair of codes a pair of exact bf16 numbers, in either of two
// nibbles of each half word, and one fused multiply-add makes it
// (q − z)·2^-7, exact: nine instructions for eight codes.  The tensor core
// multiplies X as it is by these; a group's fp32 sum is scaled into the row's
// fp32 sum, and the 2^7 is taken back when the row is written.
//
// The product is swapped (weight rows are the 16-row operand of the warp-level
// step, up to 8·kNT tokens its columns).  What bounds it: at up to 8 tokens, where
// the row count fills the SMs, the stream of codes, with 60 % of the issue slots
// spent on 500 instructions a warp for 4 KiB of them (one token, 28672 × 8192:
// 20.7 us, 87 % of the copy bandwidth); above that waits.  At 16 and 31 tokens 39
// and 41 % of the issue slots and 20 and 27 % of the tensor pipe are in use: two to
// four warps a scheduler wait for results, the math pipe, memory and one another
// (16 tokens, 8192 × 8192: 14.2 us, of 5.4 for the bytes; 31 tokens, 12300 × 4128 in
// groups of 32: 16.5, of 4.4), and whole tiles a CTA leave SMs idle between the row
// counts that fill them (one token, 20480 rows take as long as 28672).
// A warp owns 64 or 32 rows × 128 K at a time, in a ring of shared-memory stages
// filled by 16-byte asynchronous copies.  A CTA covers one row tile × kKW K steps;
// the CTAs of a cluster share the K range of the same rows.  Sums join in a fixed order: the
// kKW warps in shared memory, then the cluster's CTAs through distributed shared
// memory.
//
// The tcgen05 tensor core is not faster here: with the operands stored to tensor
// memory by the warps and the sums read back for each group, the same cases took
// 50, 17.5 and 20.6 us.  The warps' own work stays, and hand-overs come to it.
constexpr uint32_t kQ4Unit = 0x7E807E80u;      // 2^126, twice: codes that stand for q·2^-133
constexpr uint32_t kQ4UnitHigh = 0x7C807C80u;  // 2^122: for q·2^-129
constexpr uint32_t kQ4UnitMinus = 0xFE80FE80u;
constexpr float kQ4Restore = 128.f;

// How a CTA is cut: four warps, so that CTAs of even size spread evenly over the
// SMs at most row counts.  Measured at K = 8192 against CTAs of eight warps (two an
// SM up to 8 tokens, one at 16): 1 token, 10240 rows 12.2 us against 14.9, 28672
// rows 21.8 against 23.0, 2048 rows 4.8 against 4.7; 16 tokens, 12288 rows 17.1
// against 23.6, 28672 rows 28.6 against 36.0, 8192 rows 13.4 against 12.8.  With 32
// tokens two warps share the copies of X and have two row blocks each, as registers
// allow; two row tiles a CTA copy X half as often, yet take 17.8 us against 12.9 at
// 4096 rows, and 26.0 against 26.4 at 12288.
template <int kNT>
struct Q4Tile {
    static constexpr int kWarps = 4, kThreads = 32 * kWarps;
    static constexpr int kR = kNT == 4 ? 2 : 4;        // row blocks of a warp
    static constexpr int kPerSm = kNT == 2 ? 3 : 4;    // CTAs an SM, by their registers
    static constexpr int kShare = 4 / kR;            // warps that share a K step
    static constexpr int kKW = kWarps / kShare;      // K steps at a time
    static constexpr int kPitch = 64 + 4;            // floats of a token's rows while joining: conflict-free
    static constexpr int kRed = kKW * 8 * kNT * kPitch * 4;
    static_assert(kKW * kShare == kWarps, "whole K steps");
};

__device__ __forceinline__ uint32_t bf16x2_fma(uint32_t a, uint32_t b, uint32_t c) {
    uint32_t d;
    asm("fma.rn.bf16x2 %0, %1, %2, %3;" : "=r"(d) : "r"(a), "r"(b), "r"(c));
    return d;
}
// a0 += s·b0, a1 += s·b1 in one instruction.
__device__ __forceinline__ void fma_pair(float &a0, float &a1, float s, float b0, float b1) {
    asm("{\n\t.reg .b64 a, b, c;\n\t"
        "mov.b64 a, {%0, %1};\n\tmov.b64 b, {%3, %4};\n\tmov.b64 c, {%2, %2};\n\t"
        "fma.rn.f32x2 a, b, c, a;\n\tmov.b64 {%0, %1}, a;\n\t}"
        : "+f"(a0), "+f"(a1)
        : "f"(s), "f"(b0), "f"(b1));
}
__device__ __forceinline__ uint32_t bf16x2_mul(uint32_t a, uint32_t b) {
    uint32_t d;
    asm("mul.rn.bf16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
    return d;
}

__device__ __forceinline__ uint4 lds128(uint32_t at) {
    uint4 v;
    asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(at) : "memory");
    return v;
}
__device__ __forceinline__ uint2 lds64(uint32_t at) {
    uint2 v;
    asm volatile("ld.shared.v2.b32 {%0, %1}, [%2];" : "=r"(v.x), "=r"(v.y) : "r"(at) : "memory");
    return v;
}
__device__ __forceinline__ uint32_t lds32(uint32_t at) {
    uint32_t v;
    asm volatile("ld.shared.b32 %0, [%1];" : "=r"(v) : "r"(at) : "memory");
    return v;
}
__device__ __forceinline__ uint32_t lds8(uint32_t at) {
    uint32_t v;
    asm volatile("{\n\t.reg .u8 b;\n\tld.shared.u8 b, [%1];\n\tcvt.u32.u8 %0, b;\n\t}" : "=r"(v) : "r"(at) : "memory");
    return v;
}
__device__ __forceinline__ float4 ld_cluster_f4(uint32_t cluster_addr) {
    float4 v;
    asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];"
                 : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w)
                 : "r"(cluster_addr)
                 : "memory");
    return v;
}

// kGroups: groups of a 128-wide K step (1, 2 or 4).
template <int kNT, int kGroups, bool kZeros>
__global__ void __launch_bounds__(Q4Tile<kNT>::kThreads, Q4Tile<kNT>::kPerSm) q4_kernel(const Q4Params p) {
    using Tile = Q4Tile<kNT>;
    constexpr int kKW = Tile::kKW, kR = Tile::kR, kShare = Tile::kShare;
    extern __shared__ __align__(256) uint8_t smem[];
    griddep_launch_dependents();
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int part_of = warp % kShare, kw = warp / kShare;  // which of the CTA's rows, which K steps
    const int g = lane >> 2, j = lane & 3;
    const uint32_t rank = blockIdx.x % p.splits;
    const int64_t tile = blockIdx.x / p.splits;
    const int block0 = part_of * kR;  // the warp's first row block of the tile
    const int64_t m0 = blockIdx.y * int64_t(kQ4MaxTokens);
    const int M = static_cast<int>(p.M - m0 < kQ4MaxTokens ? p.M - m0 : kQ4MaxTokens);

    // A stage: each warp's codes, scales and zero points, then X for each K step.
    constexpr int kCodeBytes = kR * 1024, kScaleBytes = kGroups * kR * 32, kZeroBytes = kZeros ? kGroups * kR * 8 : 0;
    constexpr int kWarpBytes = kCodeBytes + kScaleBytes + kZeroBytes;
    constexpr int kWeights = (Tile::kWarps * kWarpBytes + 255) / 256 * 256;  // X begins on a 256-byte boundary
    const int x_bytes = M * kQ4XPitch;
    const int stage_bytes = kWeights + kKW * x_bytes;
    const uint32_t base = smem_u32(smem);
    const uint32_t my_w = base + warp * kWarpBytes, my_x = base + kWeights + kw * x_bytes;

    const uint32_t steps = static_cast<uint32_t>((p.k_blocks + 1) / 2);  // at most 2^24: 32-bit divisions
    const int step0 = static_cast<int>(steps * rank / p.splits) + kw, step1 = static_cast<int>(steps * (rank + 1) / p.splits);

    uint32_t x_row[kNT];  // this lane's place in a step's X
#pragma unroll
    for (int t = 0; t < kNT; ++t) {
        const int m = min(8 * t + g, M - 1);
        x_row[t] = m * kQ4XPitch + j * 16 + (m & 1) * 64;
    }

    float acc[kR][kNT][4];
#pragma unroll
    for (int r = 0; r < kR; ++r)
#pragma unroll
        for (int t = 0; t < kNT; ++t) acc[r][t][0] = acc[r][t][1] = acc[r][t][2] = acc[r][t][3] = 0.f;

    // Loading: pointers to this lane's next step.  A group's scales are 2·kR
    // copies of 16 bytes, its zero points kR / 2.
    const uint8_t *codes = reinterpret_cast<const uint8_t *>(p.codes) + (tile * p.k_blocks + step0 * 2) * 2048 + block0 * 512 + lane * 16;
    const int scale_group = lane / (2 * kR), zero_group = lane / (kR / 2);
    const uint8_t *scales = reinterpret_cast<const uint8_t *>(p.scales) +
                            (tile * p.groups_padded + step0 * kGroups + scale_group) * 128 + block0 * 32 + lane % (2 * kR) * 16;
    const uint8_t *zeros = kZeros ? p.zeros + (tile * p.groups_padded + step0 * kGroups + zero_group) * 32 + block0 * 8 +
                                        lane % (kR / 2) * 16
                                  : nullptr;
    const int x_first = (part_of * 32 + lane) / 16, x_chunk = lane % 16;  // first of the tokens this lane copies; its 8 K of the step
    const uint8_t *x = reinterpret_cast<const uint8_t *>(p.X + (m0 + x_first) * p.K + step0 * 128 + x_chunk * 8);
    const int x_to = (x_chunk * 16) ^ ((x_first & 1) * 64);  // all of a lane's tokens are odd, or even
    const int64_t x_next = 2 * kShare * p.K * 2;  // bytes to the lane's next token
    const int whole = static_cast<int>((p.K / 128 < step1 ? p.K / 128 : step1));  // steps below it lie inside K
    auto load = [&](int step, int slot) {
        if (step < step1) {
            const uint32_t w = my_w + slot * stage_bytes + lane * 16;
            uint32_t to = my_x + slot * stage_bytes + x_first * kQ4XPitch + x_to;
            const uint8_t *from = x;
            if (step < whole) {
#pragma unroll
                for (int i = 0; i < 2 * kR; ++i) cp_async16(w + i * 512, codes + i / kR * 2048 + i % kR * 512);
                if (scale_group < kGroups) cp_async16(w + kCodeBytes, scales);
                if (kZeros && zero_group < kGroups) cp_async16(w + kCodeBytes + kScaleBytes, zeros);
                for (int m = x_first; m < M; m += 2 * kShare, to += 2 * kShare * kQ4XPitch, from += x_next) cp_async16(to, from);
            } else {
                // K ends inside the step: the blocks of codes and the groups
                // that exist, and zeros for the rest.
                const int blocks = step * 2 + 1 < p.k_blocks ? 2 : 1;
#pragma unroll
                for (int i = 0; i < 2 * kR; ++i)
                    cp_async16(w + i * 512, i / kR < blocks ? codes + i / kR * 2048 + i % kR * 512 : codes, i / kR < blocks);
                if (scale_group < kGroups) {
                    const bool in = step * kGroups + scale_group < p.groups_padded;
                    cp_async16(w + kCodeBytes, in ? scales : codes, in);
                }
                if (kZeros && zero_group < kGroups) {
                    const bool in = step * kGroups + zero_group < p.groups_padded;
                    cp_async16(w + kCodeBytes + kScaleBytes, in ? zeros : codes, in);
                }
                const bool in = step * 128 + x_chunk * 8 < p.K;
                for (int m = x_first; m < M; m += 2 * kShare, to += 2 * kShare * kQ4XPitch, from += x_next)
                    cp_async16(to, in ? from : codes, in);
            }
            codes += kKW * 4096;
            scales += kKW * kGroups * 128;
            if (kZeros) zeros += kKW * kGroups * 32;
            x += kKW * 256;
        }
        cp_async_commit();
    };
    // The warps that share a step's X.
    auto meet = [&]() {
        if constexpr (kShare == 1)
            __syncwarp();
        else
            asm volatile("bar.sync %0, %1;" ::"r"(1 + kw), "n"(32 * kShare) : "memory");
    };

    // The first step's codes move to L2 while the kernel before this one ends (a
    // prefetch returns nothing, so it may come before the wait): 20.7 us against
    // 21.2 for one token, 28672 × 8192.  More steps, or 32 tokens, gain nothing.
    if constexpr (kNT < 4) {
        if (step0 < whole)
            asm volatile("prefetch.global.L2 [%0];" ::"l"(reinterpret_cast<const uint8_t *>(p.codes) +
                                                          (tile * p.k_blocks + step0 * 2) * 2048 + lane * 128));
    }
    griddep_wait();
    const int stages = p.stages;
    for (int s = 0; s < stages - 1; ++s) load(step0 + s * kKW, s);
    int slot = 0, slot_in = stages - 1;
    for (int step = step0; step < step1; step += kKW) {
        if (stages == 2)
            cp_async_wait<0>();
        else
            cp_async_wait<1>();
        meet();
        load(step + (stages - 1) * kKW, slot_in);
        if (++slot_in == stages) slot_in = 0;
        const uint32_t w = my_w + slot * stage_bytes, xs = my_x + slot * stage_bytes;
        if (++slot == stages) slot = 0;

        // A warp's row blocks go together: independent chains of tensor-core
        // steps that cover their latency.
        constexpr int kWords = 8 / kGroups;         // tensor-core steps of a group
        constexpr int kPiece = kWords < 4 ? 2 : 4;  // steps whose operands are loaded at once
#pragma unroll
        for (int group = 0; group < kGroups; ++group) {
            float part[kR][kNT][4];
            uint32_t z[kR][2];
#pragma unroll
            for (int r = 0; r < kR; ++r) {
                if constexpr (kZeros) {
                    const uint32_t both = lds8(w + kCodeBytes + kScaleBytes + group * kR * 8 + r * 8 + g);
                    z[r][0] = bf16x2_mul((both & 15u) * 0x00010001u, kQ4UnitMinus);
                    z[r][1] = bf16x2_mul((both >> 4) * 0x00010001u, kQ4UnitMinus);
                } else {
                    z[r][0] = z[r][1] = 0xBD80BD80u;  // −8·2^-7
                }
            }
#pragma unroll
            for (int i0 = 0; i0 < kWords; i0 += kPiece) {
                const int at = group * kWords + i0;  // of the eight steps
                // X as the second operand: column (token) g; columns past M
                // repeat the last token and are dropped.
                uint32_t b[kNT][2 * kPiece], word[kR][kPiece];
#pragma unroll
                for (int t = 0; t < kNT; ++t)
#pragma unroll
                    for (int h = 0; h < kPiece / 2; ++h) {
                        const uint4 v = lds128((xs + x_row[t]) ^ ((at / 2 + h) * 64));
                        b[t][4 * h] = v.x, b[t][4 * h + 1] = v.y, b[t][4 * h + 2] = v.z, b[t][4 * h + 3] = v.w;
                    }
#pragma unroll
                for (int r = 0; r < kR; ++r) {
                    const uint32_t from = w + (at / 4) * kR * 512 + r * 512 + lane * 16 + (at % 4) * 4;  // four steps: 16 bytes
                    if constexpr (kPiece == 4) {
                        const uint4 v = lds128(from);
                        word[r][0] = v.x, word[r][1] = v.y, word[r][2] = v.z, word[r][3] = v.w;
                    } else {
                        const uint2 v = lds64(from);
                        word[r][0] = v.x, word[r][1] = v.y;
                    }
                }
#pragma unroll
                for (int i = 0; i < kPiece; ++i)
#pragma unroll
                    for (int r = 0; r < kR; ++r) {
                        const uint32_t now = word[r][i], next = now >> 8;
                        const uint32_t a0 = bf16x2_fma(now & 0x000f000fu, kQ4Unit, z[r][0]);
                        const uint32_t a1 = bf16x2_fma(next & 0x000f000fu, kQ4Unit, z[r][1]);
                        const uint32_t a2 = bf16x2_fma(now & 0x00f000f0u, kQ4UnitHigh, z[r][0]);
                        const uint32_t a3 = bf16x2_fma(next & 0x00f000f0u, kQ4UnitHigh, z[r][1]);
#pragma unroll
                        for (int t = 0; t < kNT; ++t) {
                            if (i0 + i == 0)
                                mma16816_first<false>(part[r][t], a0, a1, a2, a3, b[t][2 * i], b[t][2 * i + 1]);
                            else
                                mma16816<false>(part[r][t], a0, a1, a2, a3, b[t][2 * i], b[t][2 * i + 1]);
                        }
                    }
            }
#pragma unroll
            for (int r = 0; r < kR; ++r) {
                const uint32_t two = lds32(w + kCodeBytes + group * kR * 32 + r * 32 + g * 4);
                const float s0 = __uint_as_float(two << 16), s1 = __uint_as_float(two & 0xffff0000u);
#pragma unroll
                for (int t = 0; t < kNT; ++t) {
                    fma_pair(acc[r][t][0], acc[r][t][1], s0, part[r][t][0], part[r][t][1]);
                    fma_pair(acc[r][t][2], acc[r][t][3], s1, part[r][t][2], part[r][t][3]);
                }
            }
        }
    }

    // Join: [K step][token][row] in shared memory (the stages are done with).
    cp_async_wait<0>();
    __syncthreads();
    float *red = reinterpret_cast<float *>(smem);
    constexpr int kPitch = Tile::kPitch, kPlane = 8 * kNT * kPitch;
#pragma unroll
    for (int r = 0; r < kR; ++r)
#pragma unroll
        for (int t = 0; t < kNT; ++t) {
            float *to = red + kw * kPlane + (8 * t + 2 * j) * kPitch + (part_of * kR + r) * 16 + g;
            to[0] = acc[r][t][0];
            to[kPitch] = acc[r][t][1];
            to[8] = acc[r][t][2];
            to[kPitch + 8] = acc[r][t][3];
        }
    __syncthreads();
    // Four rows at a time.
    constexpr uint32_t kQuads = 16;
    const uint32_t quads = M * kQuads;
    const int64_t n0 = tile * 64;
    auto store = [&](uint32_t e, float4 v) {
        const int64_t n = n0 + (e % kQuads) * 4, at = (m0 + e / kQuads) * p.N + n;
        float y[4] = {v.x * kQ4Restore, v.y * kQ4Restore, v.z * kQ4Restore, v.w * kQ4Restore};
        if (p.bias) {
#pragma unroll
            for (int i = 0; i < 4; ++i)
                if (n + i < p.N) y[i] += bf16_bits_to_float(p.bias[n + i]);
        }
        if (p.y_vec && n < p.N) {  // N is a multiple of 4
            if (p.y_f32)
                *reinterpret_cast<float4 *>(static_cast<float *>(p.Y) + at) = make_float4(y[0], y[1], y[2], y[3]);
            else
                *reinterpret_cast<uint2 *>(static_cast<uint16_t *>(p.Y) + at) =
                    make_uint2(bf16_pair(y[0], y[1]), bf16_pair(y[2], y[3]));
        } else {
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                if (n + i >= p.N) break;
                if (p.y_f32)
                    static_cast<float *>(p.Y)[at + i] = y[i];
                else
                    static_cast<__nv_bfloat16 *>(p.Y)[at + i] = __float2bfloat16_rn(y[i]);
            }
        }
    };
    if (kKW > 1 || p.splits == 1) {
        for (uint32_t e = tid; e < quads; e += Tile::kThreads) {
            float4 *at = reinterpret_cast<float4 *>(red + (e / kQuads) * kPitch + (e % kQuads) * 4);
            float4 y = *at;
#pragma unroll
            for (int k = 1; k < kKW; ++k) {
                const float4 o = at[k * kPlane / 4];
                y.x += o.x, y.y += o.y, y.z += o.z, y.w += o.w;
            }
            if (p.splits == 1)
                store(e, y);
            else
                *at = y;
        }
    }
    if (p.splits > 1) {
        cluster_arrive();
        cluster_wait();
        // Each CTA finishes a share of the elements, adding the ranks in order.
        const uint32_t e1 = quads * (rank + 1) / p.splits;
        for (uint32_t e = quads * rank / p.splits + tid; e < e1; e += Tile::kThreads) {
            if (n0 + (e % kQuads) * 4 >= p.N) continue;  // what is read is stored
            const uint32_t at = base + ((e / kQuads) * kPitch + (e % kQuads) * 4) * 4;
            float4 part[kQ4MaxSplits];
#pragma unroll
            for (int s = 0; s < kQ4MaxSplits; ++s)
                if (s < p.splits) part[s] = ld_cluster_f4(map_to_rank(at, s));
            float4 y = part[0];
#pragma unroll
            for (int s = 1; s < kQ4MaxSplits; ++s)
                if (s < p.splits) y.x += part[s].x, y.y += part[s].y, y.z += part[s].z, y.w += part[s].w;
            store(e, y);
        }
        // No CTA leaves while another reads its sums: the arrival releases, so the
        // reads come before it.  (It waits for the stores too, 0.2 us.  With all reads
        // first and the stores after the arrival, 2048 rows take 4.15 us instead of
        // 4.24, but 31 tokens in groups of 32 take 20.0 instead of 16.5.)
        cluster_arrive();
        cluster_wait();
    }
}

}  // namespace dev
}  // namespace projgb
