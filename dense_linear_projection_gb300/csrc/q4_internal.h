// Packed 4-bit weights: layout shared by the packing kernel, the projection
// kernel and the host.
//
// Weight rows are cut into tiles of 64 (four row blocks of 16) and K into
// blocks of 64.  One (row block, k-block) is 512 bytes: lane l of a warp takes
// 16 bytes, the A operands of four tensor-core steps (16 rows × 16 K each) in
// the lane's own register layout.  With r = l / 4 and j = l % 4, step i covers
// rows r and r + 8 and the four K positions q4_k_of(j, i) .. + 3.  (Which K
// positions share a step is free, as X is read by the same rule; this one gives
// a lane 16 contiguous bytes of X for two steps, and keeps a step within a
// group of 32.)  A step's word holds, in each half (even K low, odd K high):
// nibble 0 row r, K + 0/1; nibble 1 row r, K + 2/3; nibbles 2 and 3 the same of
// row r + 8.
//
//   codes   [row tile][k-block][row block 0..3][lane] 16 bytes
//   scales  [row tile][group][row block][r = 0..7] bf16 of rows r, r + 8
//   zeros   [row tile][group][row block][r] four bits of rows r, r + 8
//
// Rows past N and K past its end have code 8 and scale 0.
#pragma once

#include <stddef.h>
#include <stdint.h>

#include <cuda_runtime.h>

#include "proj_internal.h"

namespace projgb {

constexpr int kQ4TileRows = 64;
constexpr int kQ4MaxTokens = 32;  // tokens of one pass over the weights
constexpr int kQ4MaxSplits = 8;   // CTAs of a cluster that share a K range (the portable cluster size)
// Bytes between tokens of X in a stage: 128 K.  Odd tokens have the 64-byte
// halves of each 128 bytes swapped: two tokens' chunks lie on different banks.
constexpr int kQ4XPitch = 256;

PROJ_HD int q4_k_of(int j, int i) { return (i >> 1) * 32 + j * 8 + (i & 1) * 4; }

struct Q4Shape {
    int64_t row_tiles, k_blocks, groups, groups_padded;
    int64_t codes_bytes, scales_bytes, zeros_bytes;
};

inline Q4Shape q4_shape(int64_t N, int64_t K, int64_t group, bool has_zeros) {
    Q4Shape s;
    s.row_tiles = (N + kQ4TileRows - 1) / kQ4TileRows;
    s.k_blocks = (K + 63) / 64;
    s.groups = K / group;
    s.groups_padded = group <= 64 ? s.k_blocks * (64 / group) : s.groups;  // 128: K is whole groups
    s.codes_bytes = s.row_tiles * s.k_blocks * 2048;
    s.scales_bytes = s.row_tiles * s.groups_padded * 128;
    s.zeros_bytes = has_zeros ? s.row_tiles * s.groups_padded * 32 : 0;
    return s;
}

struct Q4Params {
    int64_t M, N, K, row_tiles, k_blocks, groups_padded;
    int32_t y_f32;
    int32_t y_vec;   // Y's rows start on four-element boundaries: four at a time
    uint32_t splits;  // CTAs of a cluster
    int32_t stages;  // of the ring: 2 or 3
    const uint16_t *X;
    const uint4 *codes;
    const uint32_t *scales;
    const uint8_t *zeros;  // nullptr: 8
    const uint16_t *bias;
    void *Y;
};

}  // namespace projgb
