// pack4_layout.h -- the 4-bit form of a matrix (include/cam.h), shared by the
// calls that write, read and multiply by it.
//
// The form is laid out for the product's tensor-core step (gemv4.cu). A tile
// is 16 rows x 128 columns in one contiguous record, so a warp streams whole
// records. In mma.m16n8k16 a lane l supplies rows l / 4 and l / 4 + 8 of the
// weights and any four columns per row that the other operand's lane agrees
// on; the 16 bytes of lane l in half h are its 32 weights of row
// 8 h + l / 4: word i belongs to columns 32 i .. 32 i + 31, so that a step of
// 32 columns never mixes two groups' scales. In a word, nibbles p and p + 4
// hold neighbouring columns: (word >> 4 p) & 0x000F000F is one register of
// the operand but for the conversion of its two halves.
#pragma once

#include <cstdint>

#include "cam_internal.h"

namespace cam {

constexpr int kP4Rows = 16;
constexpr int kP4Cols = 128;
constexpr int kP4Quants = kP4Rows * kP4Cols / 2;  // bytes of q in a tile

__host__ __device__ constexpr int p4_tile_bytes(int group) {
    return kP4Quants + kP4Rows * (kP4Cols / group) * 2;
}

// Byte of the tile's q that holds the word of (row, 8-column run w = 0..15).
__host__ __device__ constexpr int p4_word(int row, int w) {
    return (row >> 3) * 512 + ((row & 7) * 4 + (w & 3)) * 16 + (w >> 2) * 4;
}

// Index of the scale of (row, group j) among the tile's scales.
__host__ __device__ constexpr int p4_scale(int row, int j, int per_tile) {
    return (2 * (row & 7) + (row >> 3)) * per_tile + j;
}

// Checks of the arguments that the calls share; CAM_OK or a recorded error.
inline int p4_check(const char* fn, int64_t rows, int64_t cols, int32_t group) {
    if (rows < 0 || rows > (int64_t(1) << 40))
        return record_error(CAM_E_ARG, "%s: rows out of range", fn);
    if (cols < 0 || cols > CAM_PACK4_MAX_COLS)
        return record_error(CAM_E_ARG, "%s: cols out of range", fn);
    if (group != 32 && group != 64 && group != 128)
        return record_error(CAM_E_ARG, "%s: group must be 32, 64 or 128", fn);
    return CAM_OK;
}

// Bytes of the 4-bit form.
inline int64_t p4_bytes(int64_t rows, int64_t cols, int32_t group) {
    return ((rows + kP4Rows - 1) / kP4Rows) * ((cols + kP4Cols - 1) / kP4Cols) *
           p4_tile_bytes(group);
}

}  // namespace cam
