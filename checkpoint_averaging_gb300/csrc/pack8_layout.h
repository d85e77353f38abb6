// pack8_layout.h -- the bytes of the 8-bit form (cam_pack8) as the kernels read them.
#pragma once

#include <cstdint>

#include "cam_internal.h"

namespace cam {

constexpr int kP8Block = 128;  // columns that share a scale

// Bytes between rows of q: rows of whole 16-byte pieces, as the tensor maps need.
inline int64_t p8_ld(int64_t cols) { return (cols + 15) / 16 * 16; }

// Bytes of q, to a multiple of 512.
inline int64_t p8_q_bytes(int64_t rows, int64_t cols) {
    return (rows * p8_ld(cols) + 511) / 512 * 512;
}

inline int64_t p8_bytes(int64_t rows, int64_t cols) {
    if (rows == 0 || cols == 0) return 0;
    return p8_q_bytes(rows, cols) + 512 * ((rows + 127) / 128) * ((cols + kP8Block - 1) / kP8Block);
}

inline int p8_check(const char* fn, int64_t rows, int64_t cols) {
    if (rows < 0 || rows > (int64_t(1) << 31))
        return record_error(CAM_E_ARG, "%s: rows out of range", fn);
    if (cols < 0 || cols > CAM_PACK4_MAX_COLS)
        return record_error(CAM_E_ARG, "%s: cols out of range", fn);
    return CAM_OK;
}

// Queues the packing of a matrix on `s` (pack8.cu). Errors: CAM_E_CUDA.
int p8_pack(const char* fn, int64_t rows, int64_t cols, const void* w, int64_t stride,
            cam_dtype dtype, void* packed, cudaStream_t s);

}  // namespace cam
