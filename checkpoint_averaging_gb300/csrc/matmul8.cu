// matmul8.cu -- products of many rows with a matrix in the 8-bit form (cam_matmul8): the
// rows are brought into the same form (pack8.cu), then one product on the tensor cores
// (tile_products.cu), which multiplies e4m3 numbers exactly, applies both scales (powers of
// two) and sums in fp32. 2 M N K operations at the 8-bit rate bound it, or reading the matrix
// for few rows.
#include <algorithm>

#include "op_launch.h"
#include "pack8_layout.h"
#include "tile_products.h"

#define CAM_API extern "C" __attribute__((visibility("default")))

namespace cam {
namespace {

int check8(const char* fn, int64_t tokens, int64_t rows, int64_t cols) {
    if (const int rc = p8_check(fn, rows, cols)) return rc;
    if (tokens < 0 || tokens > (int64_t(1) << 24))
        return record_error(CAM_E_ARG, "%s: tokens out of range", fn);
    // (tiles are counted in 32 bits)
    if ((tokens + 127) / 128 * ((rows + kTileCols8 - 1) / kTileCols8) > (int64_t(1) << 30))
        return record_error(CAM_E_ARG, "%s: tokens and rows out of range", fn);
    return CAM_OK;
}

TileOperand operand8(const void* packed, int64_t rows, int64_t cols) {
    TileOperand o{};
    o.base = packed;
    o.rows = rows;
    o.k = cols;
    o.ld = p8_ld(cols);
    o.planes = 1;
    o.scales = static_cast<const char*>(packed) + p8_q_bytes(rows, cols);
    return o;
}

}  // namespace
}  // namespace cam

using cam::record_error;

CAM_API int cam_matmul8_workspace(int64_t tokens, int64_t rows, int64_t cols, int64_t* bytes) {
    const char* fn = "cam_matmul8_workspace";
    if (!bytes) return record_error(CAM_E_ARG, "%s: bytes is NULL", fn);
    if (const int rc = cam::check8(fn, tokens, rows, cols)) return rc;
    *bytes = rows ? cam::p8_bytes(tokens, cols) : 0;
    return CAM_OK;
}

CAM_API int cam_matmul8(int64_t tokens, int64_t rows, int64_t cols, const void* x, int64_t x_stride,
                        cam_dtype x_dtype, const void* packed, void* y, int64_t y_stride,
                        cam_dtype y_dtype, void* workspace, int64_t workspace_bytes, void* stream) {
    using namespace cam;
    const char* fn = "cam_matmul8";
    if (const int rc = check8(fn, tokens, rows, cols)) return rc;
    for (const cam_dtype d : {x_dtype, y_dtype})
        if (d != CAM_F32 && d != CAM_BF16)
            return record_error(CAM_E_ARG, "%s: unknown dtype %d", fn, static_cast<int>(d));
    if (tokens == 0 || rows == 0) return CAM_OK;
    if (!y || (cols > 0 && (!x || !packed)))
        return record_error(CAM_E_ARG, "%s: a pointer is NULL", fn);
    if (x_stride < cols || x_stride > (int64_t(1) << 34) || y_stride < rows ||
        y_stride > (int64_t(1) << 34))
        return record_error(CAM_E_ARG, "%s: stride out of range", fn);
    if (reinterpret_cast<uintptr_t>(packed) % 16 != 0)
        return record_error(CAM_E_ARG, "%s: packed is not 16-byte aligned", fn);
    const int x_size = x_dtype == CAM_F32 ? 4 : 2, y_size = y_dtype == CAM_F32 ? 4 : 2;
    if (reinterpret_cast<uintptr_t>(x) % x_size != 0 || reinterpret_cast<uintptr_t>(y) % y_size != 0)
        return record_error(CAM_E_ARG, "%s: an array is not aligned to its elements", fn);
    const int64_t need = p8_bytes(tokens, cols);
    if (need > 0 && (!workspace || reinterpret_cast<uintptr_t>(workspace) % 256 != 0))
        return record_error(CAM_E_ARG, "%s: workspace is NULL or not 256-byte aligned", fn);
    if (workspace_bytes < need)
        return record_error(CAM_E_ARG, "%s: workspace of %lld bytes, %lld needed", fn,
                            static_cast<long long>(workspace_bytes), static_cast<long long>(need));
    int dev = 0, sms = 0;
    cudaError_t ce = current_device(&dev, &sms);
    if (ce != cudaSuccess)
        return record_error(CAM_E_CUDA, "%s: no usable CUDA device: %s", fn, cudaGetErrorString(ce));
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    if (cols == 0) {
        ce = cudaMemset2DAsync(y, y_stride * y_size, 0, rows * y_size, tokens, s);
        return ce == cudaSuccess
                   ? CAM_OK
                   : record_error(CAM_E_CUDA, "%s: %s", fn, cudaGetErrorString(ce));
    }
    if (const int rc = p8_pack(fn, tokens, cols, x, x_stride, x_dtype, workspace, s)) return rc;
    TileProduct t{};
    t.a = operand8(workspace, tokens, cols);
    t.b = operand8(packed, rows, cols);
    t.splits = 1;
    t.out.y = y;
    t.out.ldy = y_stride;
    t.out.y_bf16 = y_dtype == CAM_BF16;
    return tile_products(fn, &t, 1, true, tokens > 128, kTileOut, sms, s);
}
