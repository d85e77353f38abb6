// pack4.cu -- cam_pack4 and cam_unpack4: a merged global's matrix into the
// 4-bit form and back (declarations and the form's definition in
// include/cam.h, its layout in pack4_layout.h).
//
// Both are streaming, HBM-bound: 4 B (fp32) or 2 B (bf16) per weight on one
// side, 1/2 + 2 / group B on the other. One warp makes one tile of 16 rows x
// 128 columns: a row of the tile is one 16-byte (fp32) or 8-byte (bf16) load
// per lane, all rows' loads in flight before the first use; a group's largest
// magnitude is a shuffle reduction among the 8, 16 or 32 lanes that hold it.
#include <cuda_runtime.h>

#include <algorithm>

#include "cam_internal.h"
#include "pack4_layout.h"

#define CAM_API extern "C" __attribute__((visibility("default")))

namespace cam {
namespace {

constexpr int kPkThreads = 256;

// Four columns of one row, widened to fp32; columns past the end are 0.
__device__ __forceinline__ void load4(const float* p, int n, bool vec, float (&v)[4]) {
    if (vec && n >= 4) {
        asm volatile("ld.global.nc.L1::no_allocate.v4.f32 {%0,%1,%2,%3}, [%4];"
                     : "=f"(v[0]), "=f"(v[1]), "=f"(v[2]), "=f"(v[3])
                     : "l"(p));
        return;
    }
#pragma unroll
    for (int j = 0; j < 4; ++j) v[j] = j < n ? __ldg(p + j) : 0.0f;
}

__device__ __forceinline__ void load4(const uint16_t* p, int n, bool vec, float (&v)[4]) {
    if (vec && n >= 4) {
        uint32_t a, b;
        asm volatile("ld.global.nc.L1::no_allocate.v2.b32 {%0,%1}, [%2];"
                     : "=r"(a), "=r"(b)
                     : "l"(p));
        v[0] = __uint_as_float(a << 16);
        v[1] = __uint_as_float(a & 0xFFFF0000u);
        v[2] = __uint_as_float(b << 16);
        v[3] = __uint_as_float(b & 0xFFFF0000u);
        return;
    }
#pragma unroll
    for (int j = 0; j < 4; ++j)
        v[j] = j < n ? __uint_as_float(static_cast<uint32_t>(__ldg(p + j)) << 16) : 0.0f;
}

__device__ __forceinline__ uint32_t to_bf16(float v) {  // nearest-even; NaN stays NaN
    const uint32_t u = __float_as_uint(v);
    if ((u & 0x7FFFFFFFu) > 0x7F800000u) return 0x7FFFu;
    return (u + 0x7FFFu + ((u >> 16) & 1u)) >> 16;
}

__device__ __forceinline__ void store4(float* p, int n, bool vec, const float (&v)[4]) {
    if (vec && n >= 4) {
        __stcs(reinterpret_cast<float4*>(p), make_float4(v[0], v[1], v[2], v[3]));
        return;
    }
#pragma unroll
    for (int j = 0; j < 4; ++j)
        if (j < n) p[j] = v[j];
}

__device__ __forceinline__ void store4(uint16_t* p, int n, bool vec, const float (&v)[4]) {
    if (vec && n >= 4) {
        __stcs(reinterpret_cast<uint2*>(p), make_uint2(to_bf16(v[0]) | (to_bf16(v[1]) << 16),
                                                       to_bf16(v[2]) | (to_bf16(v[3]) << 16)));
        return;
    }
#pragma unroll
    for (int j = 0; j < 4; ++j)
        if (j < n) p[j] = static_cast<uint16_t>(to_bf16(v[j]));
}

template <typename T, int GROUP>
__global__ void __launch_bounds__(kPkThreads)
    pack4(int64_t rows, int64_t cols, const T* __restrict__ w, int64_t stride, bool vec,
          uint8_t* __restrict__ packed, int64_t n_tiles, int32_t tiles_across) {
    constexpr int kPer = kP4Cols / GROUP;
    const int lane = threadIdx.x & 31;
    const int64_t step = int64_t(gridDim.x) * (kPkThreads / 32);
    for (int64_t tile = int64_t(blockIdx.x) * (kPkThreads / 32) + (threadIdx.x >> 5);
         tile < n_tiles; tile += step) {
        const int64_t row0 = tile / tiles_across * kP4Rows;
        const int64_t col = tile % tiles_across * kP4Cols + 4 * lane;
        const int n = static_cast<int>(max(int64_t(0), min(int64_t(4), cols - col)));
        uint8_t* out = packed + tile * p4_tile_bytes(GROUP);
        uint16_t* scales = reinterpret_cast<uint16_t*>(out + kP4Quants);
#pragma unroll
        for (int half = 0; half < 2; ++half) {
            float v[8][4];
#pragma unroll
            for (int r = 0; r < 8; ++r) {
                const int64_t row = row0 + 8 * half + r;
                load4(w + row * stride + col, row < rows ? n : 0, vec, v[r]);
            }
#pragma unroll
            for (int r = 0; r < 8; ++r) {
                // the group's largest magnitude as bits: for non-negative floats the order of
                // the bits is the order of the values, with NaN above infinity
                uint32_t big = 0;
#pragma unroll
                for (int j = 0; j < 4; ++j) big = max(big, __float_as_uint(v[r][j]) & 0x7FFFFFFFu);
#pragma unroll
                for (int o = 1; o < GROUP / 4; o *= 2)
                    big = max(big, __shfl_xor_sync(0xFFFFFFFFu, big, o));
                const bool fine = big < 0x7F800000u;
                uint32_t sb = __float_as_uint(__fdiv_rn(__uint_as_float(big), 7.0f)) & 0xFFFF0000u;
                if (sb < 0x00800000u) sb = 0;  // below 2^-126
                if (!fine) sb = 0x7FC00000u;
                const float inv = sb != 0 && fine ? __frcp_rn(__uint_as_float(sb)) : 0.0f;
                uint32_t word = 0;
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const int q = __float2int_rn(fine ? __fmul_rn(v[r][j], inv) : 0.0f);
                    const uint32_t nib = static_cast<uint32_t>(min(max(q, -7), 7) + 8);
                    // column j of the word's lower (even lane) or upper four: see the layout
                    const int c = 4 * (lane & 1) + j;
                    word |= nib << (4 * ((c >> 1) + 4 * (c & 1)));
                }
                word |= __shfl_xor_sync(0xFFFFFFFFu, word, 1);
                if ((lane & 1) == 0)
                    *reinterpret_cast<uint32_t*>(out + p4_word(8 * half + r, lane >> 1)) = word;
                if (lane % (GROUP / 4) == 0)
                    scales[p4_scale(8 * half + r, lane / (GROUP / 4), kPer)] =
                        static_cast<uint16_t>(sb >> 16);
            }
        }
    }
}

template <typename T, int GROUP>
__global__ void __launch_bounds__(kPkThreads)
    unpack4(int64_t rows, int64_t cols, const uint8_t* __restrict__ packed, T* __restrict__ values,
            int64_t stride, bool vec, int64_t n_tiles, int32_t tiles_across) {
    constexpr int kPer = kP4Cols / GROUP;
    const int lane = threadIdx.x & 31;
    const int64_t step = int64_t(gridDim.x) * (kPkThreads / 32);
    for (int64_t tile = int64_t(blockIdx.x) * (kPkThreads / 32) + (threadIdx.x >> 5);
         tile < n_tiles; tile += step) {
        const int64_t row0 = tile / tiles_across * kP4Rows;
        const int64_t col = tile % tiles_across * kP4Cols + 4 * lane;
        const int n = static_cast<int>(max(int64_t(0), min(int64_t(4), cols - col)));
        const uint8_t* in = packed + tile * p4_tile_bytes(GROUP);
        const uint16_t* scales = reinterpret_cast<const uint16_t*>(in + kP4Quants);
        uint32_t word[kP4Rows];
        float s[kP4Rows];
#pragma unroll
        for (int r = 0; r < kP4Rows; ++r) {
            word[r] = __ldg(reinterpret_cast<const uint32_t*>(in + p4_word(r, lane >> 1)));
            s[r] = __uint_as_float(
                static_cast<uint32_t>(__ldg(scales + p4_scale(r, lane / (GROUP / 4), kPer))) << 16);
        }
#pragma unroll
        for (int r = 0; r < kP4Rows; ++r) {
            const int64_t row = row0 + r;
            if (row >= rows) break;
            float v[4];
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const int c = 4 * (lane & 1) + j;
                const int nib = (word[r] >> (4 * ((c >> 1) + 4 * (c & 1)))) & 15;
                v[j] = __fmul_rn(static_cast<float>(nib - 8), s[r]);
            }
            store4(values + row * stride + col, n, vec, v);
        }
    }
}

// A launch of one warp per tile, at most 8 blocks per SM resident at once.
int blocks_for(int64_t n_tiles) {
    return static_cast<int>(std::min<int64_t>((n_tiles + kPkThreads / 32 - 1) / (kPkThreads / 32),
                                              int64_t(1) << 30));
}

bool row_aligned(const void* p, int64_t stride, int size, uintptr_t n) {
    return reinterpret_cast<uintptr_t>(p) % n == 0 && stride * size % static_cast<int64_t>(n) == 0;
}

int check_matrix(const char* fn, int64_t rows, int64_t cols, const void* m, int64_t stride,
                 cam_dtype dtype, int32_t group, const void* packed) {
    if (const int rc = p4_check(fn, rows, cols, group)) return rc;
    if (dtype != CAM_F32 && dtype != CAM_BF16)
        return record_error(CAM_E_ARG, "%s: unknown dtype %d", fn, static_cast<int>(dtype));
    if (rows == 0 || cols == 0) return CAM_OK;
    if (!m || !packed) return record_error(CAM_E_ARG, "%s: a pointer is NULL", fn);
    if (stride < cols || stride > (int64_t(1) << 58) / rows)
        return record_error(CAM_E_ARG, "%s: stride out of range", fn);
    if (reinterpret_cast<uintptr_t>(packed) % 16 != 0)
        return record_error(CAM_E_ARG, "%s: packed is not 16-byte aligned", fn);
    if (reinterpret_cast<uintptr_t>(m) % (dtype == CAM_F32 ? 4 : 2) != 0)
        return record_error(CAM_E_ARG, "%s: the matrix is not aligned to its elements", fn);
    return CAM_OK;
}

template <typename T>
const void* pack_kernel(int32_t group) {
    return group == 32   ? reinterpret_cast<const void*>(pack4<T, 32>)
           : group == 64 ? reinterpret_cast<const void*>(pack4<T, 64>)
                         : reinterpret_cast<const void*>(pack4<T, 128>);
}

template <typename T>
const void* unpack_kernel(int32_t group) {
    return group == 32   ? reinterpret_cast<const void*>(unpack4<T, 32>)
           : group == 64 ? reinterpret_cast<const void*>(unpack4<T, 64>)
                         : reinterpret_cast<const void*>(unpack4<T, 128>);
}

}  // namespace
}  // namespace cam

using cam::record_error;

CAM_API int cam_pack4_bytes(int64_t rows, int64_t cols, int32_t group, int64_t* out) {
    const char* fn = "cam_pack4_bytes";
    if (!out) return record_error(CAM_E_ARG, "%s: out is NULL", fn);
    if (const int rc = cam::p4_check(fn, rows, cols, group)) return rc;
    *out = cam::p4_bytes(rows, cols, group);
    return CAM_OK;
}

CAM_API int cam_pack4(int64_t rows, int64_t cols, const void* w, int64_t stride, cam_dtype dtype,
                      int32_t group, void* packed, void* stream) {
    const char* fn = "cam_pack4";
    if (const int rc = cam::check_matrix(fn, rows, cols, w, stride, dtype, group, packed)) return rc;
    if (rows == 0 || cols == 0) return CAM_OK;
    int32_t across = static_cast<int32_t>((cols + cam::kP4Cols - 1) / cam::kP4Cols);
    int64_t tiles = (rows + cam::kP4Rows - 1) / cam::kP4Rows * across;
    const int size = dtype == CAM_F32 ? 4 : 2;
    bool vec = cam::row_aligned(w, stride, size, 4 * size);
    void* args[] = {&rows, &cols, &w, &stride, &vec, &packed, &tiles, &across};
    const cudaError_t ce = cudaLaunchKernel(
        dtype == CAM_F32 ? cam::pack_kernel<float>(group) : cam::pack_kernel<uint16_t>(group),
        dim3(cam::blocks_for(tiles)), dim3(cam::kPkThreads), args, 0,
        static_cast<cudaStream_t>(stream));
    if (ce != cudaSuccess)
        return record_error(CAM_E_CUDA, "%s: launch: %s", fn, cudaGetErrorString(ce));
    return CAM_OK;
}

CAM_API int cam_unpack4(int64_t rows, int64_t cols, const void* packed, int32_t group,
                        void* values, int64_t stride, cam_dtype dtype, void* stream) {
    const char* fn = "cam_unpack4";
    if (const int rc = cam::check_matrix(fn, rows, cols, values, stride, dtype, group, packed))
        return rc;
    if (rows == 0 || cols == 0) return CAM_OK;
    int32_t across = static_cast<int32_t>((cols + cam::kP4Cols - 1) / cam::kP4Cols);
    int64_t tiles = (rows + cam::kP4Rows - 1) / cam::kP4Rows * across;
    const int size = dtype == CAM_F32 ? 4 : 2;
    bool vec = cam::row_aligned(values, stride, size, 4 * size);
    void* args[] = {&rows, &cols, &packed, &values, &stride, &vec, &tiles, &across};
    const cudaError_t ce = cudaLaunchKernel(
        dtype == CAM_F32 ? cam::unpack_kernel<float>(group) : cam::unpack_kernel<uint16_t>(group),
        dim3(cam::blocks_for(tiles)), dim3(cam::kPkThreads), args, 0,
        static_cast<cudaStream_t>(stream));
    if (ce != cudaSuccess)
        return record_error(CAM_E_CUDA, "%s: launch: %s", fn, cudaGetErrorString(ce));
    return CAM_OK;
}
