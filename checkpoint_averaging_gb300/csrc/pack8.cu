// pack8.cu -- the 8-bit form of a matrix (cam_pack8) and back (cam_unpack8).
//
// Per 128 columns of a row, e is the least integer >= -126 with max|w| <= 448 * 2^e and
// q = e4m3(w * 2^-e), round to nearest even. The scale is a power of two so that w * 2^-e
// is exact (the one rounding is e4m3's) and the tensor core can apply it (UE8M0).
//
// One pass over the matrix; HBM bounds it. A warp takes the same 128 columns of eight rows,
// four columns per lane, all in flight at once, and the largest magnitude is one
// integer warp reduction (of the bits without sign: NaN and infinity come out above
// every number).
#include <cuda_bf16.h>
#include <cuda_fp8.h>

#include <algorithm>

#include "op_launch.h"
#include "pack8_layout.h"

#define CAM_API extern "C" __attribute__((visibility("default")))

namespace cam {
namespace {

constexpr int kThreads8 = 128;  // (256: 5 % slower)
constexpr int kRowsAtOnce = 8;  // of a warp, in flight

// Four columns of a row as they lie in memory: loaded first, widened when all of a warp's rows
// are on their way (a load that is widened at once is waited for at once: 55,668 x 2,704 bf16
// took 248 us that way).
struct Four {
    uint32_t w[4];
};

// From rows that start on four columns' bytes (`vec`), or of any alignment: fp32 one by one,
// bf16 as the two or three aligned words that hold them. n: columns inside the matrix.
template <typename T>
__device__ __forceinline__ Four load4(const T* p, int n, bool vec) {
    Four f{{0, 0, 0, 0}};
    if (n < 4) {
#pragma unroll
        for (int i = 0; i < 3; ++i)
            if (i < n) {
                if constexpr (sizeof(T) == 4) f.w[i] = __float_as_uint(p[i]);
                else f.w[i / 2] |= uint32_t(__bfloat16_as_ushort(p[i])) << (16 * (i & 1));
            }
    } else if constexpr (sizeof(T) == 4) {
        if (vec) {
            const uint4 x = *reinterpret_cast<const uint4*>(p);
            f.w[0] = x.x, f.w[1] = x.y, f.w[2] = x.z, f.w[3] = x.w;
        } else {
#pragma unroll
            for (int i = 0; i < 4; ++i) f.w[i] = __float_as_uint(p[i]);
        }
    } else if (vec) {
        const uint2 x = *reinterpret_cast<const uint2*>(p);
        f.w[0] = x.x, f.w[1] = x.y;
    } else {
        const uintptr_t at = reinterpret_cast<uintptr_t>(p);
        const uint32_t* w = reinterpret_cast<const uint32_t*>(at & ~uintptr_t(3));
        f.w[0] = w[0], f.w[1] = w[1];
        if (at & 2) f.w[2] = w[2];
    }
    return f;
}

template <typename T>
__device__ __forceinline__ void widen4(const Four& f, const T* p, int n, float* v) {
    if constexpr (sizeof(T) == 4) {
#pragma unroll
        for (int i = 0; i < 4; ++i) v[i] = __uint_as_float(f.w[i]);
    } else {
        const bool odd = n >= 4 && (reinterpret_cast<uintptr_t>(p) & 2);
        const uint32_t x = odd ? __funnelshift_r(f.w[0], f.w[1], 16) : f.w[0];
        const uint32_t y = odd ? __funnelshift_r(f.w[1], f.w[2], 16) : f.w[1];
        v[0] = __uint_as_float(x << 16), v[1] = __uint_as_float(x & 0xFFFF0000u);
        v[2] = __uint_as_float(y << 16), v[3] = __uint_as_float(y & 0xFFFF0000u);
    }
}

// u / d, in 32 bits where they suffice.
__device__ __forceinline__ int64_t quotient(int64_t u, int32_t d) {
    return u >> 32 ? u / d : static_cast<int64_t>(static_cast<uint32_t>(u) / static_cast<uint32_t>(d));
}

// q and scale of a block, of which this lane holds four columns.
__device__ __forceinline__ uint32_t quantise(float* v, uint32_t* scale) {
    uint32_t top = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i) top = max(top, __float_as_uint(v[i]) & 0x7FFFFFFFu);
    top = __reduce_max_sync(0xFFFFFFFFu, top);
    if (top >= 0x7F800000u) {  // a NaN or an infinity: the block stands for NaN
        *scale = 127;
        return 0x7F7F7F7Fu;
    }
    // max|w| = f 2^x with f in [1, 2): 448 = 1.75 2^8, so e = x - 8, or x - 7 for f > 1.75
    const int e = max(static_cast<int>(top >> 23) - 127 - 8 + ((top & 0x7FFFFFu) > 0x600000u), -126);
    *scale = static_cast<uint32_t>(e + 127);
    if (e == 120) {  // 256 * 2^120 would be an infinity
#pragma unroll
        for (int i = 0; i < 4; ++i) v[i] = fminf(fmaxf(v[i], -240.0f * 0x1p120f), 240.0f * 0x1p120f);
    }
    const float r = __uint_as_float(static_cast<uint32_t>(127 - e) << 23);  // 2^-e, e <= 120
    const __nv_fp8x2_storage_t lo =
        __nv_cvt_float2_to_fp8x2(make_float2(v[0] * r, v[1] * r), __NV_SATFINITE, __NV_E4M3);
    const __nv_fp8x2_storage_t hi =
        __nv_cvt_float2_to_fp8x2(make_float2(v[2] * r, v[3] * r), __NV_SATFINITE, __NV_E4M3);
    return static_cast<uint32_t>(lo) | (static_cast<uint32_t>(hi) << 16);
}

// The word of a row's scale: lane r % 32 of the block of 128 rows, column r / 32 % 4.
__device__ __forceinline__ int64_t scale_at(int64_t row, int32_t kb, int64_t row_blocks) {
    return (int64_t(kb) * row_blocks + row / 128) * 128 + (row % 32) * 4 + row / 32 % 4;
}

// Unit u of the grid's warps: eight rows of one block of columns; units of the same rows
// are neighbours. Rows up to the next multiple of 128 have a scale, too.
template <typename T>
__global__ void __launch_bounds__(kThreads8) pack8_kernel(int64_t rows, int64_t cols, const T* w,
                                                          int64_t stride, bool vec, uint8_t* q,
                                                          int64_t ld, uint32_t* scales,
                                                          int32_t col_blocks, int64_t units) {
    asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    const int lane = threadIdx.x & 31;
    const int64_t row_blocks = (rows + 127) / 128;
    for (int64_t u = (int64_t(blockIdx.x) * kThreads8 + threadIdx.x) >> 5; u < units;
         u += int64_t(gridDim.x) * (kThreads8 / 32)) {
        const int64_t group = quotient(u, col_blocks);
        const int32_t kb = static_cast<int32_t>(u - group * col_blocks);
        const int64_t row0 = group * kRowsAtOnce;
        const int64_t col = int64_t(kb) * kP8Block + 4 * lane;
        const int n = static_cast<int>(min(int64_t(4), max(int64_t(0), cols - col)));
        uint32_t mine = 127;
        Four f[kRowsAtOnce];
#pragma unroll
        for (int r = 0; r < kRowsAtOnce; ++r)
            f[r] = load4(w + (row0 + r) * stride + col, row0 + r < rows ? n : 0, vec);
#pragma unroll
        for (int r = 0; r < kRowsAtOnce; ++r) {
            float v[4];
            widen4(f[r], w + (row0 + r) * stride + col, n, v);
            uint32_t scale;
            const uint32_t four = quantise(v, &scale);
            if (lane == r && row0 + r < rows) mine = scale;
            if (row0 + r < rows && col < ld)
                *reinterpret_cast<uint32_t*>(q + (row0 + r) * ld + col) = four;
        }
        if (lane < kRowsAtOnce) scales[scale_at(row0 + lane, kb, row_blocks)] = mine * 0x01010101u;
    }
}

template <typename T>
__device__ __forceinline__ void store4(T* p, int n, bool vec, const float* v) {
    if (vec && n >= 4) {
        if constexpr (sizeof(T) == 4) {
            *reinterpret_cast<float4*>(p) = make_float4(v[0], v[1], v[2], v[3]);
        } else {
            const __nv_bfloat162 a = __floats2bfloat162_rn(v[0], v[1]);
            const __nv_bfloat162 b = __floats2bfloat162_rn(v[2], v[3]);
            *reinterpret_cast<uint2*>(p) = make_uint2(*reinterpret_cast<const uint32_t*>(&a),
                                                      *reinterpret_cast<const uint32_t*>(&b));
        }
    } else if (sizeof(T) == 2 && n >= 4 && reinterpret_cast<uintptr_t>(p) % 4 == 0) {
        const __nv_bfloat162 a = __floats2bfloat162_rn(v[0], v[1]);
        const __nv_bfloat162 b = __floats2bfloat162_rn(v[2], v[3]);
        reinterpret_cast<uint32_t*>(p)[0] = *reinterpret_cast<const uint32_t*>(&a);
        reinterpret_cast<uint32_t*>(p)[1] = *reinterpret_cast<const uint32_t*>(&b);
    } else {
#pragma unroll
        for (int i = 0; i < 4; ++i)
            if (i < n) p[i] = T(v[i]);
    }
}

// The values q 2^e: four columns per lane, as pack8_kernel reads them.
template <typename T>
__global__ void __launch_bounds__(kThreads8) unpack8_kernel(int64_t rows, int64_t cols, T* out,
                                                            int64_t stride, bool vec, const uint8_t* q,
                                                            int64_t ld, const uint32_t* scales,
                                                            int32_t col_blocks, int64_t units) {
    const int lane = threadIdx.x & 31;
    const int64_t row_blocks = (rows + 127) / 128;
    for (int64_t u = (int64_t(blockIdx.x) * kThreads8 + threadIdx.x) >> 5; u < units;
         u += int64_t(gridDim.x) * (kThreads8 / 32)) {
        const int64_t group = quotient(u, col_blocks);
        const int32_t kb = static_cast<int32_t>(u - group * col_blocks);
        const int64_t row0 = group * kRowsAtOnce;
        const int64_t col = int64_t(kb) * kP8Block + 4 * lane;
        const int n = static_cast<int>(min(int64_t(4), max(int64_t(0), cols - col)));
        const uint32_t mine =
            lane < kRowsAtOnce ? scales[scale_at(row0 + lane, kb, row_blocks)] & 0xFFu : 0u;
        uint32_t four[kRowsAtOnce];
#pragma unroll
        for (int r = 0; r < kRowsAtOnce; ++r)
            four[r] = row0 + r < rows && n > 0
                          ? *reinterpret_cast<const uint32_t*>(q + (row0 + r) * ld + col)
                          : 0u;
#pragma unroll
        for (int r = 0; r < kRowsAtOnce; ++r) {
            // 2^e, e in [-126, 120]
            const float s = __uint_as_float(__shfl_sync(0xFFFFFFFFu, mine, r) << 23);
            float v[4];
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                const __half2_raw h = __nv_cvt_fp8x2_to_halfraw2(
                    static_cast<__nv_fp8x2_storage_t>(four[r] >> (16 * i)), __NV_E4M3);
                const float2 f = __half22float2(__half2(h));
                v[2 * i] = f.x * s;
                v[2 * i + 1] = f.y * s;
            }
            if (row0 + r < rows) store4(out + (row0 + r) * stride + col, n, vec, v);
        }
    }
}

bool vec_aligned(const void* p, int64_t stride, int64_t bytes, int64_t size) {
    return reinterpret_cast<uintptr_t>(p) % bytes == 0 && stride * size % bytes == 0;
}

// Blocks for `units` warps, one each.
cudaError_t grid_for(int64_t units, int* blocks) {
    int dev = 0, sms = 0;
    const cudaError_t ce = current_device(&dev, &sms);
    *blocks = static_cast<int>(
        std::max<int64_t>(1, std::min<int64_t>((units + kThreads8 / 32 - 1) / (kThreads8 / 32),
                                               int64_t(1) << 30)));
    return ce;
}

int check(const char* fn, int64_t rows, int64_t cols, const void* m, int64_t stride,
          cam_dtype dtype, const void* packed) {
    if (const int rc = p8_check(fn, rows, cols)) return rc;
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

}  // namespace

int p8_pack(const char* fn, int64_t rows, int64_t cols, const void* w, int64_t stride,
            cam_dtype dtype, void* packed, cudaStream_t s) {
    const int size = dtype == CAM_F32 ? 4 : 2;
    int32_t col_blocks = static_cast<int32_t>((cols + kP8Block - 1) / kP8Block);
    // (whole blocks of 128 rows, so that every scale of the form is written)
    int64_t units = (rows + 127) / 128 * (128 / kRowsAtOnce) * col_blocks;
    int64_t ld = p8_ld(cols);
    bool vec = vec_aligned(w, stride, 4 * size, size);
    uint8_t* q = static_cast<uint8_t*>(packed);
    uint32_t* scales = reinterpret_cast<uint32_t*>(q + p8_q_bytes(rows, cols));
    int blocks = 0;
    cudaError_t ce = grid_for(units, &blocks);
    if (ce == cudaSuccess) {
        void* args[] = {&rows, &cols, &w, &stride, &vec, &q, &ld, &scales, &col_blocks, &units};
        cudaLaunchConfig_t cfg{};
        cfg.gridDim = dim3(blocks);
        cfg.blockDim = dim3(kThreads8);
        cfg.stream = s;
        cudaLaunchAttribute at{};
        at.id = cudaLaunchAttributeProgrammaticStreamSerialization;
        at.val.programmaticStreamSerializationAllowed = 1;
        cfg.attrs = &at;
        cfg.numAttrs = 1;
        ce = cudaLaunchKernelExC(&cfg,
                                 dtype == CAM_F32 ? reinterpret_cast<const void*>(pack8_kernel<float>)
                                                  : reinterpret_cast<const void*>(pack8_kernel<__nv_bfloat16>),
                                 args);
    }
    if (ce != cudaSuccess)
        return record_error(CAM_E_CUDA, "%s: launch: %s", fn, cudaGetErrorString(ce));
    return CAM_OK;
}

}  // namespace cam

using cam::record_error;

CAM_API int cam_pack8_bytes(int64_t rows, int64_t cols, int64_t* out) {
    const char* fn = "cam_pack8_bytes";
    if (!out) return record_error(CAM_E_ARG, "%s: out is NULL", fn);
    if (const int rc = cam::p8_check(fn, rows, cols)) return rc;
    *out = cam::p8_bytes(rows, cols);
    return CAM_OK;
}

CAM_API int cam_pack8(int64_t rows, int64_t cols, const void* w, int64_t stride, cam_dtype dtype,
                      void* packed, void* stream) {
    const char* fn = "cam_pack8";
    if (const int rc = cam::check(fn, rows, cols, w, stride, dtype, packed)) return rc;
    if (rows == 0 || cols == 0) return CAM_OK;
    return cam::p8_pack(fn, rows, cols, w, stride, dtype, packed, static_cast<cudaStream_t>(stream));
}

CAM_API int cam_unpack8(int64_t rows, int64_t cols, const void* packed, void* values,
                        int64_t stride, cam_dtype dtype, void* stream) {
    const char* fn = "cam_unpack8";
    if (const int rc = cam::check(fn, rows, cols, values, stride, dtype, packed)) return rc;
    if (rows == 0 || cols == 0) return CAM_OK;
    const int size = dtype == CAM_F32 ? 4 : 2;
    int32_t col_blocks = static_cast<int32_t>((cols + cam::kP8Block - 1) / cam::kP8Block);
    int64_t units = (rows + cam::kRowsAtOnce - 1) / cam::kRowsAtOnce * col_blocks;
    int64_t ld = cam::p8_ld(cols);
    bool vec = cam::vec_aligned(values, stride, 4 * size, size);
    const uint8_t* q = static_cast<const uint8_t*>(packed);
    const uint32_t* scales =
        reinterpret_cast<const uint32_t*>(q + cam::p8_q_bytes(rows, cols));
    int blocks = 0;
    cudaError_t ce = cam::grid_for(units, &blocks);
    if (ce == cudaSuccess) {
        void* args[] = {&rows, &cols, &values, &stride, &vec, &q, &ld, &scales, &col_blocks, &units};
        ce = cudaLaunchKernel(dtype == CAM_F32
                                  ? reinterpret_cast<const void*>(cam::unpack8_kernel<float>)
                                  : reinterpret_cast<const void*>(cam::unpack8_kernel<__nv_bfloat16>),
                              dim3(blocks), dim3(cam::kThreads8), args, 0,
                              static_cast<cudaStream_t>(stream));
    }
    if (ce != cudaSuccess)
        return record_error(CAM_E_CUDA, "%s: launch: %s", fn, cudaGetErrorString(ce));
    return CAM_OK;
}
