// pack4.cu -- cam_pack4 and cam_unpack4: a merged global's matrix into the
// 4-bit form and back (declarations and the form's definition in
// include/cam.h, its layout in pack4_layout.h).
//
// Both are streaming, HBM-bound: 4 B (fp32) or 2 B (bf16) per weight on one
// side, 1/2 + 2 / group B on the other. One warp takes one tile of 16 rows x
// 128 columns, its loads in flight before their first use; four blocks of
// eight warps per SM (with two or three the bf16 pass took 82 and 68 us where
// four took 64). Measured with 20,000 rows, group 32: 6,160 fp32 columns 85 us to
// pack and to unpack (6.6 TB/s), bf16 61 us (5.1 TB/s: the scales' and roundings'
// instructions) and 48 us (6.6 TB/s); rows without alignment (6,159 columns) 95
// and 91 us in fp32, 85 and 82 us in bf16.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <algorithm>

#include "cam_internal.h"
#include "pack4_layout.h"

#define CAM_API extern "C" __attribute__((visibility("default")))

namespace cam {
namespace {

constexpr int kPkThreads = 256;

__device__ __forceinline__ float widen(uint32_t bits) { return __uint_as_float(bits << 16); }
__device__ __forceinline__ float load1(const uint16_t* p) { return widen(__ldg(p)); }

__device__ __forceinline__ uint4 load_word(const uint16_t* p) {
    uint4 v;
    asm volatile("ld.global.nc.L1::no_allocate.v4.b32 {%0,%1,%2,%3}, [%4];"
                 : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
                 : "l"(p));
    return v;
}

// Eight columns of a row as loaded. `fetch` reads them from a row aligned to 16
// bytes (`eight`: to eight elements), columns past the end as 0. Rows without
// that alignment, as every odd number of columns gives, are read four bytes to
// a lane, so that a load is still one run of memory (`gather`, of the row's 128
// columns), and turned in shared memory (`put`, then `take`). (That alone takes
// 168 us for the 20,000 x 6,159 bf16; see pack4 for tiles inside the rows.)
template <typename T>
struct Eight;

template <>
struct Eight<float> {
    static constexpr int kBatch = 4;  // steps of two rows whose loads are in flight together
    float v[8];
    struct Row {
        float e[4];
    };
    __device__ __forceinline__ void fetch(const float* p, int n, bool eight) {
        if (eight && n >= 8) {
            asm volatile(
                "ld.global.nc.L1::no_allocate.L2::evict_first.v8.f32 "
                "{%0,%1,%2,%3,%4,%5,%6,%7}, [%8];"
                : "=f"(v[0]), "=f"(v[1]), "=f"(v[2]), "=f"(v[3]), "=f"(v[4]), "=f"(v[5]),
                  "=f"(v[6]), "=f"(v[7])
                : "l"(p));
            return;
        }
        if (n >= 8) {
#pragma unroll
            for (int h = 0; h < 2; ++h)
                asm volatile("ld.global.nc.L1::no_allocate.v4.f32 {%0,%1,%2,%3}, [%4];"
                             : "=f"(v[4 * h]), "=f"(v[4 * h + 1]), "=f"(v[4 * h + 2]),
                               "=f"(v[4 * h + 3])
                             : "l"(p + 4 * h));
            return;
        }
#pragma unroll
        for (int j = 0; j < 8; ++j) v[j] = j < n ? __ldg(p + j) : 0.0f;
    }
    // n: the row's columns from p on (0 for a row past the end)
    static __device__ __forceinline__ void gather(Row& r, const float* p, int n, int lane) {
#pragma unroll
        for (int i = 0; i < 4; ++i) r.e[i] = lane + 32 * i < n ? __ldg(p + lane + 32 * i) : 0.0f;
    }
    static __device__ __forceinline__ void put(const Row& r, uint32_t* turn, int lane) {
#pragma unroll
        for (int i = 0; i < 4; ++i) turn[lane + 32 * i] = __float_as_uint(r.e[i]);
    }
    __device__ __forceinline__ void take(const uint32_t* turn, int run, const float*) {
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const float4 f = *reinterpret_cast<const float4*>(turn + 8 * run + 4 * h);
            v[4 * h] = f.x, v[4 * h + 1] = f.y, v[4 * h + 2] = f.z, v[4 * h + 3] = f.w;
        }
    }
    __device__ __forceinline__ float get(int j) const { return v[j]; }
};

template <>
struct Eight<uint16_t> {
    static constexpr int kBatch = 8;
    uint32_t u[4];
    // Word j of a row that starts in the upper half of a word (odd) has columns 2 j - 1 and
    // 2 j, else 2 j and 2 j + 1.
    struct Row {
        uint32_t e[3];
    };
    static __device__ __forceinline__ int odd(const uint16_t* p) {
        return static_cast<int>(reinterpret_cast<uintptr_t>(p) >> 1) & 1;
    }
    __device__ __forceinline__ void fetch(const uint16_t* p, int n, bool) {
        if (n >= 8) {
            asm volatile("ld.global.nc.L1::no_allocate.v4.b32 {%0,%1,%2,%3}, [%4];"
                         : "=r"(u[0]), "=r"(u[1]), "=r"(u[2]), "=r"(u[3])
                         : "l"(p));
            return;
        }
#pragma unroll
        for (int j = 0; j < 4; ++j)
            u[j] = (2 * j < n ? __ldg(p + 2 * j) : 0u) |
                   (2 * j + 1 < n ? static_cast<uint32_t>(__ldg(p + 2 * j + 1)) << 16 : 0u);
    }
    static __device__ __forceinline__ void gather(Row& r, const uint16_t* p, int n, int lane) {
        const int o = odd(p);
#pragma unroll
        for (int i = 0; i < 3; ++i) {
            const int j = lane + 32 * i, c = 2 * j - o;
            r.e[i] = 0;
            if (i == 2 && lane > 0) break;  // (word 64 alone)
            if (c >= 0 && c + 1 < n)
                r.e[i] = __ldg(reinterpret_cast<const uint32_t*>(p + c));
            else if (c >= 0 && c < n)
                r.e[i] = __ldg(p + c);
            else if (c == -1 && n > 0)
                r.e[i] = static_cast<uint32_t>(__ldg(p)) << 16;
        }
    }
    static __device__ __forceinline__ void put(const Row& r, uint32_t* turn, int lane) {
        turn[lane] = r.e[0];
        turn[lane + 32] = r.e[1];
        if (lane == 0) turn[64] = r.e[2];
    }
    __device__ __forceinline__ void take(const uint32_t* turn, int run, const uint16_t* p) {
        const uint4 w = *reinterpret_cast<const uint4*>(turn + 4 * run);
        const uint32_t last = turn[4 * run + 4];
        const int by = 16 * odd(p);
        u[0] = __funnelshift_r(w.x, w.y, by);
        u[1] = __funnelshift_r(w.y, w.z, by);
        u[2] = __funnelshift_r(w.z, w.w, by);
        u[3] = __funnelshift_r(w.w, last, by);
    }
    __device__ __forceinline__ float get(int j) const {
        return __uint_as_float((j & 1) ? u[j >> 1] & 0xFFFF0000u : u[j >> 1] << 16);
    }
};

// The 16 bytes that start `by` (0, 2, .. 14) bytes into a and b.
__device__ __forceinline__ uint4 cut(const uint4& a, const uint4& b, int by) {
    const bool two = by & 8, one = by & 4;
    const uint32_t c0 = two ? a.z : a.x, c1 = two ? a.w : a.y, c2 = two ? b.x : a.z;
    const uint32_t c3 = two ? b.y : a.w, c4 = two ? b.z : b.x, c5 = two ? b.w : b.y;
    const uint32_t d0 = one ? c1 : c0, d1 = one ? c2 : c1, d2 = one ? c3 : c2;
    const uint32_t d3 = one ? c4 : c3, d4 = one ? c5 : c4;
    const int half = 8 * (by & 2);
    return make_uint4(__funnelshift_r(d0, d1, half), __funnelshift_r(d1, d2, half),
                      __funnelshift_r(d2, d3, half), __funnelshift_r(d3, d4, half));
}

// A 16-byte word of lane `from` of each W lanes.
template <int W>
__device__ __forceinline__ uint4 word_from(const uint4& v, int from) {
    return make_uint4(__shfl_sync(0xFFFFFFFFu, v.x, from, W), __shfl_sync(0xFFFFFFFFu, v.y, from, W),
                      __shfl_sync(0xFFFFFFFFu, v.z, from, W), __shfl_sync(0xFFFFFFFFu, v.w, from, W));
}

// big / 7 rounded to nearest: the product with 1/7 and one correction by the
// remainder, which an fma gives exactly (Markstein's step); tiny dividends, whose
// remainder may not be exact, divide.
__device__ __forceinline__ float seventh(float big) {
    if (big < 1e-30f) return __fdiv_rn(big, 7.0f);
    constexpr float kSeventh = 1.0f / 7.0f;
    const float q = __fmul_rn(big, kSeventh);
    return __fmaf_rn(__fmaf_rn(-7.0f, q, big), kSeventh, q);
}

// 1 / s rounded to nearest for a normal s of 8 significant bits: one Newton step
// on the hardware's estimate (all 128 significands are tested).
__device__ __forceinline__ float reciprocal(float s) {
    float r;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(s));
    return __fmaf_rn(__fmaf_rn(-s, r, 1.0f), r, r);
}

__device__ __forceinline__ uint32_t to_bf16x2(float lo, float hi) {  // nearest-even
    const __nv_bfloat162 v = __floats2bfloat162_rn(lo, hi);
    return *reinterpret_cast<const uint32_t*>(&v);
}
__device__ __forceinline__ uint16_t to_bf16(float v) {
    return __bfloat16_as_ushort(__float2bfloat16_rn(v));
}

// 16 bytes of a row of which n columns are left.
__device__ __forceinline__ void store16(float* p, int n, const float (&v)[4]) {
    if (n >= 4) {
        __stcs(reinterpret_cast<float4*>(p), make_float4(v[0], v[1], v[2], v[3]));
        return;
    }
#pragma unroll
    for (int j = 0; j < 4; ++j)
        if (j < n) p[j] = v[j];
}

__device__ __forceinline__ void store16(uint16_t* p, int n, const float (&v)[8]) {
    if (n >= 8) {
        uint32_t u[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) u[j] = to_bf16x2(v[2 * j], v[2 * j + 1]);
        __stcs(reinterpret_cast<uint4*>(p), make_uint4(u[0], u[1], u[2], u[3]));
        return;
    }
#pragma unroll
    for (int j = 0; j < 8; ++j)
        if (j < n) p[j] = to_bf16(v[j]);
}

// One warp makes one tile: 16 lanes to a row, a lane to one word of 8 columns.
// An integer is rounded by adding 1.5 * 2^23 (+ 8, the nibbles' offset), whose
// last place is 1: the sum's low bits are q + 8, and as its high bits are the
// same for all, eight sums shifted to their nibbles and added, less what the
// high bits add up to, are the word. |w| (1 / s) is at most 7.06, so q never
// needs holding to [-7, 7].
template <typename T, int GROUP, bool ALIGNED>
__global__ void __launch_bounds__(kPkThreads, 4)
    pack4(int64_t rows, int64_t cols, const T* __restrict__ w, int64_t stride, bool eight,
          uint8_t* __restrict__ packed, int64_t n_tiles, int32_t tiles_across) {
    constexpr int kPer = kP4Cols / GROUP;
    constexpr float kRound = 12582912.0f + 8.0f;
    constexpr int kBatch = ALIGNED ? Eight<T>::kBatch : 4;
    constexpr int kTurn = 128 / (4 / sizeof(T)) + 4;  // words of a row, and one more
    __shared__ __align__(16) uint32_t turn[ALIGNED ? 1 : kPkThreads / 32][8][ALIGNED ? 4 : kTurn];
    const int lane = threadIdx.x & 31, run = lane & 15, odd = lane >> 4, warp = threadIdx.x >> 5;
    const int64_t step = int64_t(gridDim.x) * (kPkThreads / 32);
    for (int64_t tile = int64_t(blockIdx.x) * (kPkThreads / 32) + (threadIdx.x >> 5);
         tile < n_tiles; tile += step) {
        const int64_t row0 = tile / tiles_across * kP4Rows + odd;
        const int64_t col = tile % tiles_across * kP4Cols + 8 * run;
        const int n = static_cast<int>(max(int64_t(0), min(int64_t(8), cols - col)));
        uint8_t* out = packed + tile * p4_tile_bytes(GROUP);
        uint16_t* scales = reinterpret_cast<uint16_t*>(out + kP4Quants);
#pragma unroll
        for (int b = 0; b < 8 / kBatch; ++b) {
            Eight<T> v[kBatch];
            if constexpr (ALIGNED) {
#pragma unroll
                for (int r = 0; r < kBatch; ++r) {
                    const int64_t row = row0 + 2 * (b * kBatch + r);
                    v[r].fetch(w + row * stride + col, row < rows ? n : 0, eight);
                }
            } else {
                const int64_t base = tile / tiles_across * kP4Rows;
                const int64_t col0 = tile % tiles_across * kP4Cols;
                const int in_cols = static_cast<int>(min(int64_t(kP4Cols), cols - col0));
                bool done = false;
                if constexpr (sizeof(T) == 2) {
                    // Tiles inside the rows: the 17 aligned words that hold a row's 16 are read whole, and
                    // each lane cuts its eight columns from its word and the next lane's.
                    done = col0 >= 8 && col0 + kP4Cols + 8 <= cols;
                    if (done) {
                        uint4 own[kBatch], end[kBatch];
#pragma unroll
                        for (int r = 0; r < kBatch; ++r) {
                            const int64_t row = row0 + 2 * (b * kBatch + r);
                            const T* at = w + row * stride + col0;
                            at -= reinterpret_cast<uintptr_t>(at) / 2 % 8;
                            own[r] = end[r] = make_uint4(0u, 0u, 0u, 0u);
                            if (row < rows) {
                                own[r] = load_word(at + 8 * run);
                                if (run == 15) end[r] = load_word(at + kP4Cols);
                            }
                        }
#pragma unroll
                        for (int r = 0; r < kBatch; ++r) {
                            const T* at = w + (row0 + 2 * (b * kBatch + r)) * stride + col0;
                            uint4 next = word_from<16>(own[r], (run + 1) & 15);
                            if (run == 15) next = end[r];
                            const uint4 c =
                                cut(own[r], next, static_cast<int>(reinterpret_cast<uintptr_t>(at) & 15));
                            v[r].u[0] = c.x, v[r].u[1] = c.y, v[r].u[2] = c.z, v[r].u[3] = c.w;
                        }
                    }
                }
                if (!done) {
#pragma unroll
                    for (int q = 0; q < kBatch / 4; ++q) {  // eight rows at a time
                        typename Eight<T>::Row got[8];
                        const int64_t first = base + 2 * b * kBatch + 8 * q;
#pragma unroll
                        for (int r = 0; r < 8; ++r)
                            Eight<T>::gather(got[r], w + (first + r) * stride + col0,
                                             first + r < rows ? in_cols : 0, lane);
                        __syncwarp();
#pragma unroll
                        for (int r = 0; r < 8; ++r) Eight<T>::put(got[r], turn[warp][r], lane);
                        __syncwarp();
#pragma unroll
                        for (int r = 0; r < 4; ++r)
                            v[4 * q + r].take(turn[warp][2 * r + odd], run,
                                              w + (first + 2 * r + odd) * stride + col0);
                    }
                }
            }
#pragma unroll
            for (int r = 0; r < kBatch; ++r) {
                const int row = 2 * (b * kBatch + r) + odd;
                // the group's largest magnitude as bits: for non-negative floats the order of
                // the bits is the order of the values, with NaN above infinity
                uint32_t big = 0;
#pragma unroll
                for (int j = 0; j < 8; ++j) big = max(big, __float_as_uint(v[r].get(j)) & 0x7FFFFFFFu);
#pragma unroll
                for (int o = 1; o < GROUP / 8; o *= 2)
                    big = max(big, __shfl_xor_sync(0xFFFFFFFFu, big, o));
                const bool fine = big < 0x7F800000u;
                uint32_t s = __float_as_uint(seventh(__uint_as_float(big))) & 0xFFFF0000u;
                const bool live = fine && s >= 0x00800000u;  // from 2^-126
                if (!live) s = fine ? 0u : 0x7FC00000u;
                const float inv = reciprocal(__uint_as_float(live ? s : 0x3F800000u));
                // column c of the eight belongs in nibble c / 2 + 4 (c % 2)
                uint32_t word = 0, high = 0;
#pragma unroll
                for (int c = 0; c < 8; ++c) {
                    const int at = 4 * ((c >> 1) + 4 * (c & 1));
                    word += __float_as_uint(__fadd_rn(__fmul_rn(v[r].get(c), inv), kRound)) << at;
                    high += 0x4B400000u << at;
                }
                word = live ? word - high : 0x88888888u;
                *reinterpret_cast<uint32_t*>(out + p4_word(row, run)) = word;
                if (run % (GROUP / 8) == 0)
                    scales[p4_scale(row, run / (GROUP / 8), kPer)] = static_cast<uint16_t>(s >> 16);
            }
        }
    }
}

// The value of one of a word's eight columns: a nibble set into 2^23 is
// 2^23 + q + 8, exactly.
__device__ __forceinline__ float value(uint32_t word, int column, float s) {
    uint32_t u;
    asm("lop3.b32 %0, %1, %2, %3, 0xEA;"
        : "=r"(u)
        : "r"(word >> (4 * ((column >> 1) + 4 * (column & 1)))), "r"(0xFu), "r"(0x4B000000u));
    return __fmul_rn(__fsub_rn(__uint_as_float(u), 8388608.0f + 8.0f), s);
}

// One warp takes one tile. Rows are written 16 bytes to a lane, of tiles at the
// right edge without alignment an element (fp32) or an aligned pair of them
// (bf16) to a lane, so that a store is still one run of memory.
template <typename T, int GROUP, bool ALIGNED>
__global__ void __launch_bounds__(kPkThreads, ALIGNED ? 4 : 5)
    unpack4(int64_t rows, int64_t cols, const uint8_t* __restrict__ packed, T* __restrict__ values,
            int64_t stride, int64_t n_tiles, int32_t tiles_across) {
    constexpr int kPer = kP4Cols / GROUP;
    constexpr int kC = 16 / sizeof(T);       // columns of a 16-byte store
    constexpr int kRows = 32 / (128 / kC);   // rows of a warp's store
    const int lane = threadIdx.x & 31;
    const int64_t step = int64_t(gridDim.x) * (kPkThreads / 32);
    for (int64_t tile = int64_t(blockIdx.x) * (kPkThreads / 32) + (threadIdx.x >> 5);
         tile < n_tiles; tile += step) {
        const int64_t row0 = tile / tiles_across * kP4Rows;
        const int64_t col0 = tile % tiles_across * kP4Cols;
        const int in_rows = static_cast<int>(min(int64_t(kP4Rows), rows - row0));
        const int in_cols = static_cast<int>(min(int64_t(kP4Cols), cols - col0));
        const uint8_t* in = packed + tile * p4_tile_bytes(GROUP);
        const uint16_t* scales = reinterpret_cast<const uint16_t*>(in + kP4Quants);
        T* out = values + row0 * stride + col0;
        auto word_of = [&](int r, int col) {
            return __ldg(reinterpret_cast<const uint32_t*>(in + p4_word(r, col >> 3)));
        };
        auto scale_of = [&](int r, int col) {
            return load1(scales + p4_scale(r, col / GROUP, kPer));
        };
        if constexpr (ALIGNED) {
            const int col = kC * (lane % (128 / kC)), sub = lane / (128 / kC);
            uint32_t word[kP4Rows / kRows];
            float s[kP4Rows / kRows];
#pragma unroll
            for (int r = 0; r < kP4Rows / kRows; ++r) {
                word[r] = word_of(kRows * r + sub, col);
                s[r] = scale_of(kRows * r + sub, col);
            }
#pragma unroll
            for (int r = 0; r < kP4Rows / kRows; ++r) {
                const int row = kRows * r + sub;
                if (row >= in_rows) break;
                float v[kC];
#pragma unroll
                for (int j = 0; j < kC; ++j) v[j] = value(word[r], (col & 7) + j, s[r]);
                store16(out + row * stride + col, in_cols - col, v);
            }
        } else if (in_cols == kP4Cols) {
            // Whole rows of 128 columns: a lane has the columns of a 16-byte word and takes what
            // it lacks of an aligned one from the lane before. The first lane's word is the ends
            // of two: `a` columns that are the tile's last and kC - a that are its first.
            constexpr int kLanes = 128 / kC;
            const int run = lane % kLanes, sub = lane / kLanes;
#pragma unroll
            for (int r0 = 0; r0 < kP4Rows; r0 += 8 * kRows) {
                uint32_t word[8];
                float s[8];
#pragma unroll
                for (int r = 0; r < 8; ++r) {
                    word[r] = word_of(r0 + kRows * r + sub, kC * run);
                    s[r] = scale_of(r0 + kRows * r + sub, kC * run);
                }
#pragma unroll
                for (int r = 0; r < 8; ++r) {
                    const int row = r0 + kRows * r + sub;
                    uint4 own;
                    if constexpr (sizeof(T) == 4) {
                        const uint32_t half = (run & 1) ? word[r] >> 8 : word[r];
                        own = make_uint4(__float_as_uint(value(half, 0, s[r])),
                                         __float_as_uint(value(half, 1, s[r])),
                                         __float_as_uint(value(half, 2, s[r])),
                                         __float_as_uint(value(half, 3, s[r])));
                    } else {
                        uint32_t u[4];
#pragma unroll
                        for (int j = 0; j < 4; ++j)
                            u[j] = to_bf16x2(value(word[r], 2 * j, s[r]),
                                             value(word[r], 2 * j + 1, s[r]));
                        own = make_uint4(u[0], u[1], u[2], u[3]);
                    }
                    T* at = out + row * stride;
                    const int a = static_cast<int>(reinterpret_cast<uintptr_t>(at) / sizeof(T) % kC);
                    uint4 before = word_from<kLanes>(own, (run + kLanes - 1) % kLanes);
                    if (a == 0) before = own;
                    const uint4 c = cut(before, own, (16 - static_cast<int>(sizeof(T)) * a) & 15);
                    if (row >= in_rows) continue;
                    T* to = at - a + kC * run;
                    if (run > 0 || a == 0) {
                        __stcs(reinterpret_cast<uint4*>(to), c);
                        continue;
                    }
                    const uint32_t part[4] = {c.x, c.y, c.z, c.w};
                    constexpr int kE = 4 / sizeof(T);  // columns of a part
#pragma unroll
                    for (int k = 0; k < 4; ++k) {
                        if (sizeof(T) == 2 && kE * k + 1 == a) {
                            to[kP4Cols + kE * k] = static_cast<T>(part[k] & 0xFFFFu);
                            to[kE * k + 1] = static_cast<T>(part[k] >> 16);
                        } else {
                            *reinterpret_cast<uint32_t*>(to + kE * k + (kE * k < a ? kP4Cols : 0)) =
                                part[k];
                        }
                    }
                }
            }
        } else if constexpr (sizeof(T) == 4) {
#pragma unroll 4
            for (int r = 0; r < in_rows; ++r) {
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const int col = lane + 32 * i;
                    const float v = value(word_of(r, col), col & 7, scale_of(r, col));
                    if (col < in_cols) out[r * stride + col] = v;
                }
            }
        } else {
#pragma unroll 4
            for (int r = 0; r < in_rows; ++r) {
                T* at = out + r * stride;
                const int odd = static_cast<int>(reinterpret_cast<uintptr_t>(at) >> 1) & 1;
                uint32_t before = 0;  // the last pair of the block before, on every lane
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    const int col = 64 * i + 2 * lane;
                    const uint32_t word = word_of(r, col);
                    const float s = scale_of(r, col);
                    const uint32_t both = to_bf16x2(value(word, col & 7, s), value(word, (col & 7) + 1, s));
                    // columns c, c + 1 of the aligned word that starts with col, or ends with it
                    const uint32_t left = __shfl_up_sync(0xFFFFFFFFu, both, 1);
                    const int c = col - odd;
                    const uint32_t pair =
                        odd ? __funnelshift_r(lane == 0 ? before : left, both, 16) : both;
                    if (c >= 0 && c + 1 < in_cols)
                        *reinterpret_cast<uint32_t*>(at + c) = pair;
                    else if (c >= 0 && c < in_cols)
                        at[c] = static_cast<uint16_t>(pair);
                    else if (c == -1)
                        at[0] = static_cast<uint16_t>(both);
                    before = __shfl_sync(0xFFFFFFFFu, both, 31);
                }
            }
        }
    }
}

// A launch of one warp per tile.
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

template <typename T, bool ALIGNED>
const void* pack_kernel(int32_t group) {
    return group == 32   ? reinterpret_cast<const void*>(pack4<T, 32, ALIGNED>)
           : group == 64 ? reinterpret_cast<const void*>(pack4<T, 64, ALIGNED>)
                         : reinterpret_cast<const void*>(pack4<T, 128, ALIGNED>);
}

template <typename T, bool ALIGNED>
const void* unpack_kernel(int32_t group) {
    return group == 32   ? reinterpret_cast<const void*>(unpack4<T, 32, ALIGNED>)
           : group == 64 ? reinterpret_cast<const void*>(unpack4<T, 64, ALIGNED>)
                         : reinterpret_cast<const void*>(unpack4<T, 128, ALIGNED>);
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
    const bool aligned = cam::row_aligned(w, stride, size, 16);
    bool eight = cam::row_aligned(w, stride, size, 8 * size);
    void* args[] = {&rows, &cols, &w, &stride, &eight, &packed, &tiles, &across};
    const cudaError_t ce = cudaLaunchKernel(
        dtype == CAM_F32
            ? aligned ? cam::pack_kernel<float, true>(group) : cam::pack_kernel<float, false>(group)
        : aligned ? cam::pack_kernel<uint16_t, true>(group)
                  : cam::pack_kernel<uint16_t, false>(group),
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
    const bool aligned = cam::row_aligned(values, stride, size, 16);
    void* args[] = {&rows, &cols, &packed, &values, &stride, &tiles, &across};
    const cudaError_t ce = cudaLaunchKernel(
        dtype == CAM_F32
            ? aligned ? cam::unpack_kernel<float, true>(group) : cam::unpack_kernel<float, false>(group)
        : aligned ? cam::unpack_kernel<uint16_t, true>(group)
                  : cam::unpack_kernel<uint16_t, false>(group),
        dim3(cam::blocks_for(tiles)), dim3(cam::kPkThreads), args, 0,
        static_cast<cudaStream_t>(stream));
    if (ce != cudaSuccess)
        return record_error(CAM_E_CUDA, "%s: launch: %s", fn, cudaGetErrorString(ce));
    return CAM_OK;
}
