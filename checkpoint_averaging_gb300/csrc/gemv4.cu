// gemv4.cu -- cam_gemv4: products of a few rows of x with a matrix in the
// 4-bit form (declaration in include/cam.h, the form in pack4_layout.h).
//
// y[m][n] = sum over groups of s[n][group] * (sum over the group of q[n][k] * x[m][k]).
//
// The weights are 1/2 + 2 / group bytes each and read once, so a few tokens
// are bound by HBM. The sums over a group run on the tensor cores
// (mma.m16n8k16, 16 rows of the matrix x 8 columns of x): q in [-8, 7] is
// exact in bf16 and so is a bf16 x, hence every product is exact and only
// binary32 sums round. An fp32 x is cut into three bf16 terms of 8 bits each,
// x = x1 + x2 + x3 exactly, which take three columns and meet again in the
// output's sum. The group's scale multiplies the group's fp32 sum. The
// weights stay in the lane that loaded them: mma.sync takes them from
// registers, where the 4-bit words are widened (two instructions per two
// weights), while tcgen05 would have them written to shared or tensor memory
// first; at a few columns per weight the tensor cores are far from the bound
// either way.
//
// A block holds x (its share of the columns) in shared memory in the order of
// the operand and walks over units of rows. Its warps split a unit's tiles
// along the columns (and over rows where there are few columns); each streams
// its tiles through a private ring of cp.async slots, ahead across units, so
// the loads never wait for a unit's sums. A cluster of blocks splits the
// columns further where x would not fit or where there are too few rows to
// fill the GPU; sums meet in distributed shared memory, in a fixed order.
#include <cooperative_groups.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <atomic>

#include "cam_internal.h"
#include "op_launch.h"
#include "pack4_layout.h"

#define CAM_API extern "C" __attribute__((visibility("default")))

namespace cam {
namespace {

namespace cg = cooperative_groups;

constexpr int kGvThreads = 256;
constexpr int kGvWarps = kGvThreads / 32;
constexpr int kGvMaxCols = 32;  // columns of x in one pass (four 8-column operands)

struct GemvArgs {
    const void* x;
    const uint8_t* packed;
    void* y;
    int64_t x_stride, y_stride;
    int64_t rows;
    int32_t cols;
    int32_t tokens;       // of the call
    int32_t pass_tokens;  // of one pass (grid.y passes)
    int32_t n_blk;        // 128-column tiles across
    int32_t cta_blk;      // of which a block of the cluster takes so many
    int32_t n_tiles;      // 16-row tiles
    int32_t units;
    int32_t wk;           // warps along the columns; kGvWarps / wk along the rows
    int32_t red_bufs;     // 1 or 2 buffers of partial sums
    int32_t cluster;
    int32_t x_bf16, y_bf16, x_vec;
};

__device__ __forceinline__ void cp16(uint32_t smem, const void* gmem) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" : : "r"(smem), "l"(gmem) : "memory");
}

__device__ __forceinline__ void cp_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }

template <int N>
__device__ __forceinline__ void cp_wait() {
    asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

__device__ __forceinline__ void mma(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                    uint32_t a3, uint32_t b0, uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 "
        "{%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

__device__ __forceinline__ void mma_first(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                          uint32_t a3, uint32_t b0, uint32_t b1) {  // c = a b
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 "
        "{%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%10,%10,%10,%10};"
        : "=f"(c[0]), "=f"(c[1]), "=f"(c[2]), "=f"(c[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(0.0f));
}

// Nibbles p and p + 4 of a word as two bf16: 0x4300 is 128, whose last
// mantissa bit is 1, so 0x4300 | nibble is 128 + nibble, and less 136 it is q.
// (One three-input operation takes the nibbles and sets the rest.)
__device__ __forceinline__ uint32_t widen(uint32_t word, int p) {
    uint32_t u;
    asm("lop3.b32 %0, %1, %2, %3, 0xEA;"
        : "=r"(u)
        : "r"(word >> (4 * p)), "r"(0x000F000Fu), "r"(0x43004300u));
    const __nv_bfloat162 v = __hsub2(*reinterpret_cast<const __nv_bfloat162*>(&u),
                                     __nv_bfloat162(__ushort_as_bfloat16(0x4308),
                                                    __ushort_as_bfloat16(0x4308)));
    return *reinterpret_cast<const uint32_t*>(&v);
}

// The three bf16 terms of an fp32 x: the leading 8 bits of what is left, three
// times. Infinities stand in the first term alone.
__device__ __forceinline__ void terms(float x, uint32_t (&t)[3]) {
    const uint32_t u = __float_as_uint(x);
    if ((u & 0x7F800000u) == 0x7F800000u) {
        t[0] = (u & 0x007FFFFFu) ? 0x7FFFu : u >> 16;
        t[1] = t[2] = 0;
        return;
    }
    t[0] = u >> 16;
    const float r = x - __uint_as_float(u & 0xFFFF0000u);
    t[1] = __float_as_uint(r) >> 16;
    t[2] = __float_as_uint(r - __uint_as_float(__float_as_uint(r) & 0xFFFF0000u)) >> 16;
}

// x's columns of this block and pass into shared memory: 16 bytes (8
// elements) at ((block-local tile * 4 + i) * C + column) * 4 + t, elements
// 32 i + 8 t .. + 7 of the tile. Elements past the end are 0.
template <bool F32>
__device__ __forceinline__ void stage_x(const GemvArgs& a, uint4* xs, int m0, int n_tok, int C,
                                        int blk0, int n_my) {
    const int runs = n_my * 16;
    for (int idx = threadIdx.x; idx < runs * n_tok; idx += kGvThreads) {
        const int m = idx / runs, run = idx - m * runs;  // run = (tile, i, t)
        const int k = blk0 * kP4Cols + run * 8;
        const int left = min(8, a.cols - k);
        const int64_t at = int64_t(m0 + m) * a.x_stride + k;
        uint4* dst = xs + (run >> 2) * C * 4 + (run & 3);
        if constexpr (F32) {
            const float* p = static_cast<const float*>(a.x) + at;
            float v[8];
            if (a.x_vec && left == 8) {
                const float4 lo = __ldg(reinterpret_cast<const float4*>(p));
                const float4 hi = __ldg(reinterpret_cast<const float4*>(p) + 1);
                v[0] = lo.x, v[1] = lo.y, v[2] = lo.z, v[3] = lo.w;
                v[4] = hi.x, v[5] = hi.y, v[6] = hi.z, v[7] = hi.w;
            } else {
#pragma unroll
                for (int j = 0; j < 8; ++j) v[j] = j < left ? __ldg(p + j) : 0.0f;
            }
            uint32_t w[3][4];
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                uint32_t lo[3], hi[3];
                terms(v[2 * j], lo);
                terms(v[2 * j + 1], hi);
#pragma unroll
                for (int q = 0; q < 3; ++q) w[q][j] = lo[q] | (hi[q] << 16);
            }
#pragma unroll
            for (int q = 0; q < 3; ++q)
                dst[(3 * m + q) * 4] = make_uint4(w[q][0], w[q][1], w[q][2], w[q][3]);
        } else {
            const uint16_t* p = static_cast<const uint16_t*>(a.x) + at;
            uint4 v;
            if (a.x_vec && left == 8) {
                v = __ldg(reinterpret_cast<const uint4*>(p));
            } else {
                uint32_t e[8];
#pragma unroll
                for (int j = 0; j < 8; ++j) e[j] = j < left ? __ldg(p + j) : 0u;
                v = make_uint4(e[0] | (e[1] << 16), e[2] | (e[3] << 16), e[4] | (e[5] << 16),
                               e[6] | (e[7] << 16));
            }
            dst[m * 4] = v;
        }
    }
}

__device__ __forceinline__ uint16_t round_bf16(float v) {
    return __bfloat16_as_ushort(__float2bfloat16_rn(v));
}

// Ring slots per warp: enough that every SM has some 64 KB of weights on their way.
__host__ __device__ constexpr int gv_depth(int rt) { return rt == 1 ? 6 : 4; }

template <int RT, int NT, int GROUP>
__global__ void __launch_bounds__(kGvThreads, RT * NT == 1 ? 3 : NT <= 2 ? 2 : 1)
    gemv4(const __grid_constant__ GemvArgs a) {
    constexpr int kTile = p4_tile_bytes(GROUP);
    constexpr int kGvDepth = gv_depth(RT);
    constexpr int kPer = kP4Cols / GROUP;    // scales per row of a tile
    constexpr int kSlot = RT * kTile;
    constexpr int kRedRow = RT * 16 + 4;     // padded: the lanes' rows and columns miss each other's banks
    extern __shared__ __align__(128) uint8_t smem[];

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
    const int rank = a.cluster > 1 ? static_cast<int>(cg::this_cluster().block_rank()) : 0;
    const int n_clusters = gridDim.x / a.cluster, cluster_id = blockIdx.x / a.cluster;
    const int m0 = blockIdx.y * a.pass_tokens;
    const int n_tok = min(a.pass_tokens, a.tokens - m0);
    const int planes = a.x_bf16 ? 1 : 3;
    const int C = n_tok * planes;
    const int blk0 = rank * a.cta_blk;
    const int n_my = max(0, min(a.cta_blk, a.n_blk - blk0));  // this block's tiles across
    const int wr = warp / a.wk, wk = warp - wr * a.wk;
    const int wpr = kGvWarps / a.wk;                          // warps along the rows
    const int unit_tiles = wpr * RT;

    uint8_t* ring = smem + warp * (kGvDepth * kSlot);
    uint4* xs = reinterpret_cast<uint4*>(smem + kGvWarps * kGvDepth * kSlot);
    float* red = reinterpret_cast<float*>(xs + a.cta_blk * 16 * C);
    const int red_floats = kGvWarps * C * kRedRow;

    // this warp's steps: for each unit, its tiles across wk, wk + a.wk, ...
    const int per_unit = n_my > wk ? (n_my - wk + a.wk - 1) / a.wk : 0;
    int l_unit = per_unit > 0 ? cluster_id : a.units, l_b = 0;  // the next step to load
    const uint8_t* l_src[RT];
    uint32_t l_dst = static_cast<uint32_t>(__cvta_generic_to_shared(ring)) + lane * 16;
    const uint32_t ring_end = l_dst + kGvDepth * kSlot;
    const int l_jump = a.wk * kTile;
    auto load = [&]() {
        if (l_unit < a.units) {
            if (l_b == 0) {
#pragma unroll
                for (int r = 0; r < RT; ++r) {
                    const int tile = min(l_unit * unit_tiles + wr * RT + r, a.n_tiles - 1);
                    l_src[r] = a.packed + (int64_t(tile) * a.n_blk + blk0 + wk) * kTile + lane * 16;
                }
            }
#pragma unroll
            for (int r = 0; r < RT; ++r) {
                const uint32_t dst = l_dst + r * kTile;
                cp16(dst, l_src[r]);
                cp16(dst + 512, l_src[r] + 512);
                if (lane < kPer * 2) cp16(dst + 1024, l_src[r] + 1024);
                l_src[r] += l_jump;
            }
            if (++l_b == per_unit) l_b = 0, l_unit += n_clusters;
        }
        cp_commit();
        l_dst += kSlot;
        if (l_dst == ring_end) l_dst -= kGvDepth * kSlot;
    };
#pragma unroll
    for (int s = 0; s < kGvDepth - 1; ++s) load();

    if (a.x_bf16) stage_x<false>(a, xs, m0, n_tok, C, blk0, n_my);
    else stage_x<true>(a, xs, m0, n_tok, C, blk0, n_my);
    __syncthreads();

    // this lane's column of each operand; past the last column any will do, those results are
    // not kept
    int x_lane[NT];
#pragma unroll
    for (int n = 0; n < NT; ++n) x_lane[n] = min(8 * n + g, C - 1) * 4 + t;

    int slot = 0, buf = 0;
    for (int unit = cluster_id; unit < a.units; unit += n_clusters) {
        float acc[RT][NT][4];
#pragma unroll
        for (int r = 0; r < RT; ++r)
#pragma unroll
            for (int n = 0; n < NT; ++n)
#pragma unroll
                for (int j = 0; j < 4; ++j) acc[r][n][j] = 0.0f;

        for (int b = 0; b < per_unit; ++b) {
            cp_wait<kGvDepth - 2>();
            __syncwarp();  // every lane's copies are in, and every lane is done with the slot before
            load();
            const uint8_t* q = ring + slot * kSlot;
            if (++slot == kGvDepth) slot = 0;
            const uint4* xb = xs + (wk + b * a.wk) * 16 * C;
            uint4 w[RT][2];
            uint32_t sc[RT][2][kPer > 1 ? kPer / 2 : 1];  // bf16 pairs (kPer 1: both rows in one)
#pragma unroll
            for (int r = 0; r < RT; ++r) {
#pragma unroll
                for (int h = 0; h < 2; ++h)
                    w[r][h] = *reinterpret_cast<const uint4*>(q + r * kTile + h * 512 + lane * 16);
                const uint8_t* s = q + r * kTile + 1024 + g * (4 * kPer);
                if constexpr (kPer == 4) {
                    const uint4 v = *reinterpret_cast<const uint4*>(s);
                    sc[r][0][0] = v.x, sc[r][0][1] = v.y, sc[r][1][0] = v.z, sc[r][1][1] = v.w;
                } else if constexpr (kPer == 2) {
                    const uint2 v = *reinterpret_cast<const uint2*>(s);
                    sc[r][0][0] = v.x, sc[r][1][0] = v.y;
                } else {
                    sc[r][0][0] = *reinterpret_cast<const uint32_t*>(s);
                    sc[r][1][0] = sc[r][0][0] >> 16;
                }
            }
            float part[RT][NT][4];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                constexpr int kSteps = GROUP / 32;  // steps of 32 columns per group
                uint4 x[NT];
#pragma unroll
                for (int n = 0; n < NT; ++n) x[n] = xb[i * C * 4 + x_lane[n]];
#pragma unroll
                for (int r = 0; r < RT; ++r) {
                    const uint32_t lo = i == 0 ? w[r][0].x : i == 1 ? w[r][0].y : i == 2 ? w[r][0].z : w[r][0].w;
                    const uint32_t hi = i == 0 ? w[r][1].x : i == 1 ? w[r][1].y : i == 2 ? w[r][1].z : w[r][1].w;
                    uint32_t al[4], ah[4];
#pragma unroll
                    for (int p = 0; p < 4; ++p) al[p] = widen(lo, p), ah[p] = widen(hi, p);
#pragma unroll
                    for (int n = 0; n < NT; ++n) {
                        if (i % kSteps == 0)
                            mma_first(part[r][n], al[0], ah[0], al[1], ah[1], x[n].x, x[n].y);
                        else
                            mma(part[r][n], al[0], ah[0], al[1], ah[1], x[n].x, x[n].y);
                        mma(part[r][n], al[2], ah[2], al[3], ah[3], x[n].z, x[n].w);
                    }
                    if (i % kSteps == kSteps - 1) {
                        const int j = i / kSteps;
                        const float s0 = __uint_as_float((j & 1) ? sc[r][0][j >> 1] & 0xFFFF0000u
                                                                 : sc[r][0][j >> 1] << 16);
                        const float s1 = __uint_as_float((j & 1) ? sc[r][1][j >> 1] & 0xFFFF0000u
                                                                 : sc[r][1][j >> 1] << 16);
#pragma unroll
                        for (int n = 0; n < NT; ++n) {
                            acc[r][n][0] = fmaf(s0, part[r][n][0], acc[r][n][0]);
                            acc[r][n][1] = fmaf(s0, part[r][n][1], acc[r][n][1]);
                            acc[r][n][2] = fmaf(s1, part[r][n][2], acc[r][n][2]);
                            acc[r][n][3] = fmaf(s1, part[r][n][3], acc[r][n][3]);
                        }
                    }
                }
            }
        }

        // the warps' (and blocks') sums meet: [warp][column][row]
        float* mine = red + buf * red_floats + warp * C * kRedRow;
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const int c = 8 * n + 2 * t + (j & 1);
                if (c < C) {
#pragma unroll
                    for (int r = 0; r < RT; ++r)
                        mine[c * kRedRow + 16 * r + 8 * (j >> 1) + g] = acc[r][n][j];
                }
            }
        if (a.cluster > 1) cg::this_cluster().sync();
        else __syncthreads();
        const int unit_rows = unit_tiles * 16;
        const int64_t row0 = int64_t(unit) * unit_rows;
        for (int o = threadIdx.x + kGvThreads * rank; o < unit_rows * n_tok;
             o += kGvThreads * a.cluster) {
            const int m = o / unit_rows, row = o - m * unit_rows;
            const int rw = row / (RT * 16), in = row - rw * (RT * 16);
            if (row0 + row >= a.rows) continue;
            float sum = 0.0f;
            for (int p = planes - 1; p >= 0; --p) {
                const float* at = red + buf * red_floats +
                                  (rw * a.wk * C + m * planes + p) * kRedRow + in;
                for (int c = 0; c < a.cluster; ++c) {
                    const float* from = a.cluster > 1 ? cg::this_cluster().map_shared_rank(at, c) : at;
                    for (int k = 0; k < a.wk; ++k) sum += from[k * C * kRedRow];
                }
            }
            const int64_t to = int64_t(m0 + m) * a.y_stride + row0 + row;
            if (a.y_bf16) static_cast<uint16_t*>(a.y)[to] = round_bf16(sum);
            else static_cast<float*>(a.y)[to] = sum;
        }
        if (a.red_bufs == 2) {
            buf ^= 1;
        } else {
            if (a.cluster > 1) cg::this_cluster().sync();
            else __syncthreads();
        }
    }
    cp_wait<0>();
    if (a.cluster > 1) cg::this_cluster().sync();  // no block leaves while another reads its sums
}

template <int RT, int NT>
const void* kernel_for_group(int group) {
    return group == 32   ? reinterpret_cast<const void*>(gemv4<RT, NT, 32>)
           : group == 64 ? reinterpret_cast<const void*>(gemv4<RT, NT, 64>)
                         : reinterpret_cast<const void*>(gemv4<RT, NT, 128>);
}

const void* kernel_for(int rt, int nt, int group) {
    if (rt == 1)
        return nt == 1   ? kernel_for_group<1, 1>(group)
               : nt == 2 ? kernel_for_group<1, 2>(group)
                         : kernel_for_group<1, 4>(group);
    return nt == 1   ? kernel_for_group<2, 1>(group)
           : nt == 2 ? kernel_for_group<2, 2>(group)
                     : kernel_for_group<2, 4>(group);
}

}  // namespace
}  // namespace cam

using cam::record_error;

CAM_API int cam_gemv4(int64_t tokens, int64_t rows, int64_t cols, const void* x, int64_t x_stride,
                      cam_dtype x_dtype, const void* packed, int32_t group, void* y,
                      int64_t y_stride, cam_dtype y_dtype, void* stream) {
    using namespace cam;
    const char* fn = "cam_gemv4";
    if (const int rc = p4_check(fn, rows, cols, group)) return rc;
    if (rows > (int64_t(1) << 31)) return record_error(CAM_E_ARG, "%s: rows out of range", fn);
    if (tokens < 0 || tokens > (int64_t(1) << 18))
        return record_error(CAM_E_ARG, "%s: tokens out of range", fn);
    for (const cam_dtype d : {x_dtype, y_dtype})
        if (d != CAM_F32 && d != CAM_BF16)
            return record_error(CAM_E_ARG, "%s: unknown dtype %d", fn, static_cast<int>(d));
    if (tokens == 0 || rows == 0) return CAM_OK;
    if (!y || (cols > 0 && (!x || !packed)))
        return record_error(CAM_E_ARG, "%s: a pointer is NULL", fn);
    if (x_stride < cols || x_stride > (int64_t(1) << 40) || y_stride < rows ||
        y_stride > (int64_t(1) << 40))
        return record_error(CAM_E_ARG, "%s: stride out of range", fn);
    if (reinterpret_cast<uintptr_t>(packed) % 16 != 0)
        return record_error(CAM_E_ARG, "%s: packed is not 16-byte aligned", fn);
    const int x_size = x_dtype == CAM_F32 ? 4 : 2, y_size = y_dtype == CAM_F32 ? 4 : 2;
    if (reinterpret_cast<uintptr_t>(x) % x_size != 0 || reinterpret_cast<uintptr_t>(y) % y_size != 0)
        return record_error(CAM_E_ARG, "%s: an array is not aligned to its elements", fn);
    int dev = 0, sms = 0;
    cudaError_t ce = current_device(&dev, &sms);
    if (ce != cudaSuccess)
        return record_error(CAM_E_CUDA, "%s: no usable CUDA device: %s", fn, cudaGetErrorString(ce));
    cudaStream_t s = static_cast<cudaStream_t>(stream);

    GemvArgs a{};
    a.x = x;
    a.packed = static_cast<const uint8_t*>(packed);
    a.y = y;
    a.x_stride = x_stride;
    a.y_stride = y_stride;
    a.rows = rows;
    a.cols = static_cast<int32_t>(cols);
    a.tokens = static_cast<int32_t>(tokens);
    a.n_blk = static_cast<int32_t>((cols + kP4Cols - 1) / kP4Cols);
    a.n_tiles = static_cast<int32_t>((rows + kP4Rows - 1) / kP4Rows);
    a.x_bf16 = x_dtype == CAM_BF16;
    a.y_bf16 = y_dtype == CAM_BF16;
    a.x_vec = reinterpret_cast<uintptr_t>(x) % 16 == 0 && x_stride * x_size % 16 == 0;
    // tokens in as few passes over the weights as their columns allow, evenly; fewer at a time
    // where the longest rows of x would not fit even a cluster
    const int planes = a.x_bf16 ? 1 : 3;
    int most = kGvMaxCols / planes;
    int passes, C, nt, red, rt, ring;
    for (;; most /= 2) {
        if (most == 0) return record_error(CAM_E_ARG, "%s: cols too large", fn);
        passes = (a.tokens + most - 1) / most;
        a.pass_tokens = (a.tokens + passes - 1) / passes;
        passes = (a.tokens + a.pass_tokens - 1) / a.pass_tokens;
        C = a.pass_tokens * planes;
        nt = C <= 8 ? 1 : C <= 16 ? 2 : 4;
        // two row tiles per step where x's operand is wide and rows are enough: it is read once
        // for both
        rt = nt > 1 && a.n_tiles >= 4 * sms ? 2 : 1;
        ring = kGvWarps * gv_depth(rt) * rt * p4_tile_bytes(group);
        a.red_bufs = C <= 8 ? 2 : 1;
        red = a.red_bufs * kGvWarps * C * (rt * 16 + 4) * 4;
        const int x_room = kMaxSharedBytes - ring - red;
        // the columns split over a cluster until x fits, and further while blocks are fewer
        // than SMs
        a.cluster = 1;
        while (a.cluster < 8 &&
               (int64_t((a.n_blk + a.cluster - 1) / a.cluster) * 256 * C > x_room ||
                (int64_t(a.n_tiles) * passes * 2 * a.cluster <= sms && a.n_blk >= 16 * a.cluster)))
            a.cluster *= 2;
        a.cta_blk = (a.n_blk + a.cluster - 1) / a.cluster;
        if (int64_t(a.cta_blk) * 256 * C <= x_room) break;
    }
    if (passes > 65535) return record_error(CAM_E_ARG, "%s: too many tokens", fn);
    const int bytes = ring + red + a.cta_blk * 256 * C;
    const int room = 228 * 1024 / (bytes + 1024);
    const int per_sm = std::min(room, rt * nt == 1 ? 3 : nt <= 2 ? 2 : 1);
    const int slots = std::max(1, sms * per_sm / a.cluster / passes);
    // Warps along the columns: more of them even the work out over the blocks, fewer meet less
    // often. In units of one step, a meeting costs about two.
    int64_t best = INT64_MAX;
    for (int wk = 1; wk <= kGvWarps && (wk == 1 || wk <= a.cta_blk); wk *= 2) {
        const int unit_tiles = kGvWarps / wk * rt;
        const int units = (a.n_tiles + unit_tiles - 1) / unit_tiles;
        const int64_t cost =
            int64_t((units + slots - 1) / slots) * ((a.cta_blk + wk - 1) / wk + 2);
        if (cost < best) best = cost, a.wk = wk, a.units = units;
    }
    const int clusters = std::min(a.units, slots);

    const void* kern = kernel_for(rt, nt, group);
    if (bytes > 48 * 1024) {
        static std::atomic<uint64_t> shared_ok[2][3][3];
        ce = allow_shared(kern, dev,
                          shared_ok[rt - 1][nt == 4 ? 2 : nt - 1][group == 32 ? 0 : group / 64]);
    }
    if (ce == cudaSuccess) {
        cudaLaunchConfig_t cfg{};
        cfg.gridDim = dim3(clusters * a.cluster, passes);
        cfg.blockDim = dim3(kGvThreads);
        cfg.dynamicSmemBytes = bytes;
        cfg.stream = s;
        cudaLaunchAttribute attr{};
        attr.id = cudaLaunchAttributeClusterDimension;
        attr.val.clusterDim.x = a.cluster;
        attr.val.clusterDim.y = attr.val.clusterDim.z = 1;
        cfg.attrs = &attr;
        cfg.numAttrs = a.cluster > 1 ? 1 : 0;
        void* args[] = {&a};
        ce = cudaLaunchKernelExC(&cfg, kern, args);
    }
    if (ce != cudaSuccess)
        return record_error(CAM_E_CUDA, "%s: launch: %s", fn, cudaGetErrorString(ce));
    return CAM_OK;
}
