// head.cu -- log probabilities of a head's tokens from hidden states, without the logits
// (cam_head_logprobs), and the gradients of the hidden states and of the head
// (cam_head_logprobs_backward).
//
// Forward: one product of hidden [R x D] and head [V x D] on the tensor cores
// (tile_products.cu), whose epilogue reduces each tile of logits to a few numbers per row;
// stats_kernel joins them. 2 R V D operations bound it, or reading the head for few rows.
//
// Backward, by pieces of the vocabulary: the logits again, with
//
//     G_j = g (1[j = token] - p_j) - h p_j (log p_j + H)
//
// as their tiles' epilogue, kept in bf16 terms for one piece; then, in one launch,
// d head = G^T hidden of the piece and the piece's share of d hidden = G head (fp32
// partials, joined in a fixed order by join_kernel). 6 R V D operations.
//
// fp32 matrices are taken as three bf16 terms each (24 bits: the whole significand) and
// the six largest of the nine products of terms; what is left out is 2^-23 of
// |hidden| |head| at most, where fp32 products round by 2^-24 each. bf16 matrices are one
// term; their G is one bf16 term, too (2^-8 of each G_j at most: the bf16 gradients that hold
// sums of them round by as much again), or two for few rows.
#include <cuda_bf16.h>

#include <algorithm>
#include <cmath>
#include <cstdint>
#include <utility>

#include "cam_internal.h"
#include "op_launch.h"
#include "tile_device.cuh"
#include "tile_products.h"

#define CAM_API extern "C" __attribute__((visibility("default")))

namespace cam {
namespace {

using tc::term;

constexpr int kHeadThreads = 256;

// ---- terms ------------------------------------------------------------------------------

struct TermMatrix {
    const void* src;
    int64_t stride, rows, cols;
    __nv_bfloat16* out;  // [planes][rows][ld]
    int64_t ld, plane_stride;
    bool masked;  // rows without a gradient are taken as zeros
};

struct TermArgs {
    TermMatrix m[2];
    int64_t first;  // threads of the first matrix (a multiple of a block's)
    int64_t all;
    const int64_t* tokens;
    const float *g, *h;
};

// One or two matrices in one (bf16) or three (fp32) bf16 terms, eight columns per thread.
template <typename T>
__global__ void __launch_bounds__(kHeadThreads) terms_kernel(const TermArgs a) {
    asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    constexpr int kTerms = sizeof(T) == 4 ? 3 : 1;
    for (int64_t k = int64_t(blockIdx.x) * kHeadThreads + threadIdx.x; k < a.all;
         k += int64_t(gridDim.x) * kHeadThreads) {
        const bool second = k >= a.first;
        const TermMatrix& m = a.m[second];
        const int64_t i = second ? k - a.first : k, across = (m.cols + 7) / 8;
        const int64_t row = a.all >> 31 ? i / across
                                        : static_cast<int64_t>(static_cast<uint32_t>(i) /
                                                               static_cast<uint32_t>(across));
        const int64_t col = (i - row * across) * 8;
        if (row >= m.rows) continue;
        const T* src = static_cast<const T*>(m.src);
        const bool vec = reinterpret_cast<uintptr_t>(src) % 16 == 0 && m.stride * sizeof(T) % 16 == 0;
        bool keep = true;
        if (m.masked)
            keep = (a.g && a.tokens[row] >= 0 && a.g[row] != 0.0f) || (a.h && a.h[row] != 0.0f);
        float v[8];
        const T* at = src + row * m.stride + col;
        if (keep && vec && col + 8 <= m.cols) {
            if constexpr (sizeof(T) == 4) {
                const float4 x = reinterpret_cast<const float4*>(at)[0];
                const float4 y = reinterpret_cast<const float4*>(at)[1];
                v[0] = x.x, v[1] = x.y, v[2] = x.z, v[3] = x.w;
                v[4] = y.x, v[5] = y.y, v[6] = y.z, v[7] = y.w;
            } else {
                const uint4 x = *reinterpret_cast<const uint4*>(at);
                const uint32_t w[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    v[2 * j] = __uint_as_float(w[j] << 16);
                    v[2 * j + 1] = __uint_as_float(w[j] & 0xFFFF0000u);
                }
            }
        } else {
#pragma unroll
            for (int j = 0; j < 8; ++j)
                v[j] = keep && col + j < m.cols ? static_cast<float>(at[j]) : 0.0f;
        }
#pragma unroll
        for (int t = 0; t < kTerms; ++t) {
            uint32_t w[4];
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const __nv_bfloat16 lo = term(v[2 * j]), hi = term(v[2 * j + 1]);
                w[j] = __bfloat16_as_ushort(lo) | (uint32_t(__bfloat16_as_ushort(hi)) << 16);
                v[2 * j] -= __bfloat162float(lo);
                v[2 * j + 1] -= __bfloat162float(hi);
            }
            *reinterpret_cast<uint4*>(m.out + t * m.plane_stride + row * m.ld + col) =
                make_uint4(w[0], w[1], w[2], w[3]);
        }
    }
}

// ---- joining ----------------------------------------------------------------------------

struct StatArgs {
    const TileStat* stats;  // [parts][rows]
    int64_t parts, rows, vocab;
    const float* mine;
    const int64_t* tokens;
    float *logp, *entropy, *lse, *lse_lo;
};

__device__ __forceinline__ void join_lanes(TileStat& s, int by) {
    TileStat o;
    o.m = __shfl_xor_sync(0xFFFFFFFFu, s.m, by);
    o.a = __shfl_xor_sync(0xFFFFFFFFu, s.a, by);
    o.t = __shfl_xor_sync(0xFFFFFFFFu, s.t, by);
    o.any = __shfl_xor_sync(0xFFFFFFFFu, s.any, by);
    join(s, o);
}

// ROWS rows per block (eight: a part's statistics of theirs are one line of 128 bytes; one
// where there are few rows, so that their parts are read by many threads), 256 / ROWS
// threads each, sixteen parts in flight per thread.
template <int ROWS>
__global__ void __launch_bounds__(kHeadThreads) stats_kernel(const StatArgs a) {
    asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    constexpr int kAcross = kHeadThreads / ROWS, kAtOnce = 16;
    __shared__ TileStat all[kHeadThreads / 32][ROWS];
    const int r = threadIdx.x % ROWS, y = threadIdx.x / ROWS;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int64_t row = int64_t(blockIdx.x) * ROWS + r;
    TileStat s{0.0f, 0.0f, 0.0f, 0.0f};
    if (row < a.rows) {
        for (int64_t p0 = y; p0 < a.parts; p0 += kAcross * kAtOnce) {
            float4 v[kAtOnce];
#pragma unroll
            for (int k = 0; k < kAtOnce; ++k) {
                const int64_t p = p0 + k * kAcross;
                v[k] = p < a.parts
                           ? *reinterpret_cast<const float4*>(a.stats + p * a.rows + row)
                           : make_float4(0.0f, 0.0f, 0.0f, 0.0f);
            }
#pragma unroll
            for (int k = 0; k < kAtOnce; ++k) join(s, TileStat{v[k].x, v[k].y, v[k].z, v[k].w});
        }
    }
#pragma unroll
    for (int by = ROWS; by < 32; by *= 2) join_lanes(s, by);
    if (lane < ROWS) all[warp][lane] = s;
    __syncthreads();
    if (warp > 0) return;
    // the eight warps' parts: lane ROWS k + r holds warp k's of row r, two for eight rows
    constexpr int kWarps = kHeadThreads / 32, kHeld = 32 / ROWS < kWarps ? 32 / ROWS : kWarps;
    const int k0 = lane / ROWS;
    s = TileStat{0.0f, 0.0f, 0.0f, 0.0f};
    if (k0 < kHeld)
        for (int k = k0; k < kWarps; k += kHeld) join(s, all[k][r]);
#pragma unroll
    for (int by = ROWS; by < 32 && by < ROWS * kHeld; by *= 2) join_lanes(s, by);
    if (lane >= ROWS || row >= a.rows) return;
    const double sum = 1.0 + double(s.a);
    const double log_s = log1p(double(s.a));
    const bool broken = isnan(s.t);
    const float nan = __int_as_float(0x7FC00000);
    const float top = static_cast<float>(double(s.m) + log_s);
    if (a.lse) a.lse[row] = broken ? nan : top;
    if (a.lse_lo)
        a.lse_lo[row] = broken ? nan : static_cast<float>((double(s.m) - double(top)) + log_s);
    if (a.entropy) a.entropy[row] = broken ? nan : static_cast<float>(log_s - double(s.t) / sum);
    if (a.logp) {
        const int64_t token = a.tokens[row];
        float v = 0.0f;
        if (token >= 0)
            v = broken || token >= a.vocab
                    ? nan
                    : static_cast<float>((double(a.mine[row]) - double(s.m)) - log_s);
        a.logp[row] = v;
    }
}

struct JoinArgs {
    const float* part;  // [splits][rows][ld]
    int64_t rows, cols, ld;
    int32_t splits;
    void* out;
    int64_t stride;
};

// Sums of partials in the order of their ranges: a block of 32 x RUNS threads takes 128
// columns of 8 / RUNS rows, RUNS threads the ranges of one column in as many runs (one for few
// ranges, eight where there are many and few columns).
template <typename T, int RUNS>
__global__ void __launch_bounds__(kHeadThreads) join_kernel(const JoinArgs a) {
    asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    constexpr int kRowsEach = 8 / RUNS;
    __shared__ float4 runs[8][32];
    const int x = threadIdx.x & 31, warp = threadIdx.x >> 5, run = warp % RUNS;
    const int64_t across = (a.ld + 127) / 128, groups = (a.rows + kRowsEach - 1) / kRowsEach;
    const int32_t per = (a.splits + RUNS - 1) / RUNS, s0 = run * per, s1 = min(a.splits, s0 + per);
    for (int64_t t = blockIdx.x; t < across * groups; t += gridDim.x) {
        const int64_t group = t / across, col = (t - group * across) * 128 + 4 * x;
        const int64_t row = group * kRowsEach + warp / RUNS;
        const bool in = row < a.rows && col < a.ld;  // (ld is a multiple of eight)
        float4 sum = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
        if (in) {
            const float* p = a.part + row * a.ld + col;
#pragma unroll 8
            for (int32_t s = s0; s < s1; ++s) {
                const float4 v = *reinterpret_cast<const float4*>(p + int64_t(s) * a.rows * a.ld);
                sum.x += v.x, sum.y += v.y, sum.z += v.z, sum.w += v.w;
            }
        }
        if constexpr (RUNS > 1) {
            runs[warp][x] = sum;
            __syncthreads();
            if (run == 0) {
#pragma unroll
                for (int k = 1; k < RUNS; ++k) {
                    const float4 v = runs[warp + k][x];
                    sum.x += v.x, sum.y += v.y, sum.z += v.z, sum.w += v.w;
                }
            }
            __syncthreads();
        }
        if (in && run == 0) {
            T* out = static_cast<T*>(a.out) + row * a.stride + col;
            const float v[4] = {sum.x, sum.y, sum.z, sum.w};
            if (col + 4 <= a.cols && reinterpret_cast<uintptr_t>(out) % (4 * sizeof(T)) == 0) {
                if constexpr (sizeof(T) == 4) {
                    *reinterpret_cast<float4*>(out) = sum;
                } else {
                    const __nv_bfloat162 lo = __floats2bfloat162_rn(v[0], v[1]);
                    const __nv_bfloat162 hi = __floats2bfloat162_rn(v[2], v[3]);
                    *reinterpret_cast<uint2*>(out) = make_uint2(*reinterpret_cast<const uint32_t*>(&lo),
                                                                *reinterpret_cast<const uint32_t*>(&hi));
                }
            } else {
#pragma unroll
                for (int k = 0; k < 4; ++k)
                    if (col + k < a.cols) out[k] = T(v[k]);
            }
        }
    }
}

// Partials part[range][column][row] of few rows' sums, joined in the order of their ranges and
// turned: a block takes four columns of 32 rows, its warps the ranges in eight runs.
__global__ void __launch_bounds__(kHeadThreads) join_turned(const JoinArgs a) {
    asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    __shared__ float runs[8][4][32];
    const int x = threadIdx.x & 31, y = threadIdx.x >> 5;
    const int64_t across = (a.cols + 3) / 4;
    const int64_t row = blockIdx.x / across * 32 + x, col0 = blockIdx.x % across * 4;
    const int32_t per = (a.splits + 7) / 8, s0 = y * per, s1 = min(a.splits, s0 + per);
    float sum[4] = {0.0f, 0.0f, 0.0f, 0.0f};
    if (row < a.rows) {
#pragma unroll 4
        for (int32_t s = s0; s < s1; ++s)
#pragma unroll
            for (int k = 0; k < 4; ++k)
                if (col0 + k < a.cols) sum[k] += a.part[(s * a.cols + col0 + k) * a.ld + row];
    }
#pragma unroll
    for (int k = 0; k < 4; ++k) runs[y][k][x] = sum[k];
    __syncthreads();
    if (y < 4 && row < a.rows && col0 + y < a.cols) {
        float all = 0.0f;
#pragma unroll
        for (int k = 0; k < 8; ++k) all += runs[k][y][x];
        static_cast<float*>(a.out)[row * a.stride + col0 + y] = all;
    }
}

// ---- host side --------------------------------------------------------------------------

template <typename A>
cudaError_t launch(void (*kernel)(A), int64_t blocks, const A& a, cudaStream_t s) {
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3(static_cast<unsigned>(std::max<int64_t>(1, blocks)));
    cfg.blockDim = dim3(kHeadThreads);
    cfg.stream = s;
    cudaLaunchAttribute at{};
    at.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at.val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = &at;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kernel, a);
}

struct Matrix {
    const void* base;
    int64_t rows, stride;
};

struct HeadCall {
    int64_t rows, vocab, width;
    Matrix hidden, head;
    cam_dtype dtype;
    int terms;       // 1 (bf16) or 3
    int grad_terms;  // of G
    int64_t ld;      // of a matrix in terms
    bool x_direct, w_direct;  // read where they are
    bool pair;
    bool few;        // few rows of logits: as columns, the vocabulary along the tiles' rows
    bool few32;      // and in fp32: the head's terms made on the way (f32_products.cu)
};

int64_t padded(int64_t bytes) { return (bytes + 511) / 512 * 512; }

int check_head(const char* fn, HeadCall& c) {
    if (c.rows < 0 || c.rows > (int64_t(1) << 24))
        return record_error(CAM_E_ARG, "%s: rows out of range", fn);
    if (c.vocab < 1 || c.vocab > CAM_LOGPROBS_MAX_VOCAB)
        return record_error(CAM_E_ARG, "%s: vocab out of range", fn);
    if (c.width < 1 || c.width > CAM_HEAD_MAX_WIDTH)
        return record_error(CAM_E_ARG, "%s: width out of range", fn);
    // (tiles are counted in 32 bits)
    if ((c.rows + 127) / 128 * ((c.vocab + kTileCols - 1) / kTileCols) > (int64_t(1) << 30))
        return record_error(CAM_E_ARG, "%s: rows and vocab out of range", fn);
    if (c.dtype != CAM_F32 && c.dtype != CAM_BF16)
        return record_error(CAM_E_ARG, "%s: unknown dtype %d", fn, static_cast<int>(c.dtype));
    const int64_t size = c.dtype == CAM_F32 ? 4 : 2;
    if (c.rows > 0) {
        for (const Matrix& m : {c.hidden, c.head}) {
            if (!m.base) return record_error(CAM_E_ARG, "%s: a pointer is NULL", fn);
            if (m.stride < c.width || m.stride > (int64_t(1) << 34))
                return record_error(CAM_E_ARG, "%s: stride out of range", fn);
            if (reinterpret_cast<uintptr_t>(m.base) % size != 0)
                return record_error(CAM_E_ARG, "%s: an array is not aligned to its elements", fn);
        }
    }
    c.terms = c.dtype == CAM_F32 ? 3 : 1;
    // (rows of whole 128-byte lines: a box of 128 bytes of each row is then one line of it)
    c.ld = (c.width + 63) / 64 * 64;
    // (the tensor maps want rows that start on 16 bytes)
    auto direct = [&](const Matrix& m) {
        return c.dtype == CAM_BF16 && reinterpret_cast<uintptr_t>(m.base) % 16 == 0 && m.stride % 8 == 0;
    };
    c.x_direct = direct(c.hidden);
    c.w_direct = direct(c.head);
    // G of bf16 inputs: one term, whose rounding adds in squares to that of the results (0.0024
    // of their norm off 64 bits where 0.0017 is their own), over many rows; the large entries of a
    // few rows may round alike (0.0031 for 16), and a second term costs little there.
    c.grad_terms = c.terms == 3 ? 3 : c.rows > 256 ? 1 : 2;
    // a pair of SMs takes 256 rows, one SM 128
    c.pair = c.rows > 128;
    // (16 rows of 73,760 logits: a tile of 128 rows of logits has work for one warp in eight)
    // Terms on the way save writing the head's and reading them back, but a block takes 128 rows of
    // the head, whose copies it waits for: where the head is small, or narrow for so many rows,
    // its terms are written out. (Log probabilities and gradients, on the way / written out:
    // 100 rows over 4,000 x 200 33 / 33 and 52 / 38 us, over 12,000 x 1,500 63 / 92 and 160 / 178,
    // over 150,000 x 72 142 / 74 and 270 / 189; 30 over 150,000 x 72 65 / 89 and 155 / 180.)
    c.few32 = c.terms == 3 && c.rows <= kFew32 && c.vocab * c.width >= (int64_t(1) << 23) &&
              (c.rows <= kTileFew || c.width > 512);
    c.few = c.rows <= kTileFew || c.few32;
    if (c.few32) c.w_direct = true;
    return CAM_OK;
}

// Bytes of a matrix in terms.
int64_t term_bytes(const HeadCall& c, int64_t rows) { return padded(c.terms * rows * c.ld * 2); }

TileOperand operand(const HeadCall& c, const Matrix& m, int64_t rows, bool direct, const void* terms,
                    bool mn) {
    TileOperand o{};
    o.base = direct ? m.base : terms;
    o.ld = direct ? m.stride : c.ld;
    o.planes = direct ? 1 : c.terms;
    o.plane_stride = rows * o.ld;
    o.mn_major = mn;
    o.rows = mn ? c.width : rows;
    o.k = mn ? rows : c.width;
    return o;
}

// Queues the terms of up to two matrices (rows 0: none).
cudaError_t make_terms(const HeadCall& c, const Matrix& m0, int64_t rows0, void* out0, bool masked,
                       const Matrix& m1, int64_t rows1, void* out1, const int64_t* tokens,
                       const float* g, const float* h, int sms, cudaStream_t s) {
    const int64_t across = (c.width + 7) / 8;
    TermArgs a{};
    a.m[0] = {m0.base, m0.stride, rows0, c.width, static_cast<__nv_bfloat16*>(out0), c.ld, rows0 * c.ld,
              masked};
    a.m[1] = {m1.base, m1.stride, rows1, c.width, static_cast<__nv_bfloat16*>(out1), c.ld, rows1 * c.ld,
              false};
    a.first = (rows0 * across + kHeadThreads - 1) / kHeadThreads * kHeadThreads;
    a.all = a.first + rows1 * across;
    a.tokens = tokens;
    a.g = g;
    a.h = h;
    if (a.all == 0) return cudaSuccess;
    const int64_t blocks =
        std::min<int64_t>((a.all + kHeadThreads - 1) / kHeadThreads, int64_t(sms) * 32);
    return c.dtype == CAM_F32 ? launch(terms_kernel<float>, blocks, a, s)
                              : launch(terms_kernel<__nv_bfloat16>, blocks, a, s);
}

// The product of `t` (the few rows as t.b) with a piece of an fp32 head.
Few32Product head32(const HeadCall& c, const Matrix& piece, int64_t n, const TileProduct& t) {
    Few32Product q{};
    q.w = static_cast<const float*>(piece.base);
    q.w_rows = n;
    q.width = c.width;
    q.w_stride = piece.stride;
    q.b = t.b;
    q.splits = 1;
    q.out = t.out;
    return q;
}

Matrix piece_of(const HeadCall& c, int64_t at) {
    const int64_t size = c.dtype == CAM_F32 ? 4 : 2;
    return Matrix{static_cast<const char*>(c.head.base) + at * c.head.stride * size, c.vocab - at,
                  c.head.stride};
}

// Equal pieces of the vocabulary, whole tiles of columns, within `budget` bytes of `per` each.
int64_t piece_rows(const HeadCall& c, int64_t per, int64_t budget) {
    if (per == 0) return c.vocab;
    const int64_t most = std::max<int64_t>(kTileCols, budget / per / kTileCols * kTileCols);
    const int64_t n = (c.vocab + most - 1) / most;
    return ((c.vocab + n - 1) / n + kTileCols - 1) / kTileCols * kTileCols;
}

// A piece of the head in terms; a piece of G, and of the head in terms. Each piece is launches of
// its own, whose last rounds of tiles are short, and a reading of the hidden states: what smaller
// ones keep in L2 is less than that. 2^25, 2^27, 2^28, 2^29 and 2^31 bytes: log probabilities of 300
// fp32 rows over 400,000 x 1,024 3,068, 2,281, 2,056, 1,919 and 1,830 us; gradients of 1,023 fp32 rows
// over 50,304 x 128 452, 329, 325, 280 and 281, of 842 over 10,385 x 2,997 1,503, 831, 750, 751 and 751,
// of 4,096 bf16 rows over 73,760 x 2,048 2.60, 2.12, 2.05, 2.10 and 2.08 ms.
constexpr int64_t kForwardBudget = int64_t(1) << 29;
constexpr int64_t kBackwardBudget = int64_t(1) << 29;

// Parts of the vocabulary with statistics of their own.
int64_t stat_parts(const HeadCall& c) {
    return c.few ? (c.vocab + 31) / 32 : (c.vocab + kTileCols - 1) / kTileCols;
}

struct ForwardPlan {
    int64_t piece, x, w, stats, mine, bytes;  // offsets in the workspace
};

ForwardPlan forward_plan(const HeadCall& c) {
    ForwardPlan p{};
    p.piece = std::min(c.vocab, piece_rows(c, c.w_direct ? 0 : c.terms * c.ld * 2, kForwardBudget));
    int64_t at = 0;
    p.x = at;
    if (!c.x_direct) at += term_bytes(c, c.rows);
    p.w = at;
    if (!c.w_direct) at += term_bytes(c, p.piece);
    p.stats = at;
    at += padded(stat_parts(c) * c.rows * int64_t(sizeof(TileStat)));
    p.mine = at;
    at += padded(c.rows * 4);
    p.bytes = at;
    return p;
}

struct BackwardPlan {
    int64_t piece, x, w, grad, hidden, head, bytes;
    int32_t hidden_splits, head_splits;
    int32_t hidden_ranges;  // few32: of the largest piece
    int64_t part_ld, grad_ld, grad_stride;
};

// Ranges of K for a product of `tiles` tiles of `steps` steps of K, `pairs` products of terms
// each: enough units for `want`, and none longer than `most` products, but none shorter than
// eight (gradients of 40 fp32 rows over 5,000 x 300: four 35.6 us, eight 37, sixteen 33.6; of larger
// cases within 1 %).
int32_t splits_for(int64_t tiles, int64_t steps, int64_t pairs, int64_t want, int64_t most) {
    const int64_t n = std::min(std::max((want + tiles - 1) / tiles, (steps * pairs + most - 1) / most),
                               std::max<int64_t>(1, std::min(steps, steps * pairs / 8)));
    const int64_t per = (steps + n - 1) / n;
    return static_cast<int32_t>((steps + per - 1) / per);
}

BackwardPlan backward_plan(const HeadCall& c, int sms, bool want_hidden, bool want_head) {
    BackwardPlan p{};
    const int64_t per = c.grad_terms * c.rows * 2 + (c.w_direct ? 0 : c.terms * c.ld * 2);
    p.piece = piece_rows(c, per, kBackwardBudget);
    const int64_t piece = std::min(p.piece, c.vocab);
    const int64_t grid = c.pair ? sms / 2 : sms, tile = tile_rows(c.pair);
    const int64_t cols = c.width <= kTileNarrow ? kTileNarrow : kTileCols;
    const int64_t across = (c.width + cols - 1) / cols;
    const int64_t pairs = c.terms == 3 ? 6 : c.grad_terms;
    p.part_ld = (c.width + 7) / 8 * 8;
    // both products share a launch: units of like length, the longer ones first, so that its
    // last round is nearly full (at least 16, 64 or 256 products in a unit of hidden's: 1,652 bf16 rows
    // over 96,011 x 155 302, 310 and 301 us, 4,096 over 73,760 x 2,048 2.05, 2.10 and 2.12 ms, 200 over
    // 30,000 x 700 100, 104 and 104 us)
    const int64_t head_steps = (c.rows + 63) / 64, hidden_steps = (piece + 63) / 64;
    p.head_splits = splits_for((piece + tile - 1) / tile * across, head_steps, pairs, grid, INT64_MAX / 2);
    p.hidden_splits = splits_for((c.rows + tile - 1) / tile * across, hidden_steps, pairs, 2 * grid,
                                 std::max<int64_t>(64, 2 * head_steps * pairs));
    if (c.few32) {  // head^T G^T: tiles of 128 columns of the head, steps of 32 of its rows
        const int64_t steps = (piece + 31) / 32, tiles = (c.width + 127) / 128;
        p.hidden_splits = p.hidden_ranges = splits_for(tiles, steps, 6, 2 * sms, INT64_MAX / 2);
    }
    int64_t at = 0;
    p.x = at;
    at += term_bytes(c, c.rows);
    p.w = at;
    if (!c.w_direct) at += term_bytes(c, piece);
    p.grad = at;
    // G [rows][piece], or of few rows G^T [piece][rows, to a multiple of eight]
    p.grad_ld = c.few ? (c.rows + 7) / 8 * 8 : p.piece;
    p.grad_stride = p.grad_ld * (c.few ? p.piece : c.rows);
    at += padded(c.grad_terms * p.grad_stride * 2);
    p.hidden = at;
    if (want_hidden && c.few32)
        at += padded(p.hidden_splits * c.width * p.grad_ld * 4);
    else if (want_hidden && (p.hidden_splits > 1 || p.piece < c.vocab))
        at += padded(p.hidden_splits * c.rows * p.part_ld * 4);
    p.head = at;
    if (want_head && p.head_splits > 1) at += padded(p.head_splits * piece * p.part_ld * 4);
    p.bytes = at;
    return p;
}

cudaError_t join_parts(const HeadCall& c, const float* part, int64_t rows, int32_t splits, void* out,
                       int64_t stride, int sms, cudaStream_t s) {
    const int64_t ld = (c.width + 7) / 8 * 8;
    JoinArgs a{part, rows, c.width, ld, splits, out, stride};
    const bool runs = splits > 16 && rows * ld < (int64_t(1) << 20);
    const int64_t tiles = (ld + 127) / 128 * (runs ? rows : (rows + 7) / 8);
    const int64_t blocks = std::min<int64_t>(tiles, int64_t(sms) * 16);
    if (c.dtype == CAM_F32)
        return runs ? launch(join_kernel<float, 8>, blocks, a, s)
                    : launch(join_kernel<float, 1>, blocks, a, s);
    return runs ? launch(join_kernel<__nv_bfloat16, 8>, blocks, a, s)
                : launch(join_kernel<__nv_bfloat16, 1>, blocks, a, s);
}

int fail(const char* fn, cudaError_t ce) {
    return record_error(CAM_E_CUDA, "%s: launch: %s", fn, cudaGetErrorString(ce));
}

int check_workspace(const char* fn, const void* ws, int64_t bytes, int64_t need) {
    if (need > 0 && !ws) return record_error(CAM_E_ARG, "%s: workspace is NULL", fn);
    if (reinterpret_cast<uintptr_t>(ws) % 256 != 0)
        return record_error(CAM_E_ARG, "%s: workspace is not 256-byte aligned", fn);
    if (bytes < need)
        return record_error(CAM_E_ARG, "%s: workspace of %lld bytes, %lld needed", fn,
                            static_cast<long long>(bytes), static_cast<long long>(need));
    return CAM_OK;
}

int device_of(const char* fn, int* sms) {
    int dev = 0;
    const cudaError_t ce = current_device(&dev, sms);
    return ce == cudaSuccess ? CAM_OK
                             : record_error(CAM_E_CUDA, "%s: no usable CUDA device: %s", fn,
                                            cudaGetErrorString(ce));
}

}  // namespace
}  // namespace cam

using cam::record_error;

CAM_API int cam_head_logprobs_workspace(int64_t rows, int64_t vocab, int64_t width,
                                        const void* hidden, int64_t hidden_stride, const void* head,
                                        int64_t head_stride, cam_dtype dtype, int64_t* bytes) {
    using namespace cam;
    const char* fn = "cam_head_logprobs_workspace";
    if (!bytes) return record_error(CAM_E_ARG, "%s: bytes is NULL", fn);
    HeadCall c{rows, vocab, width, {hidden, rows, hidden_stride}, {head, vocab, head_stride}, dtype};
    if (const int rc = check_head(fn, c)) return rc;
    *bytes = rows ? forward_plan(c).bytes : 0;
    return CAM_OK;
}

CAM_API int cam_head_logprobs(int64_t rows, int64_t vocab, int64_t width, const void* hidden,
                              int64_t hidden_stride, const void* head, int64_t head_stride,
                              cam_dtype dtype, const int64_t* tokens, float* logp, float* entropy,
                              float* lse, float* lse_lo, void* workspace, int64_t workspace_bytes,
                              void* stream) {
    using namespace cam;
    const char* fn = "cam_head_logprobs";
    HeadCall c{rows, vocab, width, {hidden, rows, hidden_stride}, {head, vocab, head_stride}, dtype};
    if (const int rc = check_head(fn, c)) return rc;
    if ((tokens == nullptr) != (logp == nullptr) && rows > 0)
        return record_error(CAM_E_ARG, "%s: tokens and logp go together", fn);
    if (rows == 0) return CAM_OK;
    const ForwardPlan p = forward_plan(c);
    if (const int rc = check_workspace(fn, workspace, workspace_bytes, p.bytes)) return rc;
    int sms = 0;
    if (const int rc = device_of(fn, &sms)) return rc;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    char* ws = static_cast<char*>(workspace);
    TileStat* stats = reinterpret_cast<TileStat*>(ws + p.stats);
    float* mine = reinterpret_cast<float*>(ws + p.mine);
    cudaError_t ce = cudaSuccess;
    for (int64_t at = 0; at < vocab && ce == cudaSuccess; at += p.piece) {
        const int64_t n = std::min(p.piece, vocab - at);
        const Matrix piece = piece_of(c, at);
        ce = make_terms(c, c.hidden, c.x_direct || at > 0 ? 0 : rows, ws + p.x, false, piece,
                        c.w_direct ? 0 : n, ws + p.w, nullptr, nullptr, nullptr, sms, s);
        if (ce != cudaSuccess) break;
        TileProduct t{};
        t.a = operand(c, c.hidden, rows, c.x_direct, ws + p.x, false);
        if (!c.few32) t.b = operand(c, piece, n, c.w_direct, ws + p.w, false);
        if (c.few) std::swap(t.a, t.b);
        t.splits = 1;
        t.out.stats = stats + at / (c.few ? 32 : kTileCols) * rows;
        t.out.mine = mine;
        t.out.tokens = tokens;
        t.out.token0 = at;
        t.out.vocab = vocab;
        if (const int rc = c.few32 ? few32_product(fn, head32(c, piece, n, t), kTileStatsFew, sms, s)
                                   : tile_products(fn, &t, 1, false, c.pair,
                                                   c.few ? kTileStatsFew : kTileStats, sms, s))
            return rc;
    }
    if (ce == cudaSuccess) {
        StatArgs a{stats, stat_parts(c), rows, vocab, mine, tokens, logp, entropy, lse, lse_lo};
        ce = rows <= 64 ? launch(stats_kernel<1>, rows, a, s)
                        : launch(stats_kernel<8>, (rows + 7) / 8, a, s);
    }
    return ce == cudaSuccess ? CAM_OK : fail(fn, ce);
}

CAM_API int cam_head_logprobs_backward_workspace(int64_t rows, int64_t vocab, int64_t width,
                                                 const void* head, int64_t head_stride,
                                                 cam_dtype dtype, int64_t* bytes) {
    using namespace cam;
    const char* fn = "cam_head_logprobs_backward_workspace";
    if (!bytes) return record_error(CAM_E_ARG, "%s: bytes is NULL", fn);
    HeadCall c{rows, vocab, width, {head, rows, width}, {head, vocab, head_stride}, dtype};
    if (const int rc = check_head(fn, c)) return rc;
    *bytes = 0;
    if (rows == 0) return CAM_OK;
    int sms = 0;
    if (const int rc = device_of(fn, &sms)) return rc;
    *bytes = backward_plan(c, sms, true, true).bytes;
    return CAM_OK;
}

CAM_API int cam_head_logprobs_backward(int64_t rows, int64_t vocab, int64_t width,
                                       const void* hidden, int64_t hidden_stride, const void* head,
                                       int64_t head_stride, cam_dtype dtype, const int64_t* tokens,
                                       const float* lse, const float* lse_lo, const float* entropy,
                                       const float* grad_logp, const float* grad_entropy,
                                       void* grad_hidden, int64_t grad_hidden_stride,
                                       void* grad_head, int64_t grad_head_stride, void* workspace,
                                       int64_t workspace_bytes, void* stream) {
    using namespace cam;
    const char* fn = "cam_head_logprobs_backward";
    HeadCall c{rows, vocab, width, {hidden, rows, hidden_stride}, {head, vocab, head_stride}, dtype};
    if (const int rc = check_head(fn, c)) return rc;
    // (arrays of no rows may well be NULL)
    if (rows > 0 && !grad_logp && !grad_entropy)
        return record_error(CAM_E_ARG, "%s: grad_logp and grad_entropy are both NULL", fn);
    if (rows > 0 && !grad_hidden && !grad_head)
        return record_error(CAM_E_ARG, "%s: grad_hidden and grad_head are both NULL", fn);
    const int64_t size = dtype == CAM_F32 ? 4 : 2;
    const struct { void* p; int64_t stride; } out[2] = {{grad_hidden, grad_hidden_stride},
                                                        {grad_head, grad_head_stride}};
    for (const auto& o : out) {
        if (!o.p) continue;
        if (o.stride < width || o.stride > (int64_t(1) << 34))
            return record_error(CAM_E_ARG, "%s: stride of a gradient out of range", fn);
        if (reinterpret_cast<uintptr_t>(o.p) % size != 0)
            return record_error(CAM_E_ARG, "%s: a gradient is not aligned to its elements", fn);
        if (rows > 0 && (o.p == hidden || o.p == head))
            return record_error(CAM_E_ARG, "%s: a gradient in the place of an input", fn);
    }
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    int sms = 0;
    if (rows == 0) {  // a sum over no rows
        if (!grad_head) return CAM_OK;
        if (const int rc = device_of(fn, &sms)) return rc;
        const cudaError_t ce = cudaMemset2DAsync(grad_head, grad_head_stride * size, 0, width * size,
                                                 vocab, s);
        return ce == cudaSuccess ? CAM_OK : fail(fn, ce);
    }
    if (grad_logp && !tokens) return record_error(CAM_E_ARG, "%s: grad_logp without tokens", fn);
    if (grad_entropy && !entropy)
        return record_error(CAM_E_ARG, "%s: grad_entropy without entropy", fn);
    if (!lse) return record_error(CAM_E_ARG, "%s: lse is NULL", fn);
    if (!workspace) return record_error(CAM_E_ARG, "%s: workspace is NULL", fn);
    if (const int rc = device_of(fn, &sms)) return rc;
    const BackwardPlan p = backward_plan(c, sms, grad_hidden != nullptr, grad_head != nullptr);
    if (const int rc = check_workspace(fn, workspace, workspace_bytes, p.bytes)) return rc;
    char* ws = static_cast<char*>(workspace);
    cudaError_t ce = cudaSuccess;
    const bool parts = p.hidden_splits > 1 || p.piece < vocab;
    for (int64_t at = 0; at < vocab && ce == cudaSuccess; at += p.piece) {
        const int64_t n = std::min(p.piece, vocab - at);
        const Matrix piece = piece_of(c, at);
        // hidden states in terms, rows without a gradient as zeros: what they hold, NaN say,
        // then reaches nothing
        ce = make_terms(c, c.hidden, at > 0 ? 0 : rows, ws + p.x, true, piece, c.w_direct ? 0 : n,
                        ws + p.w, tokens, grad_logp, grad_entropy, sms, s);
        if (ce != cudaSuccess) break;
        TileProduct t{};
        t.a = operand(c, c.hidden, rows, false, ws + p.x, false);
        if (!c.few32) t.b = operand(c, piece, n, c.w_direct, ws + p.w, false);
        if (c.few) std::swap(t.a, t.b);
        t.splits = 1;
        t.out.y = ws + p.grad;
        t.out.ldy = p.grad_ld;
        t.out.planes = c.grad_terms;
        t.out.plane_stride = p.grad_stride;
        t.out.tokens = tokens;
        t.out.token0 = at;
        t.out.vocab = vocab;
        t.out.lse = lse;
        t.out.lse_lo = lse_lo;
        t.out.entropy = entropy;
        t.out.g = grad_logp;
        t.out.h = grad_entropy;
        if (const int rc = c.few32 ? few32_product(fn, head32(c, piece, n, t), kTileGradFew, sms, s)
                                   : tile_products(fn, &t, 1, false, c.pair,
                                                   c.few ? kTileGradFew : kTileGrad, sms, s))
            return rc;

        TileOperand grad{};
        grad.base = ws + p.grad;
        grad.ld = p.grad_ld;
        grad.planes = c.grad_terms;
        grad.plane_stride = p.grad_stride;
        TileProduct both[2] = {};
        int count = 0;
        if (grad_hidden && c.few32) {  // head^T G^T, turned by join_turned
            Few32Product q{};
            q.w = static_cast<const float*>(piece.base);
            q.w_rows = n;
            q.width = width;
            q.w_stride = piece.stride;
            q.turned = true;
            q.b = grad;
            q.b.rows = rows;
            q.b.k = n;
            q.b.mn_major = true;
            q.splits = p.hidden_splits;
            q.out.part = reinterpret_cast<float*>(ws + p.hidden);
            q.out.part_ld = p.grad_ld;
            q.out.add = at > 0;
            if (const int rc = few32_product(fn, q, kTileOut, sms, s)) return rc;
        } else if (grad_hidden) {
            TileProduct& q = both[count++];
            q.a = grad;
            q.a.rows = rows;
            q.a.k = n;
            q.a.mn_major = c.few;
            q.b = operand(c, piece, n, c.w_direct, ws + p.w, true);
            q.splits = p.hidden_splits;
            if (parts) {
                q.out.part = reinterpret_cast<float*>(ws + p.hidden);
                q.out.part_ld = p.part_ld;
                q.out.add = at > 0;
            } else {
                q.out.y = grad_hidden;
                q.out.ldy = grad_hidden_stride;
                q.out.y_bf16 = dtype == CAM_BF16;
            }
        }
        if (grad_head) {
            TileProduct& q = both[count++];
            q.a = grad;
            q.a.rows = n;
            q.a.k = rows;
            q.a.mn_major = !c.few;
            q.b = operand(c, c.hidden, rows, false, ws + p.x, true);
            q.splits = p.head_splits;
            if (p.head_splits > 1) {
                q.out.part = reinterpret_cast<float*>(ws + p.head);
                q.out.part_ld = p.part_ld;
            } else {
                q.out.y = static_cast<char*>(grad_head) + at * grad_head_stride * size;
                q.out.ldy = grad_head_stride;
                q.out.y_bf16 = dtype == CAM_BF16;
            }
        }
        if (count > 0)
            if (const int rc = tile_products(fn, both, count, false, c.pair, kTileOut, sms, s)) return rc;
        if (grad_head && p.head_splits > 1)
            ce = join_parts(c, reinterpret_cast<const float*>(ws + p.head), n, p.head_splits,
                            static_cast<char*>(grad_head) + at * grad_head_stride * size,
                            grad_head_stride, sms, s);
    }
    if (ce == cudaSuccess && grad_hidden && c.few32) {
        JoinArgs a{reinterpret_cast<const float*>(ws + p.hidden), rows, width, p.grad_ld,
                   p.hidden_ranges, grad_hidden, grad_hidden_stride};
        ce = launch(join_turned, (width + 3) / 4 * ((rows + 31) / 32), a, s);
    } else if (ce == cudaSuccess && grad_hidden && parts)
        ce = join_parts(c, reinterpret_cast<const float*>(ws + p.hidden), rows, p.hidden_splits,
                        grad_hidden, grad_hidden_stride, sms, s);
    return ce == cudaSuccess ? CAM_OK : fail(fn, ce);
}
