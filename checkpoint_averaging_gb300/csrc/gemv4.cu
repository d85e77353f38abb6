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
// group's sum (for one or two tokens in the output's). The group's scale
// multiplies the group's fp32 sum. The
// weights stay in the lane that loaded them: mma.sync takes them from
// registers, where the 4-bit words are widened (two instructions per two
// weights), while tcgen05 wants them written to shared or tensor memory first.
// A tcgen05 form (weights widened into tensor memory as the first operand, a
// group's sums read back and scaled by warps of their own) was built and
// measured over 73,760 x 2,048: 34.5 us for one bf16 token, 36 for 16, 45 for
// 32 and 108 for 32 fp32 tokens, against 23, 31, 43 and 86 us of this form then.
// One token's 22.5 us are 3.6 TB/s, 52 % of the copy rate. No unit is full: 61 %
// of the issue slots are taken (188 instructions per 2,048 weights, 88 of them
// to widen), the ALU pipe 52 %, the tensor cores 21 %, HBM 47 %, with 24 warps
// per SM. What is left is latency that so many warps do not cover. 32 fp32
// tokens take 84 us, the tensor cores 58 % busy.
//
// A block has a run of the matrix's 16-row tiles, a like share for every block,
// and holds x in shared memory in the order of the operand. Its warps share out
// the run's 128-column records evenly, in the order they lie in memory: each
// streams its part through a private ring of cp.async slots, as one straight
// read, and never waits for another until it is done. A tile that is cut
// between warps belongs to the warp that has its first record; the others leave
// their sums in shared memory, and after one barrier the owner adds them, in
// order. Where x's rows are too long for shared memory they are taken in slabs
// of columns, a tile's sums kept in shared memory from slab to slab; where there
// are too few rows to fill the GPU, the blocks of a cluster take the slabs of one
// run of tiles side by side and add up through distributed shared memory.
#include <cooperative_groups.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <atomic>
#include <type_traits>

#include "cam_internal.h"
#include "op_launch.h"
#include "pack4_layout.h"

#define CAM_API extern "C" __attribute__((visibility("default")))

namespace cam {
namespace {

namespace cg = cooperative_groups;

struct GemvArgs {
    const void* x;
    const uint8_t* packed;
    void* y;
    int64_t x_stride, y_stride;
    int64_t rows;
    int32_t cols;
    int32_t tokens;       // of the call
    int32_t pass_tokens;  // of one pass (grid.y passes)
    int32_t n_blk;        // 128-column records of a tile
    int32_t slab_blk;     // of which x has so many in shared memory at once
    int32_t tiles, more;  // 16-row tiles of a run, and the first runs that have one more
    int32_t cluster;      // blocks that share a run of tiles, each with its own slabs
    int32_t y_bf16, x_vec;
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

// Where x stands in shared memory: the 16 runs (of 8 elements, 16 bytes) of a
// record's column together, run 4 i + t (elements 32 i + 8 t .. + 7) in place
// (4 i + t) ^ (odd << 2), so that the lanes of two neighbouring columns, one of
// them odd, read different banks. An fp32 x has three columns for a token, n_tok
// apart; `odd` goes by the token, or by the column where one operand has all.
__device__ __forceinline__ int x_place(int record, int C, int column, int run, int odd) {
    return (record * C + column) * 16 + (run ^ (odd << 2));
}

// A slab of x into shared memory. Elements past the end are 0.
template <bool F32, bool kPacked, int kAhead>
__device__ __forceinline__ void stage_x(const GemvArgs& a, uint4* xs, int m0, int n_tok, int C,
                                        int blk0, int n_my) {
    using Raw = std::conditional_t<F32, float, uint16_t>;
    const Raw* x = static_cast<const Raw*>(a.x);
    const int runs = n_my * 16, n = runs * n_tok;
    for (int i0 = threadIdx.x; i0 < n; i0 += kAhead * blockDim.x) {
        alignas(16) Raw v[kAhead][8];
        uint4* dst[kAhead];  // (the first column's)
        int token[kAhead];
#pragma unroll
        for (int u = 0; u < kAhead; ++u) {
            const int idx = i0 + u * blockDim.x;
            if (idx >= n) break;
            const int m = idx / runs, run = idx - m * runs;  // run = (record, i, t)
            const int k = blk0 * kP4Cols + run * 8;
            const int left = min(8, a.cols - k);
            const Raw* p = x + int64_t(m0 + m) * a.x_stride + k;
            dst[u] = xs + x_place(run >> 4, C, m, run & 15, kPacked ? 0 : m & 1);
            token[u] = m;
            if (a.x_vec && left == 8) {
#pragma unroll
                for (int h = 0; h < (F32 ? 2 : 1); ++h)
                    reinterpret_cast<uint4*>(v[u])[h] = __ldg(reinterpret_cast<const uint4*>(p) + h);
            } else {
#pragma unroll
                for (int j = 0; j < 8; ++j) v[u][j] = j < left ? __ldg(p + j) : Raw(0);
            }
        }
#pragma unroll
        for (int u = 0; u < kAhead; ++u) {
            if (i0 + u * static_cast<int>(blockDim.x) >= n) break;
            if constexpr (F32) {
                uint32_t w[3][4];
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    uint32_t lo[3], hi[3];
                    terms(v[u][2 * j], lo);
                    terms(v[u][2 * j + 1], hi);
#pragma unroll
                    for (int q = 0; q < 3; ++q) w[q][j] = lo[q] | (hi[q] << 16);
                }
#pragma unroll
                for (int q = 0; q < 3; ++q) {
                    const int column = q * n_tok + token[u];
                    uint4* to = dst[u] + q * n_tok * 16;
                    if (kPacked && (column & 1))  // (the run's place in a pair of fours)
                        to = xs + (static_cast<int>(to - xs) ^ 4);
                    *to = make_uint4(w[q][0], w[q][1], w[q][2], w[q][3]);
                }
            } else {
                uint32_t w[4];
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    w[j] = v[u][2 * j] | (static_cast<uint32_t>(v[u][2 * j + 1]) << 16);
                *dst[u] = make_uint4(w[0], w[1], w[2], w[3]);
            }
        }
    }
}

__device__ __forceinline__ uint16_t round_bf16(float v) {
    return __bfloat16_as_ushort(__float2bfloat16_rn(v));
}

// The forms of the kernel by columns of x: NT operands of 8 columns. bf16: up to
// 8, 16 or 32 tokens (NT 1, 2, 4). fp32: up to 2 tokens packed in one operand
// (NT 1), else three operands for each 8 tokens (NT 3, 6) that add up in the
// same accumulators. Few columns take many small blocks per SM, many
// columns one large one, whose warps share its x.
template <bool F32, int NT>
struct GvForm {
    static constexpr bool kPacked = F32 && NT == 1;
    static constexpr int kWarps = NT <= 2 ? 8 : 16;
    static constexpr int kBlocks = NT == 1 ? 3 : NT == 2 ? 2 : 1;  // per SM
    static constexpr int kDepth = NT <= 2 ? 6 : 4;                 // ring slots per warp
    // Runs of x that a thread stages at once. More loads in flight help long rows, more registers
    // cost the loop. In us with 1 / 2 / 4 / 6 of them:
    //   bf16  8 tokens  16,384 x 9,000 26.7 25.8 25.8 26.2  73,760 x 2,048 21.4 20.5 20.7 21.4
    //        10         16,384 x 9,000 32.4 31.4 29.9 29.5  3,000 x 16,000 22.2 20.7 18.6 18.2
    //        32         16,384 x 9,000 52.2 50.0 47.5 52.0  3,000 x 16,000 42.9 41.2 38.5 46.9
    //   fp32  1         16,384 x 9,000 21.6 23.0 23.2 27.2  73,760 x 2,048 21.1 22.3 22.5 25.0
    //         8         16,384 x 9,000 34.7 34.5 34.4 35.4  40,000 x 3,700 29.9 29.5 29.5 30.7
    //        32         16,384 x 9,000 91.5 92.5 95.7 98.7  73,760 x 2,048 84.1 84.9 88.1 93.3
    static constexpr int kAhead = F32 ? (NT == 3 ? 2 : 1) : NT == 4 ? 4 : NT == 2 ? 6 : 2;
    static constexpr int kOut = F32 && NT > 1 ? NT / 3 : NT;       // operands of sums kept
    static constexpr int kTokens = F32 ? (NT == 1 ? 2 : 8 * NT / 3) : 8 * NT;
};

template <bool F32, int NT, int GROUP>
__global__ void __launch_bounds__(GvForm<F32, NT>::kWarps * 32, GvForm<F32, NT>::kBlocks)
    gemv4(const __grid_constant__ GemvArgs a) {
    using Form = GvForm<F32, NT>;
    constexpr int kTile = p4_tile_bytes(GROUP), kPer = kP4Cols / GROUP;
    constexpr int kWarps = Form::kWarps, kDepth = Form::kDepth, kOut = Form::kOut;
    extern __shared__ __align__(128) uint8_t smem[];
    int* slot_tile = reinterpret_cast<int*>(smem);  // (128 bytes)

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
    const int m0 = blockIdx.y * a.pass_tokens;
    const int n_tok = min(a.pass_tokens, a.tokens - m0);
    const int C = F32 ? 3 * n_tok : n_tok;
    const int rank = a.cluster > 1 ? static_cast<int>(cg::this_cluster().block_rank()) : 0;
    const int run = a.cluster > 1 ? blockIdx.x / a.cluster : blockIdx.x;
    int tile0 = run * a.tiles + min(run, a.more);
    int my_tiles = a.tiles + (run < a.more ? 1 : 0);
    asm volatile("" : "+r"(tile0), "+r"(my_tiles));  // (kept, not worked out again at each use)
    const bool slabs = a.slab_blk < a.n_blk;
    const int first_blk = rank * a.slab_blk, next_slab = a.cluster * a.slab_blk;

    // the rings, the slots of cut tiles' sums, x, and (slabs) every tile's sums
    uint8_t* ring = smem + 128 + warp * (kDepth * kTile);
    float4* slot = reinterpret_cast<float4*>(smem + 128 + kWarps * kDepth * kTile);
    uint4* xs = reinterpret_cast<uint4*>(slot + kWarps * kOut * 32);
    float4* kept = reinterpret_cast<float4*>(xs + a.slab_blk * 16 * C);

    // this warp's records of the slab that starts at record blk0 of each tile
    auto range = [&](int blk0, int& begin, int& end) {
        const int64_t n = int64_t(my_tiles) * min(a.slab_blk, a.n_blk - blk0);
        begin = static_cast<int>(n * warp / kWarps);
        end = static_cast<int>(n * (warp + 1) / kWarps);
    };

    // loads run ahead of the sums, over tiles and slabs
    int l_blk0 = first_blk, l_nb = 0, l_run = 0, l_left = 0;  // l_run: records in one piece
    bool l_more = a.n_blk > 0;
    const uint8_t* l_src = nullptr;
    auto open_slab = [&]() {  // to the first of this warp's records, from slab l_blk0 on
        for (; l_more; l_blk0 += next_slab) {
            if (l_blk0 >= a.n_blk) {
                l_more = false;
                return;
            }
            int begin, end;
            range(l_blk0, begin, end);
            l_nb = min(a.slab_blk, a.n_blk - l_blk0);
            if (begin == end) continue;
            const int tile = begin / l_nb, at = begin - tile * l_nb;
            l_left = end - begin;
            l_run = slabs ? min(l_nb - at, l_left) : l_left;
            l_left -= l_run;
            l_src = a.packed + (int64_t(tile0 + tile) * a.n_blk + l_blk0 + at) * kTile + lane * 16;
            return;
        }
    };
    open_slab();
    uint32_t l_dst = static_cast<uint32_t>(__cvta_generic_to_shared(ring)) + lane * 16;
    const uint32_t ring_end = l_dst + kDepth * kTile;
    auto load = [&]() {
        if (l_more) {
            cp16(l_dst, l_src);
            cp16(l_dst + 512, l_src + 512);
            if (lane < kPer * 2) cp16(l_dst + 1024, l_src + 1024);
            l_src += kTile;
            if (--l_run == 0) {
                if (l_left > 0) {  // (of a slab: on to the next tile's)
                    l_src += int64_t(a.n_blk - l_nb) * kTile;
                    l_run = min(l_nb, l_left);
                    l_left -= l_run;
                } else {
                    l_blk0 += next_slab;
                    open_slab();
                }
            }
        }
        cp_commit();
        l_dst += kTile;
        if (l_dst == ring_end) l_dst -= kDepth * kTile;
    };
#pragma unroll
    for (int s = 0; s < kDepth - 1; ++s) load();

    // this lane's column of each operand; past the last token any will do, its results are not
    // kept
    int x_lane[NT];
    const int x_odd = -8 * (g & 1);  // (steps change places in pairs)
#pragma unroll
    for (int n = 0; n < NT; ++n) {
        if constexpr (F32 && NT > 1)
            x_lane[n] = x_place(0, C, n / kOut * n_tok + min(8 * (n % kOut) + g, n_tok - 1), t, g & 1);
        else
            x_lane[n] = x_place(0, C, min(8 * n + g, C - 1), t, g & 1);
    }

    // A tile's finished sums. v[n]: rows g (x, y) and g + 8 (z, w), columns 8 n + 2 t and + 1.
    auto write = [&](int tile, const float4 (&v)[kOut]) {
        const int64_t row = int64_t(tile) * kP4Rows + g;
        auto put = [&](int m, int64_t r, float value) {
            if (m >= n_tok || r >= a.rows) return;
            const int64_t to = int64_t(m0 + m) * a.y_stride + r;
            if (a.y_bf16) static_cast<uint16_t*>(a.y)[to] = round_bf16(value);
            else static_cast<float*>(a.y)[to] = value;
        };
        if constexpr (Form::kPacked) {
            // a token's three columns stand in neighbouring lanes
            for (int m = 0; m < n_tok; ++m) {
                float lo = 0.0f, hi = 0.0f;
                for (int q = 2; q >= 0; --q) {
                    const int c = q * n_tok + m, from = (lane & ~3) | (c >> 1);
                    const float x = __shfl_sync(0xFFFFFFFFu, v[0].x, from);
                    const float y = __shfl_sync(0xFFFFFFFFu, v[0].y, from);
                    const float z = __shfl_sync(0xFFFFFFFFu, v[0].z, from);
                    const float w = __shfl_sync(0xFFFFFFFFu, v[0].w, from);
                    lo += (c & 1) ? y : x;
                    hi += (c & 1) ? w : z;
                }
                if (t == 0) put(m, row, lo);
                if (t == 1) put(m, row + 8, hi);
            }
        } else {
#pragma unroll
            for (int n = 0; n < kOut; ++n) {
                const int m = 8 * n + 2 * t;
                put(m, row, v[n].x);
                put(m + 1, row, v[n].y);
                put(m, row + 8, v[n].z);
                put(m + 1, row + 8, v[n].w);
            }
        }
    };
    auto add = [](float4& s, const float4& v) {
        s.x += v.x, s.y += v.y, s.z += v.z, s.w += v.w;
    };
    // ... of this slab: to the result, or onto what the slabs before left
    auto finish = [&](int tile, int blk0, float4 (&v)[kOut]) {
        if (slabs) {
            float4* k = kept + (tile - tile0) * kOut * 32 + lane;
            const bool last = a.cluster == 1 && blk0 + next_slab >= a.n_blk;
#pragma unroll
            for (int n = 0; n < kOut; ++n) {
                if (blk0 > first_blk) {
                    float4 s = k[n * 32];
                    add(s, v[n]);
                    v[n] = s;
                }
                if (!last) k[n * 32] = v[n];
            }
            if (!last) return;
        }
        write(tile, v);
    };

    int at = 0;  // the ring's slot under way
    for (int blk0 = first_blk; blk0 == 0 || blk0 < a.n_blk; blk0 += next_slab) {
        const int nb = min(a.slab_blk, a.n_blk - blk0);
        if (blk0 > first_blk) __syncthreads();  // every warp is done with the slab of x before
        stage_x<F32, Form::kPacked, Form::kAhead>(a, xs, m0, n_tok, C, blk0, nb);
        if (lane == 0) slot_tile[warp] = -1;
        __syncthreads();
        if (nb == 0) {  // no columns: the sums are 0
            float4 zero[kOut];
#pragma unroll
            for (int n = 0; n < kOut; ++n) zero[n] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
            for (int i = warp; i < my_tiles; i += kWarps) write(tile0 + i, zero);
            return;
        }
        int begin, end;
        range(blk0, begin, end);
        int tile = begin / nb, b = begin - tile * nb;
        tile += tile0;
        bool owner = b == 0, open = false;  // the tile under way: has its first record; not finished
        float acc[kOut][4];
        float4 v[kOut];
        auto gather = [&]() {
#pragma unroll
            for (int n = 0; n < kOut; ++n)
                v[n] = make_float4(acc[n][0], acc[n][1], acc[n][2], acc[n][3]);
        };
        auto leave = [&]() {  // another warp's tile
            gather();
#pragma unroll
            for (int n = 0; n < kOut; ++n) slot[(warp * kOut + n) * 32 + lane] = v[n];
            if (lane == 0) slot_tile[warp] = tile;
        };
#pragma unroll
        for (int n = 0; n < kOut; ++n)
#pragma unroll
            for (int j = 0; j < 4; ++j) acc[n][j] = 0.0f;
        for (int left = end - begin; left > 0;) {  // a tile's records at a time
            int here = min(left, nb - b);
            left -= here;
            open = b + here < nb;
            const uint4* xb = xs + b * 16 * C;
#pragma unroll 1
            for (; here > 0; --here, xb += 16 * C) {
                cp_wait<kDepth - 2>();
                __syncwarp();  // every lane's copies are in, and every lane is done with the slot before
                load();
                const uint8_t* q = ring + at;
                at += kTile;
                if (at == kDepth * kTile) at = 0;
                const uint4 wl = *reinterpret_cast<const uint4*>(q + lane * 16);
                const uint4 wh = *reinterpret_cast<const uint4*>(q + 512 + lane * 16);
                uint32_t sl[kPer > 1 ? kPer / 2 : 1], sh[kPer > 1 ? kPer / 2 : 1];  // bf16 pairs
                const uint8_t* sp = q + 1024 + g * (4 * kPer);
                if constexpr (kPer == 4) {
                    const uint4 s = *reinterpret_cast<const uint4*>(sp);
                    sl[0] = s.x, sl[1] = s.y, sh[0] = s.z, sh[1] = s.w;
                } else if constexpr (kPer == 2) {
                    const uint2 s = *reinterpret_cast<const uint2*>(sp);
                    sl[0] = s.x, sh[0] = s.y;
                } else {
                    sl[0] = *reinterpret_cast<const uint32_t*>(sp);
                    sh[0] = sl[0] >> 16;
                }
                constexpr int kSteps = GROUP / 32;  // steps of 32 columns per group
#pragma unroll
                for (int j = 0; j < kPer; ++j) {
                    uint32_t al[kSteps][4], ah[kSteps][4];
#pragma unroll
                    for (int k = 0; k < kSteps; ++k) {
                        const int i = j * kSteps + k;
                        const uint32_t lo = i == 0 ? wl.x : i == 1 ? wl.y : i == 2 ? wl.z : wl.w;
                        const uint32_t hi = i == 0 ? wh.x : i == 1 ? wh.y : i == 2 ? wh.z : wh.w;
#pragma unroll
                        for (int p = 0; p < 4; ++p) al[k][p] = widen(lo, p), ah[k][p] = widen(hi, p);
                    }
                    // a token's three terms in one sum, over the whole group the smallest first (step
                    // by step the sum's error is three times as large at group 128; in sums of their
                    // own 32 tokens over 73,760 x 2,048 took 100 us where this took 92)
                    float part[kOut][4];
#pragma unroll
                    for (int q = NT / kOut - 1; q >= 0; --q)
#pragma unroll
                        for (int k = 0; k < kSteps; ++k)
#pragma unroll
                            for (int n = 0; n < kOut; ++n) {
                                const int i = j * kSteps + k;
                                const uint4 x = xb[x_lane[q * kOut + n] + 4 * i + ((i & 1) ? x_odd : 0)];
                                if (q == NT / kOut - 1 && k == 0)
                                    mma_first(part[n], al[k][0], ah[k][0], al[k][1], ah[k][1], x.x, x.y);
                                else
                                    mma(part[n], al[k][0], ah[k][0], al[k][1], ah[k][1], x.x, x.y);
                                mma(part[n], al[k][2], ah[k][2], al[k][3], ah[k][3], x.z, x.w);
                            }
                    const float s0 = __uint_as_float((j & 1) ? sl[j >> 1] & 0xFFFF0000u : sl[j >> 1] << 16);
                    const float s1 = __uint_as_float((j & 1) ? sh[j >> 1] & 0xFFFF0000u : sh[j >> 1] << 16);
#pragma unroll
                    for (int n = 0; n < kOut; ++n) {
                        acc[n][0] = fmaf(s0, part[n][0], acc[n][0]);
                        acc[n][1] = fmaf(s0, part[n][1], acc[n][1]);
                        acc[n][2] = fmaf(s1, part[n][2], acc[n][2]);
                        acc[n][3] = fmaf(s1, part[n][3], acc[n][3]);
                    }
                }
            }
            if (!open) {
                if (owner) {
                    gather();
                    finish(tile, blk0, v);
                } else {
                    leave();
                }
#pragma unroll
                for (int n = 0; n < kOut; ++n)
#pragma unroll
                    for (int j = 0; j < 4; ++j) acc[n][j] = 0.0f;
                b = 0, ++tile;
                owner = true;
            }
        }
        if (open && !owner) leave();
        __syncthreads();
        if (open && owner) {
            gather();
            for (int w = warp + 1; w < kWarps; ++w) {
                if (slot_tile[w] != tile) continue;
#pragma unroll
                for (int n = 0; n < kOut; ++n) add(v[n], slot[(w * kOut + n) * 32 + lane]);
            }
            finish(tile, blk0, v);
        }
    }
    cp_wait<0>();
    if (a.cluster > 1) {
        // a tile's sums from all blocks, in the order of their slabs
        cg::cluster_group cluster = cg::this_cluster();
        cluster.sync();
        for (int i = rank * kWarps + warp; i < my_tiles; i += a.cluster * kWarps) {
            float4 v[kOut];
#pragma unroll
            for (int n = 0; n < kOut; ++n) v[n] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
            for (int r = 0; r < a.cluster; ++r) {
                const float4* k = cluster.map_shared_rank(kept, r) + i * kOut * 32 + lane;
#pragma unroll
                for (int n = 0; n < kOut; ++n) add(v[n], k[n * 32]);
            }
            write(tile0 + i, v);
        }
        cluster.sync();  // no block leaves while another reads its sums
    }
}

template <bool F32, int NT>
const void* kernel_for_group(int group) {
    return group == 32   ? reinterpret_cast<const void*>(gemv4<F32, NT, 32>)
           : group == 64 ? reinterpret_cast<const void*>(gemv4<F32, NT, 64>)
                         : reinterpret_cast<const void*>(gemv4<F32, NT, 128>);
}

// A form's launch: its kernel, and what the host needs to know of it.
struct GvPlan {
    const void* kernel;
    int warps, blocks, depth, out, tokens;
    std::atomic<uint64_t>* shared_ok;
};

template <bool F32, int NT>
GvPlan plan_of(int group) {
    using Form = GvForm<F32, NT>;
    static std::atomic<uint64_t> shared_ok[3];
    return {kernel_for_group<F32, NT>(group), Form::kWarps,  Form::kBlocks, Form::kDepth,
            Form::kOut,                       Form::kTokens, &shared_ok[group == 32 ? 0 : group / 64]};
}

GvPlan plan_for(bool f32, int tokens, int group) {
    if (f32)
        return tokens <= 2 ? plan_of<true, 1>(group)
               : tokens <= 8 ? plan_of<true, 3>(group)
                             : plan_of<true, 6>(group);
    return tokens <= 8    ? plan_of<false, 1>(group)
           : tokens <= 16 ? plan_of<false, 2>(group)
                          : plan_of<false, 4>(group);
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
    const auto n_tiles = static_cast<int32_t>((rows + kP4Rows - 1) / kP4Rows);
    a.y_bf16 = y_dtype == CAM_BF16;
    a.x_vec = reinterpret_cast<uintptr_t>(x) % 16 == 0 && x_stride * x_size % 16 == 0;
    // as few passes over the weights as the widest form allows, evenly
    const bool f32 = x_dtype == CAM_F32;
    const int most = f32 ? GvForm<true, 6>::kTokens : GvForm<false, 4>::kTokens;
    int passes = (a.tokens + most - 1) / most;
    a.pass_tokens = (a.tokens + passes - 1) / passes;
    passes = (a.tokens + a.pass_tokens - 1) / a.pass_tokens;
    if (passes > 65535) return record_error(CAM_E_ARG, "%s: too many tokens", fn);
    const GvPlan p = plan_for(f32, a.pass_tokens, group);
    // Shared memory: rings and slots, then x, whole if it fits beside the other blocks of the SM
    // or, alone, in what the tiles' sums leave.
    const int record = 256 * (f32 ? 3 : 1) * a.pass_tokens;  // bytes of x per record of a tile
    const int fixed = 128 + p.warps * (p.depth * p4_tile_bytes(group) + p.out * 512);
    const int64_t all_x = int64_t(record) * a.n_blk;
    int per_sm = p.blocks;
    auto room_of = [&](int k) { return (k > 1 ? 228 * 1024 / k - 1280 : kMaxSharedBytes) - fixed; };
    while (per_sm > 1 && all_x > room_of(per_sm)) {
        // (two blocks whose slabs are two at most, in pairs, do better than one: 8 bf16 tokens over
        // 16,384 x 9,000 33 us against 38; with three slabs 3,000 x 16,000 takes 26 against 21)
        if (per_sm == 2 && 2 * all_x <= 7 * int64_t(room_of(2))) break;
        --per_sm;
    }
    const int room = room_of(per_sm);
    const int64_t blocks_most = std::max(1, sms * per_sm / passes);
    int64_t blocks = std::min<int64_t>(n_tiles, blocks_most);
    int kept = 0;
    a.slab_blk = a.n_blk;
    // few rows: a cluster for each tile or so, as long as a warp has a few records
    a.cluster = 1;
    while (a.cluster < 8 && blocks * passes * a.cluster * 2 <= sms &&
           a.n_blk >= a.cluster * 4 * p.warps)
        a.cluster *= 2;
    // x in slabs: where the tiles' sums leave room, the blocks of a pair take them side by side
    // and stage half as many each (32 tokens over 16,384 x 9,000: bf16 66 -> 54 us, fp32 120 ->
    // 100; larger clusters leave SMs out and take 90 and 180)
    if (a.cluster == 1 && all_x > room && blocks > 1) {
        auto slabs = [&](int c) {  // of a block
            const int64_t runs = std::min<int64_t>(n_tiles, blocks_most / c);
            const int64_t sums = (n_tiles + runs - 1) / runs * p.out * 512;
            const int64_t slab = (room - sums) / record;
            return slab < 1 ? INT64_MAX : (a.n_blk + c * slab - 1) / (c * slab);
        };
        if (slabs(2) < slabs(1)) {
            a.cluster = 2;
            blocks = std::min<int64_t>(n_tiles, blocks_most / 2);
        }
    }
    if (a.cluster > 1 || all_x > room) {
        const int kept_room = room - record, per_tile = p.out * 512;
        const int64_t tiles = kept_room / per_tile;  // a block may have at most
        blocks = std::max(blocks, (n_tiles + tiles - 1) / tiles);
        kept = static_cast<int>((n_tiles + blocks - 1) / blocks) * per_tile;
        a.slab_blk = std::max(1, (room - kept) / record);
        int slabs = (a.n_blk + a.slab_blk - 1) / a.slab_blk;
        slabs = (slabs + a.cluster - 1) / a.cluster * a.cluster;
        a.slab_blk = (a.n_blk + slabs - 1) / slabs;
    }
    a.slab_blk = std::max(1, a.slab_blk);
    a.tiles = static_cast<int32_t>(n_tiles / blocks);
    a.more = static_cast<int32_t>(n_tiles % blocks);
    const int bytes = fixed + kept + a.slab_blk * record;

    if (bytes > 48 * 1024) ce = allow_shared(p.kernel, dev, *p.shared_ok);
    if (ce == cudaSuccess) {
        void* args[] = {&a};
        cudaLaunchConfig_t cfg{};
        cfg.gridDim = dim3(static_cast<unsigned>(blocks * a.cluster), passes);
        cfg.blockDim = dim3(p.warps * 32);
        cfg.dynamicSmemBytes = bytes;
        cfg.stream = s;
        cudaLaunchAttribute attr{};
        attr.id = cudaLaunchAttributeClusterDimension;
        attr.val.clusterDim.x = a.cluster;
        attr.val.clusterDim.y = attr.val.clusterDim.z = 1;
        cfg.attrs = &attr;
        cfg.numAttrs = a.cluster > 1 ? 1 : 0;
        ce = cudaLaunchKernelExC(&cfg, p.kernel, args);
    }
    if (ce != cudaSuccess)
        return record_error(CAM_E_CUDA, "%s: launch: %s", fn, cudaGetErrorString(ce));
    return CAM_OK;
}
