// f32_products.cu -- products of a large fp32 matrix with few rows (few32_product in
// tile_products.h): the logits of few rows by an fp32 head, their gradients, and the
// gradients of the rows' hidden states.
//
// Reading the matrix once bounds these (126 rows by 152,602 x 822: 74 us; its three bf16 terms
// written out, read back six times and multiplied took 497). So the terms are made on the way:
// eight warps copy 128 x 32 fp32 elements per K step into shared memory (cp.async, several steps
// ahead, 16 or 4 bytes each by the rows' alignment), split them into three bf16 tiles in the
// layout that the tensor core reads, and the MMA thread multiplies each with the few rows'
// terms (TMA): the leading product into one TMEM accumulator, the five small ones into another,
// so that what the tensor core's additions lose (tile_products.cu) stays with the few of the
// leading product; its sums are cut into runs of 128 terms.
//
// A persistent grid of one block per SM, 18 warps:
//   warp 0 (one lane)  TMA producer of the few rows' terms
//   warp 1 (one lane)  MMA issuer: D[128 rows of the matrix][64 or 128 few rows]
//   warps 2..9         in two groups that take the steps in turn, 32 rows of the matrix's
//                      tile (or 8 rows of K) each: copied, split
//   warps 10..17       epilogue: a lane is a row of the matrix, its registers the few rows
//
// 18 warps leave 96 registers a thread, which the epilogues do not fit in: for 128 columns 740
// bytes of stores and 992 of loads a thread are spilled for the statistics, 524 and 520 for G, 132 and
// 156 for the gradients' products, for 64 columns 160 and 144, 116 and 112, and 8 and 16.
//
// Waits are bounded as in tile_products.cu.
#include <algorithm>
#include <atomic>
#include <cstring>

#include "cam_internal.h"
#include "op_launch.h"
#include "tc_device.cuh"
#include "tile_device.cuh"

namespace cam {
namespace tc {
namespace {

constexpr int kF32Threads = 576;
constexpr int kRows32 = 128;       // of the matrix's tile
constexpr int kStep = 32;          // elements of K
constexpr int kTermBytes = kRows32 * kStep * 2;  // one term of the matrix's tile
constexpr int kSplitWarps = 8;
constexpr int kGroup = 4;          // of them work on one step (all eight on each: 30 % slower)
constexpr int kSlot = 4096;        // a warp's share of a step, fp32
// Steps of a run: 126 rows over 152,602 x 824 take 280 us, with eight 246; the entropy of one row
// over 11,241 x 1,469 is off by 9.9e-7 of itself, with eight 1.8e-6.
constexpr int kRun32 = 4;

struct alignas(128) Args32 {
    CUtensorMap tx;       // the few rows' terms
    const float* w;
    int64_t w_rows, width, stride;
    int32_t vec;          // rows of w start on 16 bytes
    int32_t m_tiles, units, steps, per_split, tail;
    int64_t M, N;
    TileOut o;
    int32_t* status;
};

// Rings of their own for the matrix's terms, which are made at once when a stage is free, and
// the few rows', whose copies take longer to come (one ring of three stages: 20 rows over
// 152,602 x 824 200 us instead of 193). No more of either than is needed: copies of 4 bytes hold
// lines of L1 while they are under way, and L1 is what shared memory leaves. With six and three
// stages of the few rows' terms for 64 and 128 columns, and with these four and two: 2 rows over
// 18,495 x 3,934 174 and 142 us, 126 over 152,602 x 822 370 and 314; with rows that start on
// 16 bytes (copied past L1) 2 over 18,495 x 3,932 108 and 113, 126 over 152,602 x 824 298 and 280.
template <int COLS>
struct Geo32 {
    static constexpr int kXBytes = 3 * COLS * kStep * 2;
    static constexpr int kWBytes = 3 * kTermBytes;
    static constexpr int kWStages = 3;
    static constexpr int kXStages = COLS == 64 ? 4 : 2;
    static constexpr int kDepth = 2;  // steps that a group copies ahead
    static constexpr int kXAt = kWStages * kWBytes;
    static constexpr int kRawAt = kXAt + kXStages * kXBytes;
    static constexpr int kRowsAt = kRawAt + kSplitWarps * kDepth * kSlot;
    static constexpr int kBarsAt = (kRowsAt + kFew32 * int(sizeof(GradRow)) + 15) / 16 * 16;
    static constexpr int kBars = 2 * kWStages + 2 * kXStages + 5;
    static constexpr int kSmem = kBarsAt + 8 * kBars + 16 + 1024;
    static_assert(kSmem <= kMaxSharedBytes, "over the per-block shared memory limit");
};

// K-major rows of 64 bytes under the 64-byte swizzle, groups of eight rows 512 bytes apart.
__device__ __forceinline__ uint64_t smem_desc64(uint32_t addr) {
    return static_cast<uint64_t>((addr & 0x3FFFFu) >> 4) | (uint64_t(1) << 16) |
           (uint64_t(512 >> 4) << 32) | (uint64_t(1) << 46) | (uint64_t(4) << 61);
}

// Copies `bytes` (at most 16 or 4) and fills the rest with zeros.
__device__ __forceinline__ void copy16(uint32_t dst, const float* src, int bytes) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(bytes)
                 : "memory");
}
__device__ __forceinline__ void copy4(uint32_t dst, const float* src, int bytes) {
    asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(dst), "l"(src), "r"(bytes)
                 : "memory");
}

__device__ __forceinline__ void lds4(uint32_t at, float* v) {
    asm volatile("ld.shared.v4.f32 {%0, %1, %2, %3}, [%4];"
                 : "=f"(v[0]), "=f"(v[1]), "=f"(v[2]), "=f"(v[3])
                 : "r"(at)
                 : "memory");
}

// Eight elements' three terms, to the same place of the three tiles.
__device__ __forceinline__ void split8(float* v, uint32_t at) {
#pragma unroll
    for (int t = 0; t < 3; ++t) {
        uint32_t w[4], high = 0;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            w[i] = bf16x2(v[2 * i], v[2 * i + 1]);
            high |= ((w[i] & 0x7F80u) == 0x7F80u) | ((w[i] & 0x7F800000u) == 0x7F800000u);
        }
        if (t == 0 && high) {  // rounded to an infinity, or one itself
#pragma unroll
            for (int i = 0; i < 4; ++i)
                w[i] = __bfloat16_as_ushort(term(v[2 * i])) |
                       (uint32_t(__bfloat16_as_ushort(term(v[2 * i + 1]))) << 16);
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            v[2 * i] -= __uint_as_float(w[i] << 16);
            v[2 * i + 1] -= __uint_as_float(w[i] & 0xFFFF0000u);
        }
        asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(at + t * kTermBytes), "r"(w[0]),
                     "r"(w[1]), "r"(w[2]), "r"(w[3])
                     : "memory");
    }
}

// A place in a block's sequence of steps.
struct Cursor {
    int u, s, s1, mt;
};
__device__ __forceinline__ void enter(const Args32& a, Cursor& c) {
    const int split = c.u / a.m_tiles;
    c.mt = c.u - split * a.m_tiles;
    c.s = split * a.per_split;
    c.s1 = min(a.steps, c.s + a.per_split);
}
__device__ __forceinline__ void advance(const Args32& a, Cursor& c) {
    if (++c.s == c.s1) {
        c.u += gridDim.x;
        if (c.u < a.units) enter(a, c);
    }
}

template <bool TURNED, int EPI, int COLS>
__global__ void __launch_bounds__(kF32Threads, 1) f32_kernel(const __grid_constant__ Args32 a) {
    using G = Geo32<COLS>;
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>(
        (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    uint64_t* bars = reinterpret_cast<uint64_t*>(smem + G::kBarsAt);
    const uint32_t ring = su32(smem);
    const uint32_t xfull0 = su32(bars);
    const uint32_t xempty0 = xfull0 + 8 * G::kXStages;
    const uint32_t ready0 = xempty0 + 8 * G::kXStages;
    const uint32_t empty0 = ready0 + 8 * G::kWStages;
    const uint32_t tfull0 = empty0 + 8 * G::kWStages;
    const uint32_t tempty0 = tfull0 + 16;
    const uint32_t drain = tempty0 + 16;
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(bars + G::kBars);
    volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
    const int warp = __shfl_sync(0xffffffffu, int(threadIdx.x >> 5), 0), lane = threadIdx.x & 31;

    if (threadIdx.x == 0) {
        for (int s = 0; s < 2 * G::kXStages; ++s) bar_init(xfull0 + 8 * s, 1);  // (and xempty)
        for (int s = 0; s < G::kWStages; ++s) {
            bar_init(ready0 + 8 * s, kGroup);
            bar_init(empty0 + 8 * s, 1);
        }
        for (int i = 0; i < 2; ++i) {
            bar_init(tfull0 + 8 * i, 1);
            bar_init(tempty0 + 8 * i, 8);
        }
        bar_init(drain, 1);
        *abort_flag = 0;
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    if (warp == 1) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], 512;" ::"r"(
                         su32(tmem_slot))
                     : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *tmem_slot;
    asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");

    Cursor c{int(blockIdx.x), 0, 0, 0};
    if (c.u < a.units) enter(a, c);
    if (warp == 0 && elect_one()) {
        // ---- producer of the few rows' terms ----
        int stage = 0;
        uint32_t phase = 0, issued = 0, filled_parity = 0;
        while (c.u < a.units) {
            if (!bar_wait(xempty0 + 8 * stage, phase ^ 1, abort_flag, a.status)) break;
            const uint32_t sx = ring + G::kXAt + stage * G::kXBytes, fb = xfull0 + 8 * stage;
            bar_expect(fb, G::kXBytes);
            if constexpr (TURNED) {
#pragma unroll
                for (int h = 0; h < COLS / 64; ++h)
                    tma_load(sx + h * 3 * 64 * kStep * 2, &a.tx, 64 * h, c.s * kStep, 0, fb);
            } else {
                tma_load(sx, &a.tx, c.s * kStep, 0, 0, fb);
            }
            issued |= 1u << stage;
            filled_parity = (filled_parity & ~(1u << stage)) | (phase << stage);
            if (++stage == G::kXStages) {
                stage = 0;
                phase ^= 1;
            }
            advance(a, c);
        }
        if (*abort_flag) {  // let the copies in flight land
            for (int s = 0; s < G::kXStages; ++s)
                if ((issued >> s) & 1) {
                    const unsigned long long t0 = now_ns();
                    while (!bar_test(xfull0 + 8 * s, (filled_parity >> s) & 1))
                        if (now_ns() - t0 > kTcWaitLimitNs) break;
                }
        }
    } else if (warp == 1 && elect_one()) {
        // ---- MMA issuer ----
        // fp32 accumulator, bf16 operands, majorness in bits 15 and 16, N / 8, M / 16
        constexpr uint32_t idesc = (1u << 4) | (1u << 7) | (1u << 10) |
                                   (uint32_t(TURNED) << 15) | (uint32_t(TURNED) << 16) |
                                   (uint32_t(COLS >> 3) << 17) | (uint32_t(kRows32 >> 4) << 24);
        // 16 elements of K further: 32 bytes along a row, or 16 rows
        constexpr uint64_t kAdvance = TURNED ? 16 * 128 / 16 : 2;
        constexpr int kXTerm = TURNED ? 64 * kStep * 2 : COLS * kStep * 2;
        const uint64_t wdesc = TURNED ? smem_desc_mn(ring, 64 * kStep * 2) : smem_desc64(ring);
        const uint64_t xdesc = TURNED ? smem_desc_mn(ring + G::kXAt, 3 * 64 * kStep * 2)
                                      : smem_desc64(ring + G::kXAt);
        int stage = 0, xstage = 0, acc = 0, in_run = 0;
        uint32_t phase = 0, xphase = 0, acc_phase = 0;
        while (c.u < a.units) {
            if (in_run == 0) {
                if (!bar_wait(tempty0 + 8 * acc, acc_phase ^ 1, abort_flag, a.status)) break;
                tc_fence_after();
            }
            if (!bar_wait(xfull0 + 8 * xstage, xphase, abort_flag, a.status) ||
                !bar_wait(ready0 + 8 * stage, phase, abort_flag, a.status))
                break;
            tc_fence_after();
            const uint32_t d = tmem + uint32_t(acc * 2 * COLS);
            const uint64_t w0 = wdesc + uint32_t(stage * G::kWBytes / 16);
            const uint64_t x0 = xdesc + uint32_t(xstage * G::kXBytes / 16);
            const int pieces = c.s + 1 == a.steps ? a.tail : 2;
#pragma unroll
            for (int i = 0; i < 3; ++i)
#pragma unroll
                for (int j = 0; j + i < 3; ++j)
#pragma unroll
                    for (int k = 0; k < 2; ++k) {
                        if (k >= pieces) break;
                        // the leading product into the first accumulator, the others into the
                        // second, whose first of a run is (0, 1)
                        const bool fresh = in_run == 0 && k == 0 && i == 0 && j <= 1;
                        mma<true>(d + (i + j > 0 ? COLS : 0),
                                  w0 + uint64_t(i * kTermBytes / 16) + kAdvance * k,
                                  x0 + uint64_t(j * kXTerm / 16) + kAdvance * k, idesc,
                                  fresh ? 0u : 1u);
                    }
            mma_commit(empty0 + 8 * stage);
            mma_commit(xempty0 + 8 * xstage);
            if (++stage == G::kWStages) {
                stage = 0;
                phase ^= 1;
            }
            if (++xstage == G::kXStages) {
                xstage = 0;
                xphase ^= 1;
            }
            const bool last = c.s + 1 == c.s1;
            if (++in_run == kRun32 || last) {
                mma_commit(tfull0 + 8 * acc);
                in_run = 0;
                if (++acc == 2) {
                    acc = 0;
                    acc_phase ^= 1;
                }
            }
            advance(a, c);
        }
        if (*abort_flag) {  // every MMA issued so far completes before TMEM is freed
            mma_commit(drain);
            const unsigned long long t0 = now_ns();
            while (!bar_test(drain, 0))
                if (now_ns() - t0 > kTcWaitLimitNs) break;
        }
    } else if (warp >= 2 && warp < 2 + kSplitWarps) {
        // ---- the matrix, copied ahead and split into terms ----
        const int group = (warp - 2) / kGroup, mine = (warp - 2) % kGroup;
        const uint32_t raw = ring + G::kRawAt + (warp - 2) * G::kDepth * kSlot;
        auto fetch = [&](const Cursor& f, uint32_t slot) {
            if (f.u < a.units) {
                if constexpr (TURNED) {  // eight rows of K, 128 columns
                    const int64_t row0 = int64_t(f.s) * kStep + 8 * mine, col0 = int64_t(f.mt) * kRows32;
                    const int rows = a.w_rows - row0 < 8 ? int(a.w_rows - row0) : 8;
                    const float* src = a.w + row0 * a.stride + col0;
                    const int cols = a.width - col0 < 128 ? int(a.width - col0) : 128;
                    if (a.vec) {
                        const int left = (cols - 4 * lane) * 4, most = max(0, min(left, 16));
                        src += 4 * lane;
#pragma unroll
                        for (int r = 0; r < 8; ++r, src += a.stride) {
                            const int bytes = r < rows ? most : 0;
                            copy16(slot + r * 512 + lane * 16, bytes ? src : a.w, bytes);
                        }
                    } else {
                        src += lane;
#pragma unroll
                        for (int r = 0; r < 8; ++r, src += a.stride)
#pragma unroll
                            for (int k = 0; k < 4; ++k) {
                                const bool ok = r < rows && 32 * k + lane < cols;
                                copy4(slot + r * 512 + (32 * k + lane) * 4, ok ? src + 32 * k : a.w,
                                      ok ? 4 : 0);
                            }
                    }
                } else {  // 32 rows of 32 elements of K, 16-byte pieces c at c ^ (row % 8)
                    const int64_t row0 = int64_t(f.mt) * kRows32 + 32 * mine, col0 = int64_t(f.s) * kStep;
                    const int64_t left_rows = a.w_rows - row0;
                    const int rows = left_rows < 32 ? int(left_rows) : 32;  // (may be none)
                    const float* src = a.w + row0 * a.stride + col0;
                    if (a.vec) {
                        const int piece = lane & 7;
                        const int64_t left = (a.width - col0 - 4 * piece) * 4;
                        const int most = left > 0 ? int(min(left, int64_t(16))) : 0;
                        src += (lane >> 3) * a.stride + 4 * piece;
#pragma unroll
                        for (int k = 0; k < 8; ++k, src += 4 * a.stride) {
                            const int r = (lane >> 3) + 4 * k;
                            const int bytes = r < rows ? most : 0;
                            copy16(slot + r * 128 + ((piece ^ (r & 7)) * 16), bytes ? src : a.w, bytes);
                        }
                    } else {
                        const int most = col0 + lane < a.width ? rows : 0;
                        src += lane;
#pragma unroll
                        for (int r = 0; r < 32; ++r, src += a.stride) {
                            const bool ok = r < most;
                            copy4(slot + r * 128 + ((lane * 4) ^ ((r & 7) << 4)), ok ? src : a.w, ok ? 4 : 0);
                        }
                    }
                }
            }
            asm volatile("cp.async.commit_group;" ::: "memory");
        };
        auto skip = [&](Cursor& f) {  // the other group's step
            if (f.u < a.units) advance(a, f);
        };
        if (group == 1) skip(c);
        Cursor ahead = c;
        for (int k = 0; k < G::kDepth; ++k) {
            fetch(ahead, raw + k * kSlot);
            skip(ahead);
            skip(ahead);
        }
        int stage = group, slot = 0;
        uint32_t phase = 0;
        while (c.u < a.units) {
            asm volatile("cp.async.wait_group %0;" ::"n"(G::kDepth - 1) : "memory");
            __syncwarp();
            const bool ok = bar_wait(empty0 + 8 * stage, phase ^ 1, abort_flag, a.status);
            if (!__all_sync(0xffffffffu, ok)) break;
            const uint32_t from = raw + slot * kSlot, to = ring + stage * G::kWBytes;
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                float v[8];
                if constexpr (TURNED) {
                    const int r = (lane >> 4) + 2 * k, octet = lane & 15, kr = 8 * mine + r;
                    lds4(from + r * 512 + octet * 32, v);
                    lds4(from + r * 512 + octet * 32 + 16, v + 4);
                    split8(v, to + (octet >> 3) * 64 * kStep * 2 + kr * 128 + (((octet & 7) ^ (kr & 7)) * 16));
                } else {
                    const int R = 32 * mine + lane;
                    lds4(from + lane * 128 + (((2 * k) ^ (lane & 7)) * 16), v);
                    lds4(from + lane * 128 + (((2 * k + 1) ^ (lane & 7)) * 16), v + 4);
                    split8(v, to + R * 64 + ((k ^ ((R >> 1) & 3)) * 16));
                }
            }
            fence_async_smem();
            __syncwarp();  // (and the slot is read: it may be filled again)
            if (lane == 0) bar_arrive(ready0 + 8 * stage);
            fetch(ahead, from);
            skip(ahead);
            skip(ahead);
            if (++slot == G::kDepth) slot = 0;
            stage += 2;
            if (stage >= G::kWStages) {
                stage -= G::kWStages;
                phase ^= 1;
            }
            skip(c);
            skip(c);
        }
        asm volatile("cp.async.wait_all;" ::: "memory");
    } else if (warp >= 2 + kSplitWarps) {
        // ---- epilogue ----
        const int quarter = warp & 3, part = (warp - 2 - kSplitWarps) >> 2;
        constexpr int kPart = COLS / 2;
        GradRow* few_rows = reinterpret_cast<GradRow*>(smem + G::kRowsAt);
        if constexpr (EPI == kTileGradFew) {
            const int i = threadIdx.x - 32 * (2 + kSplitWarps);
            if (i < a.N) few_rows[i] = grad_row(a.o, i, a.M);
            asm volatile("bar.sync 1, 256;" ::: "memory");
        }
        int acc = 0;
        uint32_t acc_phase = 0;
        bool ok = true;
        for (; c.u < a.units && ok;) {
            const int64_t row0 = int64_t(c.mt) * kRows32 + quarter * 32, row = row0 + lane;
            const int64_t col0 = part * kPart;
            const bool in = row < a.M, work = row0 < a.M && col0 < a.N;
            float sum[kPart];
            const int split = c.u / a.m_tiles;
            for (int s = c.s; s < c.s1; s += kRun32) {
                ok = bar_wait(tfull0 + 8 * acc, acc_phase, abort_flag, a.status);
                ok = __all_sync(0xffffffffu, ok);
                if (!ok) break;
                tc_fence_after();
                if (work) {
                    const uint32_t at =
                        tmem + (uint32_t(quarter * 32) << 16) + uint32_t(acc * 2 * COLS + col0);
#pragma unroll
                    for (int k = 0; k < kPart; k += 16) {
                        float v[16];
                        tmem_ld16(at + k, v);
#pragma unroll
                        for (int i = 0; i < 16; ++i) sum[k + i] = s == c.s ? v[i] : sum[k + i] + v[i];
                        tmem_ld16(at + COLS + k, v);
#pragma unroll
                        for (int i = 0; i < 16; ++i) sum[k + i] += v[i];
                    }
                }
                tc_fence_before();
                __syncwarp();
                if (lane == 0) bar_arrive(tempty0 + 8 * acc);
                if (++acc == 2) {
                    acc = 0;
                    acc_phase ^= 1;
                }
            }
            if (!ok) break;
            if (work) {
#pragma unroll
                for (int k = 0; k < kPart; k += 32) {
                    if (col0 + k >= a.N) break;
                    float* v = sum + k;
                    if constexpr (EPI == kTileStatsFew) {
                        few_stats(a.o, a.M, a.N, v, row0, col0 + k, in, lane);
                    } else if constexpr (EPI == kTileGradFew) {
                        few_grad(a.o, a.N, few_rows + col0 + k, v, row, col0 + k, in);
                    } else if (in) {  // (rows of whole groups of eight)
                        float* y = a.o.part + (int64_t(split) * a.M + row) * a.o.part_ld + col0 + k;
#pragma unroll
                        for (int i = 0; i < 32; i += 4) {
                            if (col0 + k + i >= a.o.part_ld) break;
                            float4 x = make_float4(v[i], v[i + 1], v[i + 2], v[i + 3]);
                            if (a.o.add) {
                                const float4 z = *reinterpret_cast<const float4*>(y + i);
                                x.x += z.x, x.y += z.y, x.z += z.z, x.w += z.w;
                            }
                            *reinterpret_cast<float4*>(y + i) = x;
                        }
                    }
                }
            }
            c.u += gridDim.x;
            if (c.u < a.units) enter(a, c);
        }
    }
    __syncwarp();
    tc_fence_before();
    __syncthreads();
    if (warp == 1) {
        tc_fence_after();
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, 512;" ::"r"(tmem) : "memory");
    }
}

template <bool TURNED, int EPI, int COLS>
cudaError_t launch32(const Args32& a, int dev, int sms, cudaStream_t s) {
    static std::atomic<uint64_t> allowed{0};
    auto* kernel = f32_kernel<TURNED, EPI, COLS>;
    cudaError_t ce = allow_shared(reinterpret_cast<const void*>(kernel), dev, allowed);
    if (ce != cudaSuccess) return ce;
    cudaLaunchConfig_t cfg;
    std::memset(&cfg, 0, sizeof cfg);
    cfg.gridDim = dim3(std::min(a.units, sms));
    cfg.blockDim = dim3(kF32Threads);
    cfg.dynamicSmemBytes = Geo32<COLS>::kSmem;
    cfg.stream = s;
    cudaLaunchAttribute at[1];
    at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = at;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kernel, a);
}

template <int COLS>
cudaError_t launch32_any(const Args32& a, TileEpilogue epi, int dev, int sms, cudaStream_t s) {
    switch (epi) {
        case kTileStatsFew: return launch32<false, kTileStatsFew, COLS>(a, dev, sms, s);
        case kTileGradFew: return launch32<false, kTileGradFew, COLS>(a, dev, sms, s);
        default: return launch32<true, kTileOut, COLS>(a, dev, sms, s);
    }
}

}  // namespace
}  // namespace tc

int few32_product(const char* fn, const Few32Product& p, TileEpilogue epilogue, int sms,
                  cudaStream_t stream) {
    using namespace tc;
    Args32 a;
    std::memset(&a, 0, sizeof a);
    int dev = 0;
    cudaError_t ce = cudaGetDevice(&dev);
    if (ce == cudaSuccess) ce = operators_status(dev, &a.status);
    if (ce != cudaSuccess) return record_error(CAM_E_CUDA, "%s: %s", fn, cudaGetErrorString(ce));
    const int cols = p.b.rows <= 64 ? 64 : 128;
    const TileOperand& b = p.b;
    const CUtensorMapDataType bf = CU_TENSOR_MAP_DATA_TYPE_BFLOAT16;
    const bool ok =
        p.turned ? encode(&a.tx, bf, b.base, b.rows, b.k, 3, b.ld * 2, b.plane_stride * 2, 64, kStep,
                          CU_TENSOR_MAP_SWIZZLE_128B, 3)
                 : encode(&a.tx, bf, b.base, b.k, b.rows, 3, b.ld * 2, b.plane_stride * 2, kStep, cols,
                          CU_TENSOR_MAP_SWIZZLE_64B, 3);
    if (!ok) return record_error(CAM_E_CUDA, "%s: cuTensorMapEncodeTiled failed", fn);
    a.w = p.w;
    a.w_rows = p.w_rows;
    a.width = p.width;
    a.stride = p.w_stride;
    a.vec = reinterpret_cast<uintptr_t>(p.w) % 16 == 0 && p.w_stride % 4 == 0;
    a.M = p.turned ? p.width : p.w_rows;
    a.N = b.rows;
    const int64_t K = p.turned ? p.w_rows : p.width;
    a.m_tiles = static_cast<int32_t>((a.M + kRows32 - 1) / kRows32);
    a.steps = static_cast<int32_t>((K + kStep - 1) / kStep);
    a.tail = K - int64_t(a.steps - 1) * kStep > 16 ? 2 : 1;
    const int splits = std::max(1, std::min(p.splits, a.steps));
    a.per_split = (a.steps + splits - 1) / splits;
    a.units = a.m_tiles * ((a.steps + a.per_split - 1) / a.per_split);
    a.o = p.out;
    ce = cols == 64 ? launch32_any<64>(a, epilogue, dev, sms, stream)
                    : launch32_any<128>(a, epilogue, dev, sms, stream);
    if (ce != cudaSuccess)
        return record_error(CAM_E_CUDA, "%s: launch: %s", fn, cudaGetErrorString(ce));
    return CAM_OK;
}

}  // namespace cam
