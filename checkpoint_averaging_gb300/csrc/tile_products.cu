// tile_products.cu -- the kernel behind tile_products.h.
//
// A persistent grid, one block per SM or one pair of blocks (a cluster of two) per pair of
// SMs; unit u of the launch (a tile of one product, or one K range of it) goes to block
// (pair) u, u + grid, ... Warps with fixed roles:
//
//   warp 0 (one lane)  TMA producer: per K step of 128 bytes, this SM's 128 rows of A
//                    and its share of B (the tile's columns, or half of them in a
//                    pair) into a ring of shared-memory stages;
//   warp 1 (one lane)  MMA issuer (of a pair: the first block's): four tcgen05.mma
//                    of 32 bytes of K per stage into one of two TMEM accumulators;
//                    e4m3 operands' scales go from the stage into TMEM first
//                    (tcgen05.cp) and are applied by the tensor core;
//   warps 2..        epilogue, 16 or 8: TMEM lanes 32 (warp % 4) .. + 31, each four of
//                    them a part of the columns. A thread holds its part of one row of the
//                    tile in registers.
//
// A pair of SMs works on one 256-row tile (cta_group::2): each stages its own rows of A
// and half of B's columns, so an SM fetches 32 KB per 128 x 256 x 64 products
// instead of 48.
//
// The tensor core adds to its accumulator without rounding to nearest: what is lost grows
// with the number of additions and leans to zero. Where that would show in the result (fp32
// results of long rows) the sum is cut into runs of K steps, each accumulated in TMEM and
// added to the thread's registers in fp32.
//
// Every mbarrier wait is bounded; one that runs out sets CAM_STATUS_GEMM_TIMEOUT in the
// library's status word (cam_operators_status) and an abort flag of the block. Every role
// then leaves its loop, the producer waits (bounded) for its copies, the issuer for its
// MMAs, and the TMEM is freed.
#include "tile_products.h"

#include <cuda_bf16.h>

#include <algorithm>
#include <atomic>
#include <cstring>

#include "cam_internal.h"
#include "op_launch.h"
#include "tc_device.cuh"
#include "tile_device.cuh"

#define CAM_API extern "C" __attribute__((visibility("default")))

namespace cam {
namespace tc {
namespace {

__device__ int32_t g_status;

constexpr int kRows = 128;       // TMEM lanes: rows of an SM's tile
constexpr int kStepBytes = 128;  // bytes of K per stage
constexpr int kMnBox = 64 * kStepBytes;  // MN-major box: 64 K rows of 64 elements
constexpr int kShared = 226 * 1024;  // for the ring and the epilogue's buffers
struct alignas(128) Prob {
    CUtensorMap ta, tb;    // operands
    CUtensorMap tsa, tsb;  // e4m3: their scales
    CUtensorMap ty;        // results: boxes of 64 bytes by 32 rows
    int32_t m_tiles, n_tiles, m_fast;
    int32_t steps;         // K steps of one pair of terms
    int32_t tail;          // 32-byte pieces of the last of them
    int32_t pairs;         // of terms
    int32_t per_split;     // K steps of a unit's range
    int32_t run;           // K steps that are accumulated in TMEM, every pair's
    int32_t a_mn, b_mn;
    int32_t unit0;
    int32_t boxes;         // results go through ty
    uint32_t terms_a, terms_b;  // the terms of each pair, four bits each
    int64_t M, N;
    TileOut o;
};

struct alignas(128) Args {
    Prob prob[2];
    int32_t n_prob, n_units;
};

template <bool E4M3, bool PAIR, int EPI, int COLS>
struct Geo {
    static constexpr int kCols = COLS;
    // Warps of the epilogue: 16 where each has 64 columns of a quarter of the rows then
    // (two per scheduler do not cover their own latencies), 8 for narrower tiles. 18 warps leave 96
    // registers a thread: 136 bytes of stores and 156 of loads are spilled for results, 84 and 104 for
    // G, 12 and 12 for the statistics.
    static constexpr int kWarps = COLS == kTileCols ? 16 : 8;
    static constexpr int kThreads = 64 + 32 * kWarps;
    static constexpr int kParts = kWarps / 4;      // of a tile's columns
    static constexpr int kPart = COLS / kParts;
    // buffers: results, the parts' statistics of three tiles, few rows' data
    static constexpr int kOutBytes = EPI == kTileStats   ? 3 * 32 * kWarps * 16
                                     : EPI == kTileStatsFew ? 0
                                     : EPI == kTileGradFew  ? 4096
                                                            : kWarps * 2 * kBox;
    static constexpr int kRing = kShared - kOutBytes - 1024;
    static constexpr int kBCols = PAIR ? kCols / 2 : kCols;  // B rows an SM stages
    static constexpr int kABytes = kRows * kStepBytes;
    static constexpr int kBBytes = kBCols * kStepBytes;
    static constexpr int kScaleA = E4M3 ? 512 : 0;   // one block of 128 rows
    static constexpr int kScaleB = E4M3 ? 1024 : 0;  // two blocks cover 192 columns
    static constexpr int kTx = kABytes + kBBytes + kScaleA + kScaleB;
    static constexpr int kStage = (kTx + 1023) / 1024 * 1024;
    static constexpr int kStages = kRing / kStage < 8 ? kRing / kStage : 8;
    static constexpr int kBars = 2 * kStages + 5 + 12;
    static constexpr int kOutAt = kStages * kStage;
    static constexpr int kBarsAt = kOutAt + kOutBytes;
    static constexpr int kSmem = kBarsAt + 8 * kBars + 16 + 1024;
    static_assert(kSmem <= kMaxSharedBytes, "over the per-block shared memory limit");
};

constexpr int kScaleColumn = 2 * kTileCols8;  // TMEM column of the scales

// ---- what a pair of blocks adds to tc_device.cuh --------------------------------------

__device__ __forceinline__ uint32_t cluster_rank() {
    uint32_t r;
    asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
    return r;
}
__device__ __forceinline__ void cluster_sync() {
    asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
    asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
}
// The address of the first block's copy of a shared variable.
__device__ __forceinline__ uint32_t first_block(uint32_t addr) {
    uint32_t r;
    asm volatile("mapa.shared::cluster.u32 %0, %1, 0;" : "=r"(r) : "r"(addr));
    return r;
}
__device__ __forceinline__ void bar_arrive_cluster(uint32_t bar) {
    asm volatile("mbarrier.arrive.release.cluster.shared::cluster.b64 _, [%0];" ::"r"(bar)
                 : "memory");
}

// The load of a pair: `bar` may be the other block's.
template <bool PAIR>
__device__ __forceinline__ void load(uint32_t dst, const CUtensorMap* map, int x, int y, int z,
                                     uint32_t bar) {
    if constexpr (PAIR)
        asm volatile(
            "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
            ".cta_group::2 [%0], [%1, {%2, %3, %4}], [%5];" ::"r"(dst),
            "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(z), "r"(bar)
            : "memory");
    else
        tma_load(dst, map, x, y, z, bar);
}

template <bool PAIR>
__device__ __forceinline__ void commit(uint32_t bar) {
    if constexpr (PAIR)
        asm volatile(
            "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster"
            ".multicast::cluster.b64 [%0], %1;" ::"r"(bar),
            "h"(static_cast<uint16_t>(3))
            : "memory");
    else
        mma_commit(bar);
}

// Instruction descriptors: fp32 accumulator; bf16 operands (formats 1, majorness in bits
// 15 and 16), or e4m3 operands (formats 0) with one UE8M0 scale per 32 elements of K (bit
// 23), scale bytes 0 of their words. N / 8 in bits 17-22, M / 16 in bits 24-28.
template <bool E4M3, bool PAIR, int COLS>
__device__ __forceinline__ uint32_t instruction(uint32_t a_mn, uint32_t b_mn) {
    constexpr uint32_t n = COLS >> 3, m = (PAIR ? 256 : 128) >> 4;
    if constexpr (E4M3)
        return (n << 17) | (1u << 23) | (m << 24);
    else
        return (1u << 4) | (1u << 7) | (1u << 10) | (a_mn << 15) | (b_mn << 16) | (n << 17) |
               (m << 24);
}

template <bool E4M3, bool PAIR>
__device__ __forceinline__ void multiply(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc,
                                         uint32_t accumulate, uint32_t sa, uint32_t sb) {
    if constexpr (E4M3 && PAIR)
        asm volatile(
            "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
            "tcgen05.mma.cta_group::2.kind::mxf8f6f4.block_scale [%0], %1, %2, %3, [%5], [%6], "
            "p;\n\t}" ::"r"(d),
            "l"(a), "l"(b), "r"(idesc), "r"(accumulate), "r"(sa), "r"(sb)
            : "memory");
    else if constexpr (E4M3)
        asm volatile(
            "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
            "tcgen05.mma.cta_group::1.kind::mxf8f6f4.block_scale [%0], %1, %2, %3, [%5], [%6], "
            "p;\n\t}" ::"r"(d),
            "l"(a), "l"(b), "r"(idesc), "r"(accumulate), "r"(sa), "r"(sb)
            : "memory");
    else if constexpr (PAIR)
        asm volatile(
            "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
            "tcgen05.mma.cta_group::2.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
            "l"(a), "l"(b), "r"(idesc), "r"(accumulate)
            : "memory");
    else
        mma<true>(d, a, b, idesc, accumulate);
}

// 128 rows' scales (32 lanes of 16 bytes) into four TMEM columns, for every quarter of lanes.
template <bool PAIR>
__device__ __forceinline__ void copy_scales(uint32_t taddr, uint32_t smem) {
    // no swizzle, 8 x 16-byte core matrices 128 bytes apart
    const uint64_t desc = static_cast<uint64_t>((smem & 0x3FFFFu) >> 4) | (uint64_t(8) << 16) |
                          (uint64_t(8) << 32) | (uint64_t(1) << 46);
    if constexpr (PAIR)
        asm volatile("tcgen05.cp.cta_group::2.32x128b.warpx4 [%0], %1;" ::"r"(taddr), "l"(desc)
                     : "memory");
    else
        asm volatile("tcgen05.cp.cta_group::1.32x128b.warpx4 [%0], %1;" ::"r"(taddr), "l"(desc)
                     : "memory");
}

// ---- units -----------------------------------------------------------------------------

struct Unit {
    int p, mt, nt, split;
    int k0, k1;  // K steps
};

__device__ __forceinline__ Unit unit_of(const Args& a, int u) {
    Unit t;
    t.p = a.n_prob > 1 && u >= a.prob[1].unit0 ? 1 : 0;
    const Prob& P = a.prob[t.p];
    u -= P.unit0;
    const int per = P.m_tiles * P.n_tiles;
    t.split = u / per;
    u -= t.split * per;
    if (P.m_fast) {
        t.nt = u / P.m_tiles;
        t.mt = u - t.nt * P.m_tiles;
    } else {
        t.mt = u / P.n_tiles;
        t.nt = u - t.mt * P.n_tiles;
    }
    t.k0 = t.split * P.per_split;
    t.k1 = min(P.steps, t.k0 + P.per_split);
    return t;
}

// ---- the kernel ------------------------------------------------------------------------

template <bool E4M3, bool PAIR, int EPI, int COLS>
__global__ void __launch_bounds__(Geo<E4M3, PAIR, EPI, COLS>::kThreads, 1)
    tile_kernel(const __grid_constant__ Args a) {
    using G = Geo<E4M3, PAIR, EPI, COLS>;
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>(
        (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    uint64_t* bars = reinterpret_cast<uint64_t*>(smem + G::kBarsAt);
    const uint32_t full0 = su32(bars);
    const uint32_t empty0 = full0 + 8 * G::kStages;
    const uint32_t tfull0 = empty0 + 8 * G::kStages;
    const uint32_t tempty0 = tfull0 + 16;
    const uint32_t drain = tempty0 + 16;
    const uint32_t parts0 = drain + 8;  // kTileStats: of each quarter of rows, of three tiles
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(bars + G::kBars);
    volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
    int32_t* status = &g_status;
    const int warp = __shfl_sync(0xffffffffu, int(threadIdx.x >> 5), 0), lane = threadIdx.x & 31;
    const uint32_t rank = PAIR ? cluster_rank() : 0;
    const int worker = PAIR ? int(blockIdx.x >> 1) : int(blockIdx.x);
    const int workers = PAIR ? int(gridDim.x >> 1) : int(gridDim.x);

    if (threadIdx.x == 0) {
        for (int s = 0; s < G::kStages; ++s) {
            bar_init(full0 + 8 * s, 1);
            bar_init(empty0 + 8 * s, 1);
        }
        for (int i = 0; i < 2; ++i) {
            bar_init(tfull0 + 8 * i, 1);
            bar_init(tempty0 + 8 * i, (PAIR ? 2 : 1) * G::kWarps);
        }
        bar_init(drain, 1);
        for (int i = 0; i < 12; ++i) bar_init(parts0 + 8 * i, G::kParts > 1 ? G::kParts - 1 : 1);
        *abort_flag = 0;
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    if (warp == 1) {
        if constexpr (PAIR) {
            asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], 512;" ::"r"(
                             su32(tmem_slot))
                         : "memory");
            asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
        } else {
            asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], 512;" ::"r"(
                             su32(tmem_slot))
                         : "memory");
            asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
        }
    }
    tc_fence_before();
    __syncthreads();
    if constexpr (PAIR) cluster_sync();
    tc_fence_after();
    const uint32_t tmem = *tmem_slot;
    // a programmatic dependent of the kernel before it: set-up overlapped that kernel's end
    asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");

    if (warp == 0 && elect_one()) {
        // ---- producer ----
        const uint32_t ring = su32(smem);
        const uint32_t to_full0 = PAIR ? first_block(full0) : full0;
        int stage = 0;
        uint32_t phase = 0, issued = 0, filled_parity = 0;
        bool ok = true;
        for (int u = worker; u < a.n_units && ok; u += workers) {
            const Unit t = unit_of(a, u);
            const Prob& P = a.prob[t.p];
            const int arow = (t.mt * (PAIR ? 2 : 1) + int(rank)) * kRows;
            const int bcol = t.nt * G::kCols, brow = bcol + int(rank) * G::kBCols;
            const int k1 = t.k1, run = P.run, pairs = P.pairs;
            const bool a_mn = P.a_mn, b_mn = P.b_mn;
            const CUtensorMap *ta = &P.ta, *tb = &P.tb;
            int pair = 0, ks = t.k0, za = P.terms_a & 15, zb = P.terms_b & 15;
            int from = ks, to = min(k1 - from, run) + from;  // the run
            while (from < k1) {
                if (!bar_wait(empty0 + 8 * stage, phase ^ 1, abort_flag, status)) {
                    ok = false;
                    break;
                }
                const uint32_t sa = ring + stage * G::kStage, sb = sa + G::kABytes;
                const uint32_t fb = to_full0 + 8 * stage;
                if (rank == 0) bar_expect(full0 + 8 * stage, (PAIR ? 2 : 1) * G::kTx);
                if constexpr (E4M3) {
                    const int x = ks * kStepBytes;
                    load<PAIR>(sa, ta, x, arow, 0, fb);
                    load<PAIR>(sb, tb, x, brow, 0, fb);
                    const uint32_t ss = sb + G::kBBytes;
                    load<PAIR>(ss, &P.tsa, 0, arow / 128, ks, fb);
                    load<PAIR>(ss + G::kScaleA, &P.tsb, 0, bcol / 128, ks, fb);
                } else {
                    const int x = ks * 64;
                    if (a_mn) {
#pragma unroll
                        for (int i = 0; i < kRows / 64; ++i)
                            load<PAIR>(sa + i * kMnBox, ta, arow + 64 * i, x, za, fb);
                    } else {
                        load<PAIR>(sa, ta, x, arow, za, fb);
                    }
                    if (b_mn) {
#pragma unroll
                        for (int i = 0; i < G::kBCols / 64; ++i)
                            load<PAIR>(sb + i * kMnBox, tb, brow + 64 * i, x, zb, fb);
                    } else {
                        load<PAIR>(sb, tb, x, brow, zb, fb);
                    }
                }
                issued |= 1u << stage;
                filled_parity = (filled_parity & ~(1u << stage)) | (phase << stage);
                if (++stage == G::kStages) {
                    stage = 0;
                    phase ^= 1;
                }
                if (++ks == to) {
                    if (++pair == pairs) {
                        pair = 0;
                        from = to;
                        to = min(k1 - from, run) + from;
                    }
                    ks = from;
                    za = P.terms_a >> (4 * pair) & 15;
                    zb = P.terms_b >> (4 * pair) & 15;
                }
            }
        }
        if (*abort_flag && rank == 0) {  // let the copies in flight land
            for (int s = 0; s < G::kStages; ++s)
                if ((issued >> s) & 1) {
                    const unsigned long long t0 = now_ns();
                    while (!bar_test(full0 + 8 * s, (filled_parity >> s) & 1))
                        if (now_ns() - t0 > kTcWaitLimitNs) break;
                }
        }
    } else if (warp == 1 && rank == 0 && elect_one()) {
        // ---- MMA issuer ----
        const uint32_t ring = su32(smem);
        int stage = 0, acc = 0;
        uint32_t phase = 0, acc_phase = 0;
        uint32_t scale_at = 0;
        bool ok = true;
        for (int u = worker; u < a.n_units && ok; u += workers) {
            const Unit t = unit_of(a, u);
            const Prob& P = a.prob[t.p];
            const uint32_t idesc = instruction<E4M3, PAIR, COLS>(P.a_mn, P.b_mn);
            // 32 bytes further along a K-major row, or 16 rows further down an MN-major box
            const uint64_t step_a = P.a_mn ? 16 * kStepBytes / 16 : 2;
            const uint64_t step_b = P.b_mn ? 16 * kStepBytes / 16 : 2;
            const uint64_t desc_a = P.a_mn ? smem_desc_mn(ring, kMnBox) : smem_desc(ring);
            const uint64_t desc_b = P.b_mn ? smem_desc_mn(ring, kMnBox) : smem_desc(ring);
            const int last = P.steps - 1, tail = P.tail, k1 = t.k1, run = P.run, pairs = P.pairs;
            for (int from = t.k0; from < k1 && ok;) {
                const int to = min(k1 - from, run) + from;
                if (!bar_wait(tempty0 + 8 * acc, acc_phase ^ 1, abort_flag, status)) {
                    ok = false;
                    break;
                }
                tc_fence_after();
                const uint32_t d = tmem + uint32_t(acc * G::kCols);
                uint32_t accumulate = 0;
                int ks = from;
                for (int left = (to - from) * pairs; left > 0; --left) {
                    if (!bar_wait(full0 + 8 * stage, phase, abort_flag, status)) {
                        ok = false;
                        break;
                    }
                    tc_fence_after();
                    // (addresses below 256 KB: no carry out of the descriptors' field)
                    const uint64_t da = desc_a + uint32_t(stage * G::kStage / 16);
                    const uint64_t db = desc_b + uint32_t((stage * G::kStage + G::kABytes) / 16);
                    uint32_t ta = 0, tb = 0;
                    if constexpr (E4M3) {
                        // four columns of A's scales, eight of B's; a tile that starts in the
                        // middle of a block of 128 starts two columns into them
                        ta = tmem + kScaleColumn + scale_at;
                        tb = ta + 4;
                        const uint32_t ss = ring + stage * G::kStage + G::kABytes + G::kBBytes;
                        copy_scales<PAIR>(ta, ss);
                        copy_scales<PAIR>(tb, ss + 512);
                        copy_scales<PAIR>(tb + 4, ss + 1024);
                        tb += (t.nt & 1) ? 2 : 0;
                        scale_at ^= 16;
                    }
                    const int pieces = ks == last ? tail : kStepBytes / 32;
                    if (++ks == to) ks = from;
#pragma unroll
                    for (int k = 0; k < kStepBytes / 32; ++k) {
                        if (k >= pieces) break;
                        multiply<E4M3, PAIR>(d, da + step_a * k, db + step_b * k,
                                             idesc, accumulate, ta, tb);
                        accumulate = 1;
                    }
                    commit<PAIR>(empty0 + 8 * stage);
                    if (++stage == G::kStages) {
                        stage = 0;
                        phase ^= 1;
                    }
                }
                if (!ok) break;
                from = to;
                commit<PAIR>(tfull0 + 8 * acc);
                if (++acc == 2) {
                    acc = 0;
                    acc_phase ^= 1;
                }
            }
        }
        if (*abort_flag) {  // every MMA issued so far completes before TMEM is freed
            commit<PAIR>(drain);
            const unsigned long long t0 = now_ns();
            while (!bar_test(drain, 0))
                if (now_ns() - t0 > kTcWaitLimitNs) break;
        }
    } else if (warp >= 2) {
        // ---- epilogue ----
        const int quarter = warp & 3, part = (warp - 2) >> 2;
        uint8_t* out_at = smem + G::kOutAt + (warp - 2) * 2 * kBox;
        const uint32_t out_buf = su32(out_at);
        float* turn = reinterpret_cast<float*>(out_at);
        int which = 0, turn_of = 0;
        uint32_t turn_phase = 0;
        constexpr int kPart = G::kPart, kGroups = kPart / 32;
        int acc = 0;
        uint32_t acc_phase = 0;
        bool ok = true;
        GradRow* few_rows = reinterpret_cast<GradRow*>(smem + G::kOutAt);
        if constexpr (EPI == kTileGradFew) {  // the rows' data, for every thread of the epilogue
            const int i = threadIdx.x - 64;
            if (i < a.prob[0].N) few_rows[i] = grad_row(a.prob[0].o, i, a.prob[0].M);
            asm volatile("bar.sync 1, 256;" ::: "memory");
        }
        for (int u = worker; u < a.n_units && ok; u += workers) {
            const Unit t = unit_of(a, u);
            const Prob& P = a.prob[t.p];
            const TileOut& o = P.o;
            const int64_t row0 =
                int64_t(t.mt * (PAIR ? 2 : 1) + int(rank)) * kRows + quarter * 32;
            const int64_t row = row0 + lane;
            const int64_t col0 = int64_t(t.nt) * G::kCols + part * kPart;
            const bool in = row < P.M;
            // what a row brings, asked for before its tile is done
            int64_t token = -1;  // its column in this product
            GradRow mine{};
            if constexpr (EPI == kTileStats) {
                if (in && o.tokens) token = o.tokens[row] - o.token0;
            }
            if constexpr (EPI == kTileGrad) {
                if (in) mine = grad_row(o, row, P.N);
            }
            const bool work = row0 < P.M && col0 < P.N;  // (of the warp)
            // the thread's part of the row, summed over the runs of K
            float sum[kPart];
            const int k1 = t.k1, run = P.run;
            for (int from = t.k0; from < k1;) {
                const bool first = from == t.k0;
                from += min(k1 - from, run);
                ok = bar_wait(tfull0 + 8 * acc, acc_phase, abort_flag, status);
                ok = __all_sync(0xffffffffu, ok);
                if (!ok) break;
                tc_fence_after();
                if (work) {
                    const uint32_t tbase = tmem + (uint32_t(quarter * 32) << 16) +
                                           uint32_t(acc * G::kCols + part * kPart);
                    if (first) {
#pragma unroll
                        for (int c = 0; c < kGroups; ++c) tmem_ld32(tbase + uint32_t(c * 32), sum + 32 * c);
                    } else {
#pragma unroll
                        for (int c = 0; c < kPart / 16; ++c) {
                            float v[16];
                            tmem_ld16(tbase + uint32_t(c * 16), v);
#pragma unroll
                            for (int i = 0; i < 16; ++i) sum[16 * c + i] += v[i];
                        }
                    }
                }
                // the accumulator is free for the run after the next
                tc_fence_before();
                __syncwarp();
                if (lane == 0) {
                    if constexpr (PAIR) bar_arrive_cluster(first_block(tempty0 + 8 * acc));
                    else bar_arrive(tempty0 + 8 * acc);
                }
                if (++acc == 2) {
                    acc = 0;
                    acc_phase ^= 1;
                }
            }
            if (!ok) break;
            if constexpr (EPI == kTileStats) {
                // Joined with the other parts' of these rows by the first. A part may be two
                // tiles ahead of it (the accumulators are handed back before this), hence three
                // buffers in turn with a barrier each.
                if (row0 >= P.M) continue;
                const uint32_t joined = parts0 + 8 * (3 * quarter + turn_of);
                TileStat* parts = reinterpret_cast<TileStat*>(smem + G::kOutAt) +
                                  turn_of * 32 * G::kWarps + quarter * 32 + lane;
                RowStat stat;
                stat.m = stat.a = stat.t = 0.0f;
                if (work) {
#pragma unroll
                    for (int c = 0; c < kGroups; ++c) {
                        const int64_t col = col0 + 32 * c;
                        if (col >= P.N) break;
                        const float* v = sum + 32 * c;
                        const int n = P.N - col < 32 ? int(P.N - col) : 32;
                        if (n == 32) stat.add(v, 32, c == 0);
                        else stat.add(v, n, c == 0);
                        const int64_t at = token - col;
                        if (in && at >= 0 && at < n) o.mine[row] = pick(v, at);
                    }
                }
                TileStat all{stat.m, stat.a, stat.t, work ? 1.0f : 0.0f};
                if (part > 0) {
                    parts[part * 128] = all;
                    __syncwarp();
                    if (lane == 0) bar_arrive(joined);
                } else {
                    ok = bar_wait(joined, turn_phase, abort_flag, status);
                    ok = __all_sync(0xffffffffu, ok);
                    if (!ok) break;
#pragma unroll
                    for (int k = 1; k < G::kParts; ++k) join(all, parts[k * 128]);
                    if (in) o.stats[int64_t(t.nt) * P.M + row] = all;
                }
                if (++turn_of == 3) {
                    turn_of = 0;
                    turn_phase ^= 1;
                }
                continue;
            }
            if (!work) continue;
            if constexpr (EPI == kTileStatsFew) {
                few_stats(o, P.M, P.N, sum, row0, col0, in, lane);
                continue;
            }
            if constexpr (EPI == kTileGradFew) {
                few_grad(o, P.N, few_rows + col0, sum, row, col0, in);
                continue;
            }
            if constexpr (EPI == kTileOut || EPI == kTileGrad)
#pragma unroll
            for (int c = 0; c < kGroups; ++c) {
                const int64_t col = col0 + 32 * c;
                if (col >= P.N) break;
                float* v = sum + 32 * c;
                const int n = P.N - col < 32 ? int(P.N - col) : 32;
                if constexpr (EPI == kTileGrad) {
                    if (__any_sync(0xffffffffu, mine.far != 0.0f)) {
#pragma unroll
                        for (int i = 0; i < 32; ++i) v[i] = near(v[i], mine);
                    }
                    int own = -1;  // the row's token, if it is among these
                    if (mine.token >= 0 && mine.token - int(col) >= 0 && mine.token - int(col) < 32) {
                        own = mine.token - int(col);
                        put(v, own, own_grad(pick(v, own), mine));
                    }
                    if (o.planes == 3) {
#pragma unroll
                        for (int i = 0; i < 32; ++i)
                            v[i] = own == i ? v[i] : other_grad<true>(v[i], mine);
                    } else {
#pragma unroll
                        for (int i = 0; i < 32; ++i)
                            v[i] = own == i ? v[i] : other_grad<false>(v[i], mine);
                    }
                    for (int k = 0; k < o.planes; ++k) {
                        store_bf16(&P.ty, out_buf, which, v, lane, int(col), int(row0), k);
                        if (k + 1 < o.planes) {
#pragma unroll
                            for (int i = 0; i < 32; ++i)
                                v[i] -= __bfloat162float(__float2bfloat16_rn(v[i]));
                        }
                    }
                } else if (P.boxes) {
                    if (o.y_bf16)
                        store_bf16(&P.ty, out_buf, which, v, lane, int(col), int(row0), 0);
                    else
                        store_f32(&P.ty, out_buf, which, v, n, lane, int(col), int(row0), t.split,
                                  o.add != 0);
                } else {
                    if (elect_one()) bulk_wait_read0();  // (boxes of the launch's other product)
                    const int rows = P.M - row0 < 32 ? int(P.M - row0) : 32;
                    const int64_t at = row0 * o.ldy + col;
                    if (o.y_bf16)
                        store_turned(turn, static_cast<__nv_bfloat16*>(o.y) + at, o.ldy, v, rows, n, lane);
                    else
                        store_turned(turn, static_cast<float*>(o.y) + at, o.ldy, v, rows, n, lane);
                }
            }
        }
        if (elect_one()) bulk_wait_all();  // stores done before the block (and its buffers) goes
    }
    __syncwarp();
    tc_fence_before();
    __syncthreads();
    if constexpr (PAIR) cluster_sync();  // (nothing of the other block's is in flight here)
    if (warp == 1) {
        tc_fence_after();
        if constexpr (PAIR)
            asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, 512;" ::"r"(tmem)
                         : "memory");
        else
            asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, 512;" ::"r"(tmem)
                         : "memory");
    }
}

// ---- host side --------------------------------------------------------------------------

// bf16 terms: boxes of 64 elements of K by `rows` rows, or MN-major of 64 rows by 64 of K.
bool operand_map(CUtensorMap* map, const TileOperand& o, int rows) {
    const CUtensorMapDataType bf = CU_TENSOR_MAP_DATA_TYPE_BFLOAT16;
    const CUtensorMapSwizzle sw = CU_TENSOR_MAP_SWIZZLE_128B;
    return o.mn_major
               ? encode(map, bf, o.base, o.rows, o.k, o.planes, o.ld * 2, o.plane_stride * 2, 64, 64, sw)
               : encode(map, bf, o.base, o.k, o.rows, o.planes, o.ld * 2, o.plane_stride * 2, 64, rows,
                        sw);
}

// e4m3: boxes of 128 columns by `rows` rows; scales: blocks of 128 words.
bool operand_map8(CUtensorMap* map, CUtensorMap* scales, const TileOperand& o, int rows, int blocks) {
    const int64_t row_blocks = (o.rows + 127) / 128, col_blocks = (o.k + 127) / 128;
    return encode(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, o.base, o.ld, o.rows, 1, o.ld, o.ld * o.rows,
                  kStepBytes, rows, CU_TENSOR_MAP_SWIZZLE_128B) &&
           encode(scales, CU_TENSOR_MAP_DATA_TYPE_UINT32, o.scales, 128, row_blocks, col_blocks, 512,
                  512 * row_blocks, 128, blocks, CU_TENSOR_MAP_SWIZZLE_NONE);
}

template <bool E4M3, bool PAIR, int EPI, int COLS>
cudaError_t launch(const Args& a, int sms, cudaStream_t s) {
    using G = Geo<E4M3, PAIR, EPI, COLS>;
    static std::atomic<uint64_t> allowed{0};
    auto* kernel = tile_kernel<E4M3, PAIR, EPI, COLS>;
    int dev = 0;
    cudaError_t ce = cudaGetDevice(&dev);
    if (ce == cudaSuccess) ce = allow_shared(reinterpret_cast<const void*>(kernel), dev, allowed);
    if (ce != cudaSuccess) return ce;
    cudaLaunchConfig_t cfg;
    std::memset(&cfg, 0, sizeof cfg);
    cfg.gridDim = dim3(PAIR ? 2 * std::min(a.n_units, sms / 2) : std::min(a.n_units, sms));
    cfg.blockDim = dim3(G::kThreads);
    cfg.dynamicSmemBytes = G::kSmem;
    cfg.stream = s;
    cudaLaunchAttribute at[2];
    at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[0].val.programmaticStreamSerializationAllowed = 1;
    at[1].id = cudaLaunchAttributeClusterDimension;
    at[1].val.clusterDim.x = PAIR ? 2 : 1;
    at[1].val.clusterDim.y = at[1].val.clusterDim.z = 1;
    cfg.attrs = at;
    cfg.numAttrs = PAIR ? 2 : 1;
    return cudaLaunchKernelEx(&cfg, kernel, a);
}

template <bool PAIR>
cudaError_t launch_any(const Args& a, bool e4m3, TileEpilogue epi, int cols, int sms, cudaStream_t s) {
    if (e4m3) return launch<true, PAIR, kTileOut, kTileCols8>(a, sms, s);
    switch (epi) {
        case kTileOut:
            return cols == kTileNarrow ? launch<false, PAIR, kTileOut, kTileNarrow>(a, sms, s)
                                       : launch<false, PAIR, kTileOut, kTileCols>(a, sms, s);
        case kTileStats: return launch<false, PAIR, kTileStats, kTileCols>(a, sms, s);
        case kTileGrad: return launch<false, PAIR, kTileGrad, kTileCols>(a, sms, s);
        case kTileStatsFew: return launch<false, false, kTileStatsFew, kTileFew>(a, sms, s);
        default: return launch<false, false, kTileGradFew, kTileFew>(a, sms, s);
    }
}

}  // namespace
}  // namespace tc

int tile_products(const char* fn, const TileProduct* ps, int n, bool e4m3, bool pair,
                  TileEpilogue epilogue, int sms, cudaStream_t stream) {
    using namespace tc;
    Args a;
    std::memset(&a, 0, sizeof a);
    const bool few = epilogue == kTileStatsFew || epilogue == kTileGradFew;
    if (few) pair = false;
    // (products of at most 128 columns: half of a wide tile would be of none)
    bool narrow = epilogue == kTileOut && !e4m3;
    for (int i = 0; i < n; ++i) narrow = narrow && ps[i].b.rows <= kTileNarrow;
    const int cols = e4m3 ? kTileCols8 : few ? kTileFew : narrow ? kTileNarrow : kTileCols;
    const int rows = tile_rows(pair);
    const int b_rows = pair ? cols / 2 : cols;
    int32_t units = 0;
    for (int i = 0; i < n; ++i) {
        const TileProduct& p = ps[i];
        Prob& P = a.prob[i];
        const bool ok = e4m3 ? operand_map8(&P.ta, &P.tsa, p.a, kRows, 1) &&
                                   operand_map8(&P.tb, &P.tsb, p.b, b_rows, 2)
                             : operand_map(&P.ta, p.a, kRows) && operand_map(&P.tb, p.b, b_rows);
        if (!ok) return record_error(CAM_E_CUDA, "%s: cuTensorMapEncodeTiled failed", fn);
        P.M = p.a.rows;
        P.N = p.b.rows;
        P.m_tiles = static_cast<int32_t>((P.M + rows - 1) / rows);
        P.n_tiles = static_cast<int32_t>((P.N + cols - 1) / cols);
        // tiles that run at once share the longer side's operand
        P.m_fast = P.m_tiles <= P.n_tiles;
        P.a_mn = p.a.mn_major;
        P.b_mn = p.b.mn_major;
        // Pairs of terms, smallest products first: the sums of the small ones round at their
        // own size. Of three terms each, those of 2^-24 and less of the whole are left out.
        int pairs = 0;
        for (int sum = std::min(2, p.a.planes + p.b.planes - 2); sum >= 0; --sum)
            for (int k = 0; k <= sum; ++k)
                if (k < p.a.planes && sum - k < p.b.planes) {
                    P.terms_a |= uint32_t(k) << (4 * pairs);
                    P.terms_b |= uint32_t(sum - k) << (4 * pairs++);
                }
        const int step = e4m3 ? 128 : 64;
        P.steps = static_cast<int32_t>((p.a.k + step - 1) / step);
        P.tail = static_cast<int32_t>((p.a.k - (P.steps - 1) * int64_t(step) + step / 4 - 1) / (step / 4));
        P.pairs = pairs;
        // Runs: of fp32 inputs 256 terms of each pair (all pairs of a run are close in time, so
        // that the terms' second and third reads come from L2; of 128 the logits' errors are 40 %
        // smaller and calls up to 5 % slower), of two-term G 512, of bf16 logits 768 (of 512: 3 %
        // slower; the gradients take the logits by the same sums as the statistics, as 1 - p of
        // a row's token is a difference between the two), of e4m3 2,048 (whose steps add twice as
        // many terms), of the gradients' one-term products 8,192: what 512 additions lose, 2^-15
        // of a sum at most, is hidden in bf16 results, but not what a sum over 2^18 rows loses
        // in one run.
        const bool logits = epilogue != kTileOut;
        P.run = pairs > 2 ? 4 : pairs == 2 ? 8 : e4m3 ? 16 : logits ? 12 : 128;
        const int splits = std::max(1, std::min(p.splits, P.steps));
        P.per_split = (P.steps + splits - 1) / splits;
        const int ranges = (P.steps + P.per_split - 1) / P.per_split;
        P.unit0 = units;
        if (epilogue == kTileOut || epilogue == kTileGrad) {
            const bool part = p.out.part != nullptr, bf16 = epilogue == kTileGrad || p.out.y_bf16;
            const int64_t size = bf16 ? 2 : 4, ld = part ? p.out.part_ld : p.out.ldy;
            const void* y = part ? p.out.part : p.out.y;
            const int64_t planes = part ? ranges
                                        : epilogue == kTileGrad ? p.out.planes : 1;
            const int64_t plane = epilogue == kTileGrad ? p.out.plane_stride : P.M * ld;
            // The tensor maps want rows that start on 16 bytes, and a box that a row ends in may
            // be written past the row's end (a bf16 row of 223 columns: the 224th, too): into a
            // workspace's padding, not into what a caller has beside the result.
            const bool own = part || epilogue == kTileGrad;
            P.boxes = reinterpret_cast<uintptr_t>(y) % 16 == 0 && ld * size % 16 == 0 &&
                      (own || P.N * size % 16 == 0);
            if (P.boxes &&
                !encode(&P.ty, bf16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT32,
                        y, P.N, P.M, planes, ld * size, plane * size, static_cast<int>(64 / size), 32,
                        CU_TENSOR_MAP_SWIZZLE_64B))
                return record_error(CAM_E_CUDA, "%s: cuTensorMapEncodeTiled failed", fn);
        }
        P.o = p.out;
        units += P.m_tiles * P.n_tiles * ranges;
    }
    a.n_prob = n;
    a.n_units = units;
    const cudaError_t ce = pair ? launch_any<true>(a, e4m3, epilogue, cols, sms, stream)
                                : launch_any<false>(a, e4m3, epilogue, cols, sms, stream);
    if (ce != cudaSuccess)
        return record_error(CAM_E_CUDA, "%s: launch: %s", fn, cudaGetErrorString(ce));
    return CAM_OK;
}

}  // namespace cam

cudaError_t cam::operators_status(int dev, int32_t** at) {
    static std::atomic<int32_t*> known[kMaxDevices];
    const bool keep = dev < kMaxDevices;
    *at = keep ? known[dev].load(std::memory_order_relaxed) : nullptr;
    if (*at) return cudaSuccess;
    void* p = nullptr;
    const cudaError_t ce = cudaGetSymbolAddress(&p, cam::tc::g_status);
    *at = static_cast<int32_t*>(p);
    if (ce == cudaSuccess && keep) known[dev].store(*at, std::memory_order_relaxed);
    return ce;
}

CAM_API int cam_operators_status(int32_t* out) {
    const char* fn = "cam_operators_status";
    if (!out) return cam::record_error(CAM_E_ARG, "%s: out is NULL", fn);
    cudaError_t ce = cudaDeviceSynchronize();
    if (ce == cudaSuccess) ce = cudaMemcpyFromSymbol(out, cam::tc::g_status, sizeof *out);
    if (ce != cudaSuccess)
        return cam::record_error(CAM_E_CUDA, "%s: %s", fn, cudaGetErrorString(ce));
    return CAM_OK;
}
