// logprobs.cu -- cam_token_logprobs and cam_token_logprobs_backward: what a
// model says of given tokens, and its gradient (declarations, definitions and
// the cases without a distribution in include/cam.h).
//
// Forward, for a row x with largest logit M:
//   r = sum exp(x - M), t = sum exp(x - M) (x - M),
//   log s = log r,  lse = M + log s,  logp = (x_token - M) - log s,
//   entropy = log s - t / r.
// Each logit is read once from HBM (2 or 4 B and one exponential each). A
// thread keeps both sums relative to a reference of its own, the largest logit
// of its first batch, and moves it only when a later batch passes it by 16: no
// term overflows, none that counts is lost, and no thread waits for M. (Holding
// the row on the SM until M is known, in registers or a ring of shared memory,
// took 156 us where this takes 70.) A row's sums go to one of three selecting
// warps of the block through named barriers, and the streaming warps carry on
// with the next row. Where one logit has nearly all the probability (r < 1.5),
// what the others add would drown in r; their sum is taken again without M and
// log s = log1p(it), which keeps a loss of 1e-15 apart from 0.
//
// The largest `top` logits. Each thread also leaves the largest logit of every
// unit (an eighth of its vectors of the row). The top-th largest of 32 sets of
// threads' largest is a bound that at least `top` logits reach; a selecting
// warp looks again at the few units that reach it, and each candidate counts
// the candidates before it (larger, or equal with a lower id), which is its
// place. Rows with more candidates than the list holds (many equal logits) and
// rows with a NaN take one maximum at a time.
//
// Blocks take rows in turn, two blocks of 352 + 96 threads per SM for a long
// row; where rows are fewer than blocks, the blocks of a cluster share a row.
// Rows short enough for the registers of one block take a form of their own
// (token_logprobs_held), with M known before the sums.
// Measured: 2,048 x 73,760 bf16 with 10 alternatives 69 us (4.4 TB/s, 5.7 for
// each further row: 4,864 rows 140 us), 4,096 x 50,257 fp32 with one 138 us
// (5.9 TB/s). In bf16 no unit is full even at 16 rows per block (55 % of the
// issue slots, HBM 66 %, exponentials 27 %, ALU 35 %): the streaming warps, 22
// per SM, wait for their loads; a launch's ramp and last selection are 9 us.
//
// Backward. One elementwise pass, read and written once, HBM-bound: 4,096 x
// 73,760 bf16 with the entropy's term 182 us (6.6 TB/s).
#include <cooperative_groups.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <cmath>

#include "cam_internal.h"
#include "op_launch.h"

#define CAM_API extern "C" __attribute__((visibility("default")))

namespace cam {
namespace {

namespace cg = cooperative_groups;

constexpr int kLpBatch = 4;          // vectors of a thread in flight while as many are summed
constexpr int kLpMaxStream = 352;    // streaming threads of a block
constexpr int kLpSelect = 3;         // selecting warps: every third row each
constexpr int kLpBufs = kLpSelect;   // rows whose sums are handed over or being made
constexpr int kLpUnits = 8;          // parts of a thread's share of a row, each with its largest logit
constexpr int kLpMaxBlock = kLpMaxStream + 32 * kLpSelect;
constexpr int kLpList = 1024;        // candidates a block's share of a row may have
constexpr int kLpFewVectors = 128;   // vectors looked through at once
constexpr int kLpFewThreads = 96;    // threads whose vectors are scanned as a matter of course
constexpr int kLpMaxCluster = 8;
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;
constexpr float kInf = INFINITY;
// Rows with logits beyond this are summed with care, relative to their largest.
constexpr float kHuge = 1e36f;
// The streaming form's: a term's exponent is x log2(e) less the reference's rounded product, so
// even of x = reference it is what that rounding left out, up to 64 here and 2^7 from 2^31 on.
// Rows whose largest logit lies beyond are summed by one warp; below its negative logits are masks,
// which need no reference (exp of their distance from any other row's largest is 0).
constexpr float kFar = 1073741824.0f;

struct LogprobArgs {
    const void* logits;
    int64_t stride;
    const int64_t* tokens;
    float* logp;
    float* entropy;
    float* lse;
    float* lse_lo;
    float* top_logp;
    int64_t* top_ids;
    int32_t rows;
    int32_t vocab;
    int32_t top;
    int32_t cluster;
    int32_t stream;   // streaming threads of a block, a multiple of 32
    int32_t iters;    // vectors of a thread per row at most
    int32_t unit;     // of which a unit has so many (a multiple of kLpBatch)
};

__device__ __forceinline__ float ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

__device__ __forceinline__ float max_nan(float a, float b) {  // NaN if either is
    float m;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(m) : "f"(a), "f"(b));
    return m;
}

// Two binary32 in one 64-bit register and the operations on both at once.
using Pair = unsigned long long;
__device__ __forceinline__ Pair pair(float lo, float hi) {
    Pair p;
    asm("mov.b64 %0, {%1, %2};" : "=l"(p) : "f"(lo), "f"(hi));
    return p;
}
__device__ __forceinline__ void split(Pair p, float& lo, float& hi) {
    asm("mov.b64 {%0, %1}, %2;" : "=f"(lo), "=f"(hi) : "l"(p));
}
__device__ __forceinline__ Pair add2(Pair a, Pair b) {
    Pair d;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
    return d;
}
__device__ __forceinline__ Pair mul2(Pair a, Pair b) {
    Pair d;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
    return d;
}
__device__ __forceinline__ Pair fma2(Pair a, Pair b, Pair c) {
    Pair d;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(d) : "l"(a), "l"(b), "l"(c));
    return d;
}

// One 16-byte vector of logits, widened on access.
template <typename T>
struct Vec16;

template <>
struct Vec16<float> {
    static constexpr int kN = 4;
    uint4 u;
    __device__ __forceinline__ float get(int j) const {
        return __uint_as_float(j == 0 ? u.x : j == 1 ? u.y : j == 2 ? u.z : u.w);
    }
    static __device__ __forceinline__ uint4 nothing() {  // -inf
        return make_uint4(0xFF800000u, 0xFF800000u, 0xFF800000u, 0xFF800000u);
    }
    __device__ __forceinline__ float largest() const {  // NaN apart
        return fmaxf(fmaxf(get(0), get(1)), fmaxf(get(2), get(3)));
    }
    // the largest of N vectors, NaN if one holds a NaN
    template <int N>
    static __device__ __forceinline__ float largest_nan(const Vec16 (&v)[N]) {
        float m = v[0].get(0);
#pragma unroll
        for (int i = 0; i < N; ++i)
#pragma unroll
            for (int j = 0; j < 4; ++j) m = max_nan(m, v[i].get(j));
        return m;
    }
    using Floor = float;
    static __device__ __forceinline__ Floor floor_at(float low) { return low; }
    __device__ __forceinline__ Vec16 held_at(Floor low) const {  // NaN stays
        Vec16 v;
        v.u = make_uint4(hold(u.x, low), hold(u.y, low), hold(u.z, low), hold(u.w, low));
        return v;
    }
    __device__ __forceinline__ Vec16 held_finite() const { return held_at(-2e38f); }
    static __device__ __forceinline__ uint32_t hold(uint32_t w, Floor low) {
        return __float_as_uint(max_nan(__uint_as_float(w), low));
    }
};

template <>
struct Vec16<uint16_t> {
    static constexpr int kN = 8;
    uint4 u;
    __device__ __forceinline__ float get(int j) const {
        const uint32_t w = j < 2 ? u.x : j < 4 ? u.y : j < 6 ? u.z : u.w;
        return __uint_as_float((j & 1) ? w & 0xFFFF0000u : w << 16);
    }
    static __device__ __forceinline__ uint4 nothing() {
        return make_uint4(0xFF80FF80u, 0xFF80FF80u, 0xFF80FF80u, 0xFF80FF80u);
    }
    __device__ __forceinline__ float largest() const {
        const __nv_bfloat162 m =
            __hmax2(__hmax2(as2(u.x), as2(u.y)), __hmax2(as2(u.z), as2(u.w)));
        return fmaxf(__low2float(m), __high2float(m));
    }
    template <int N>
    static __device__ __forceinline__ float largest_nan(const Vec16 (&v)[N]) {
        __nv_bfloat162 m = as2(v[0].u.x);
#pragma unroll
        for (int i = 0; i < N; ++i)
            m = __hmax2_nan(__hmax2_nan(m, __hmax2_nan(as2(v[i].u.x), as2(v[i].u.y))),
                            __hmax2_nan(as2(v[i].u.z), as2(v[i].u.w)));
        return max_nan(__low2float(m), __high2float(m));
    }
    using Floor = __nv_bfloat162;
    static __device__ __forceinline__ Floor floor_at(float low) {  // the next bf16 below, twice
        return __bfloat162bfloat162(__float2bfloat16_rd(low));
    }
    __device__ __forceinline__ Vec16 held_at(Floor low) const {  // NaN stays
        Vec16 v;
        v.u = make_uint4(hold(u.x, low), hold(u.y, low), hold(u.z, low), hold(u.w, low));
        return v;
    }
    __device__ __forceinline__ Vec16 held_finite() const { return held_at(as2(0xFF16FF16u)); }
    static __device__ __forceinline__ uint32_t hold(uint32_t w, Floor low) {
        const __nv_bfloat162 m = __hmax2_nan(as2(w), low);
        return *reinterpret_cast<const uint32_t*>(&m);
    }
    static __device__ __forceinline__ __nv_bfloat162 as2(uint32_t w) {
        return *reinterpret_cast<const __nv_bfloat162*>(&w);
    }
};

template <typename T>
__device__ __forceinline__ Vec16<T> load16(const T* p) {
    Vec16<T> v;
    asm volatile("ld.global.nc.v4.b32 {%0,%1,%2,%3}, [%4];"
                 : "=r"(v.u.x), "=r"(v.u.y), "=r"(v.u.z), "=r"(v.u.w)
                 : "l"(p));
    return v;
}

__device__ __forceinline__ float widen1(float v) { return v; }
__device__ __forceinline__ float widen1(uint16_t v) {
    return __uint_as_float(static_cast<uint32_t>(v) << 16);
}

__device__ __forceinline__ float warp_max(float v) {  // NaN apart
    float m;
    asm("redux.sync.max.f32 %0, %1, 0xffffffff;" : "=f"(m) : "f"(v));
    return m;
}
__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
    for (int o = 16; o > 0; o /= 2) v += __shfl_xor_sync(0xFFFFFFFFu, v, o);
    return v;
}

// Named barriers of a block: a row's sums handed to its selecting warp, and its
// buffers handed back. There is one of each for every selecting warp, so that
// none comes to a barrier in another's place.
constexpr int kBarFull = 1, kBarFree = kBarFull + kLpSelect;
static_assert(kBarFree + kLpSelect <= 16, "a block has 16 barriers");
__device__ __forceinline__ void bar_sync(int id, int n) {
    asm volatile("barrier.cta.sync %0, %1;" ::"r"(id), "r"(n) : "memory");
}
__device__ __forceinline__ void bar_arrive(int id, int n) {
    asm volatile("barrier.cta.arrive %0, %1;" ::"r"(id), "r"(n) : "memory");
}
__device__ __forceinline__ void cluster_arrive() {
    asm volatile("barrier.cluster.arrive.release;" ::: "memory");
}
__device__ __forceinline__ void cluster_wait() {
    asm volatile("barrier.cluster.wait.acquire;" ::: "memory");
}

// A logit and its id as one whole number: larger for a larger logit (NaN
// above +inf, -0 as +0) and, among equals, for a lower id. Never 0 nor ~0.
using Key = unsigned long long;
__device__ __forceinline__ Key make_key(float x, uint32_t id) {
    uint32_t u = __float_as_uint(x + 0.0f);
    if ((u & 0x7FFFFFFFu) > 0x7F800000u) u = 0x7FFFFFFEu;
    u ^= (u >> 31) ? 0xFFFFFFFFu : 0x80000000u;
    return (static_cast<Key>(u) << 32) | (0xFFFFFFFFu - id);
}
__device__ __forceinline__ float key_logit(Key key) {
    const uint32_t u = static_cast<uint32_t>(key >> 32);
    return __uint_as_float(u ^ ((u >> 31) ? 0x80000000u : 0xFFFFFFFFu));
}
__device__ __forceinline__ int64_t key_id(Key key) {
    return 0xFFFFFFFFu - static_cast<uint32_t>(key);
}
__device__ __forceinline__ Key warp_max_key(Key v) {
#pragma unroll
    for (int o = 16; o > 0; o /= 2) v = max(v, __shfl_xor_sync(0xFFFFFFFFu, v, o));
    return v;
}

// The n-th largest (n = 1..32) of the warp's 32 values, on every lane: a
// bitonic sort, descending.
__device__ __forceinline__ float nth_of_warp(float v, int n) {
    const int lane = threadIdx.x & 31;
#pragma unroll
    for (int size = 2; size <= 32; size *= 2)
#pragma unroll
        for (int o = size / 2; o > 0; o /= 2) {
            const float w = __shfl_xor_sync(0xFFFFFFFFu, v, o);
            const bool up = ((lane & size) == 0) == ((lane & o) == 0);  // keeps the larger
            v = up ? fmaxf(v, w) : fminf(v, w);
        }
    return __shfl_sync(0xFFFFFFFFu, v, n - 1);
}

// What a block knows of its share of a row.
struct Share {
    float m;  // largest logit (NaN apart), -inf where there is none
    float c;  // logits equal to m
    float r;  // sum of exp(x - m) over the others
    float t;  // sum of exp(x - m) (x - m)
};

// What a row's share says of the row. (No distribution: c and r are 0; a NaN or
// +inf: r is NaN.)
struct RowResult {
    Share s;
    float log_s;
    bool dead;
    __device__ __forceinline__ explicit RowResult(const Share& share) : s(share) {
        if (s.m == kInf) s.r = NAN;
        dead = s.m == -kInf && s.r == 0.0f;
        log_s = dead ? 0.0f : log1pf((s.c - 1.0f) + s.r);
    }
    __device__ __forceinline__ float logp_of(float v) const {
        return dead ? -kInf : (v - s.m) - log_s;
    }
    __device__ __forceinline__ void write(const LogprobArgs& a, int64_t row, int64_t token,
                                          float x_token) const {
        const float lse = dead ? -kInf : s.m + log_s;
        if (a.lse) a.lse[row] = lse;
        if (a.lse_lo) {  // what the sum's rounding left out, exactly (the order of the two is free)
            const float b = __fsub_rn(lse, s.m);
            const float lo = __fadd_rn(__fsub_rn(s.m, __fsub_rn(lse, b)), __fsub_rn(log_s, b));
            a.lse_lo[row] = isfinite(lse) ? lo : 0.0f;
        }
        if (a.entropy) a.entropy[row] = dead ? 0.0f : log_s - __fdividef(s.t, s.c + s.r);
        if (a.logp)
            a.logp[row] = token >= a.vocab ? NAN : token >= 0 ? logp_of(x_token) : 0.0f;
    }
    __device__ __forceinline__ void write_top(const LogprobArgs& a, int64_t row, int place,
                                              Key key) const {
        if (a.top_ids) a.top_ids[row * a.top + place] = key_id(key);
        if (a.top_logp) a.top_logp[row * a.top + place] = logp_of(key_logit(key));
    }
};

// How many of a descending list's n <= 32 keys are above a key.
__device__ __forceinline__ int count_above(const Key* list, int n, Key key) {
    int at = 0;
#pragma unroll
    for (int step = 32; step > 0; step /= 2)
        if (at + step <= n && list[at + step - 1] > key) at += step;
    return at;
}

// What a streaming warp hands over of its vectors of a row. Sums are of
// 2^(x log2(e) - m log2(e)) and of that times its exponent; those of the lane
// that holds m stand apart, so that a confident row can leave m itself out.
struct WarpSums {
    float m;             // largest logit
    float s, t;          // sums of the lanes whose largest is less
    float top_s, top_t;  // and of the others
    int top_lane;        // one of the others
};

struct LogprobShared {
    WarpSums warps[kLpBufs][kLpMaxStream / 32];
    float thread_max[kLpBufs][kLpMaxStream];  // largest logit of each thread's vectors
    Key list[kLpSelect][kLpList];
    uint4 vectors[kLpSelect][kLpFewVectors];
    int vector_ids[kLpSelect][kLpFewVectors];
    Key best[kLpSelect][CAM_LOGPROBS_MAX_TOP];
    Key all_best[kLpMaxCluster][CAM_LOGPROBS_MAX_TOP];  // the leader's: every block's
    Share shares[kLpMaxCluster];                        // the leader's
    uint16_t threads[kLpSelect][kLpMaxStream];
    uint16_t units[kLpSelect][kLpFewThreads * kLpUnits];
    // then, [kLpBufs][stream][kLpUnits]: the largest logit of each unit
};

// Where a row's vectors lie: [0, head) and the last `tail` logits singly (by
// the leader of the cluster), 16-byte vectors between, dealt out to the
// cluster's streaming threads in turn.
template <typename T>
struct RowPlan {
    const T* x;
    int head, n_vec, tail;
    __device__ __forceinline__ RowPlan(const T* row, int vocab) : x(row) {
        head = min(vocab, static_cast<int>((16 - (reinterpret_cast<uintptr_t>(row) & 15)) & 15) /
                              static_cast<int>(sizeof(T)));
        n_vec = (vocab - head) / Vec16<T>::kN;
        tail = vocab - head - n_vec * Vec16<T>::kN;
    }
    __device__ __forceinline__ int single_id(int i, int vocab) const {  // i in [0, head + tail)
        return i < head ? i : vocab - tail + (i - head);
    }
};

// The block's largest logits into `out[0..top)`, in order (0 where there are
// none), by one warp. `bad`: the share holds a NaN.
// (Loops stay rolled, here and in select_rows: this code runs once per row beside the streaming
// warps, whose instructions it displaces. 8,192 x 30,000 bf16 with one alternative takes 124 us,
// with the loops as the compiler unrolls them 129, unrolled by four 152.)
template <typename T>
__device__ __noinline__ void select(const LogprobArgs& a, LogprobShared& sh, const RowPlan<T>& row,
                                    int buf, int rank, bool bad, Key* out) {
    constexpr int kN = Vec16<T>::kN;
    constexpr uint32_t kAll = 0xFFFFFFFFu;
    Key* list = sh.list[buf];
    uint16_t* threads = sh.threads[buf];
    uint16_t* units = sh.units[buf];
    uint4* vectors = sh.vectors[buf];
    int* vector_ids = sh.vector_ids[buf];
    const float* thread_max = sh.thread_max[buf];
    const float* unit_max = reinterpret_cast<const float*>(&sh + 1) + buf * a.stream * kLpUnits;
    const int lane = threadIdx.x & 31;
    const uint32_t below = (1u << lane) - 1u;
    const int singles = rank == 0 ? row.head + row.tail : 0;
    const int across = a.stream * a.cluster;
    int n = 0;  // candidates so far, the same on every lane
    auto put = [&](bool hit, float v, int id) {
        const uint32_t who = __ballot_sync(kAll, hit);
        if (hit) {
            const int at = n + __popc(who & below);
            if (at < kLpList) list[at] = make_key(v, static_cast<uint32_t>(id));
        }
        n += __popc(who);
    };
    // vectors with something wanted, kept until they are looked through
    int n_vectors = 0;
    auto keep = [&](bool hit, const Vec16<T>& v, int id) {
        const uint32_t who = __ballot_sync(kAll, hit);
        if (hit) {
            const int at = n_vectors + __popc(who & below);
            vectors[at] = v.u;
            vector_ids[at] = id;
        }
        n_vectors += __popc(who);
    };
    auto look_through = [&](auto&& wanted) {  // a lane to a logit
        __syncwarp();
        const T* flat = reinterpret_cast<const T*>(vectors);
#pragma unroll 1
        for (int i = lane; i < ((n_vectors * kN + 31) & ~31); i += 32) {
            const bool valid = i < n_vectors * kN;
            const float v = valid ? widen1(flat[i]) : 0.0f;
            put(valid && wanted(v), v, valid ? vector_ids[i / kN] + i % kN : 0);
        }
        n_vectors = 0;
        __syncwarp();
    };
    if (!bad) {
        // 32 sets of threads: the top-th largest of the sets' largest is a bound that at least
        // `top` logits reach
        float m = -kInf;
#pragma unroll 1
        for (int j = lane; j < a.stream; j += 32) m = fmaxf(m, thread_max[j]);
        const float bound = a.top == 1 ? warp_max(m) : nth_of_warp(m, a.top);
        if (singles > 0) {
            const int id = lane < singles ? row.single_id(lane, a.vocab) : 0;
            const float v = lane < singles ? widen1(row.x[id]) : 0.0f;
            put(lane < singles && v >= bound, v, id);
        }
        // the threads that reach the bound (or pass it)
        int n_thr = 0;
        auto list_threads = [&](auto&& wanted) {
            n_thr = 0;
#pragma unroll 1
            for (int j = lane; j < a.stream; j += 32) {
                const bool hit = wanted(thread_max[j]);
                const uint32_t who = __ballot_sync(kAll, hit);
                if (hit) threads[n_thr + __popc(who & below)] = static_cast<uint16_t>(j);
                n_thr += __popc(who);
            }
            __syncwarp();
        };
        // what of their vectors does: the units that reach it, four lanes to a unit's vectors
        auto scan_threads = [&](auto&& wanted) {
#pragma unroll 1
            for (int q0 = 0; q0 < n_thr; q0 += kLpFewThreads) {
                const int pairs = min(n_thr - q0, kLpFewThreads) * kLpUnits;
                int n_units = 0;
#pragma unroll 1
                for (int u0 = 0; u0 < pairs; u0 += 32) {
                    const int u = u0 + lane;
                    int at = 0;
                    bool hit = false;
                    if (u < pairs) {
                        at = threads[q0 + u / kLpUnits] * kLpUnits + u % kLpUnits;
                        hit = wanted(unit_max[at]);
                    }
                    const uint32_t who = __ballot_sync(kAll, hit);
                    if (hit) units[n_units + __popc(who & below)] = static_cast<uint16_t>(at);
                    n_units += __popc(who);
                }
                __syncwarp();
#pragma unroll 1
                for (int i0 = 0; i0 < a.unit; i0 += 4)
#pragma unroll 1
                    for (int u0 = 0; u0 < n_units; u0 += 32) {
                        Vec16<T> v[4];
                        int w[4];
#pragma unroll
                        for (int k = 0; k < 4; ++k) {
                            const int u = u0 + 8 * k + (lane >> 2);
                            w[k] = row.n_vec;
                            if (u < n_units) {
                                const int at = units[u], i = at % kLpUnits * a.unit + i0 + (lane & 3);
                                if (i < a.iters)
                                    w[k] = i * across + rank * a.stream + at / kLpUnits;
                            }
                            if (w[k] < row.n_vec) v[k] = load16(row.x + row.head + w[k] * kN);
                        }
#pragma unroll
                        for (int k = 0; k < 4; ++k)
                            if (u0 + 8 * k < n_units)
                                keep(w[k] < row.n_vec && wanted(v[k].largest()), v[k],
                                     row.head + w[k] * kN);
                        look_through(wanted);
                    }
            }
        };
        const auto reaches = [&](float v) { return v >= bound; };
        const auto passes = [&](float v) { return v > bound; };
        list_threads(reaches);
        if (n_thr <= kLpFewThreads) {
            scan_threads(reaches);
        } else {
            // many logits equal to the bound: those above it from their threads, and of the
            // equal ones the first `top` in the order of ids
            list_threads(passes);
            scan_threads(passes);
            const int enough = n + a.top;
#pragma unroll 1
            for (int u = lane; n < enough; u += 32) {
                // the share's vector number u, in the order of ids
                const int w = (u / a.stream) * across + rank * a.stream + u % a.stream;
                if (__all_sync(kAll, w >= row.n_vec)) break;
                Vec16<T> v;
                bool hit = false;
                if (w < row.n_vec) {
                    v = load16(row.x + row.head + w * kN);
#pragma unroll
                    for (int j = 0; j < kN; ++j) hit |= v.get(j) == bound;
                }
                keep(hit, v, row.head + w * kN);
                look_through([&](float e) { return e == bound; });
            }
        }
        __syncwarp();
    }
    if (!bad && n <= kLpList) {
        if (lane < a.top && lane >= n) out[lane] = 0;
        if (n <= 128) {  // a candidate's place is the number before it
#pragma unroll 1
            for (int i = lane; i < n; i += 32) {
                const Key key = list[i];
                int place = 0;
#pragma unroll 4
                for (int k = 0; k < n; ++k) place += list[k] > key;
                if (place < a.top) out[place] = key;
            }
        } else {
            Key last = ~0ull;
#pragma unroll 1
            for (int p = 0; p < a.top; ++p) {
                Key key = 0;
#pragma unroll 1
                for (int i = lane; i < n; i += 32) {
                    const Key u = list[i];
                    if (u < last) key = max(key, u);
                }
                last = warp_max_key(key);
                if (lane == 0) out[p] = last;
            }
        }
    } else {
        // a NaN, or more candidates than the list holds: one maximum at a time over the share
        Key last = ~0ull;
#pragma unroll 1
        for (int p = 0; p < a.top; ++p) {
            Key key = 0;
            auto look = [&](float v, int id) {
                const Key u = make_key(v, static_cast<uint32_t>(id));
                if (u < last) key = max(key, u);
            };
#pragma unroll 1
            for (int i = lane; i < singles; i += 32) {
                const int id = row.single_id(i, a.vocab);
                look(widen1(row.x[id]), id);
            }
#pragma unroll 1
            for (int u = lane;; u += 32) {
                const int w = (u / a.stream) * across + rank * a.stream + u % a.stream;
                if (w >= row.n_vec) break;
                const Vec16<T> v = load16(row.x + row.head + w * kN);
#pragma unroll
                for (int j = 0; j < kN; ++j) look(v.get(j), row.head + w * kN + j);
            }
            last = warp_max_key(key);
            if (lane == 0) out[p] = last;
        }
    }
    __syncwarp();
}

// A share summed by one warp, its largest logit first: for rows with a NaN or
// logits beyond kFar.
template <typename T>
__device__ __noinline__ Share careful(const LogprobArgs& a, const RowPlan<T>& row, int rank) {
    constexpr int kN = Vec16<T>::kN;
    const int lane = threadIdx.x & 31, singles = rank == 0 ? row.head + row.tail : 0;
    const int across = a.stream * a.cluster;
    auto each = [&](auto&& f) {
        for (int i = lane; i < singles; i += 32) f(widen1(row.x[row.single_id(i, a.vocab)]));
        for (int i = 0; i < a.iters; ++i)
            for (int j = lane; j < a.stream; j += 32) {
                const int w = i * across + rank * a.stream + j;
                if (w >= row.n_vec) continue;
                const Vec16<T> v = load16(row.x + row.head + int64_t(w) * kN);
#pragma unroll
                for (int e = 0; e < kN; ++e) f(v.get(e));
            }
    };
    float m = -kInf, r = 0.0f, c = 0.0f, t = 0.0f;
    each([&](float x) {
        m = fmaxf(m, x);
        if (x != x || x == kInf) r = NAN;
    });
    m = warp_max(m);
    const float from = m == -kInf ? 0.0f : m;
    each([&](float x) {
        if (x == m) {
            if (m != -kInf) c += 1.0f;
        } else {
            const float d = max_nan(x - from, -200.0f), e = ex2(d * kLog2e);
            r += e;
            t += e * d;
        }
    });
    return Share{m, warp_sum(c), warp_sum(r), warp_sum(t)};
}

// A selecting warp: the results of rows par, par + kLpSelect, ... of the block
// while later rows stream.
template <typename T>
__device__ __noinline__ void select_rows(const LogprobArgs& a, LogprobShared& sh, int par,
                                         int rank, int first, int step, int n_rows) {
    constexpr int kN = Vec16<T>::kN;
    const int lane = threadIdx.x & 31, n_warps = a.stream >> 5, both = a.stream + 32;
    const bool clustered = a.cluster > 1;
    const int across = a.stream * a.cluster;
    const int buf = par;
    const bool ask = a.logp && rank == 0;
    int64_t next_token = ask && par < n_rows ? a.tokens[first + int64_t(par) * step] : -1;
#pragma unroll 1
    for (int k = par; k < n_rows; k += kLpSelect) {
        const int64_t r_at = first + int64_t(k) * step;
        const RowPlan<T> row(static_cast<const T*>(a.logits) + r_at * a.stride, a.vocab);
        const int singles = rank == 0 ? row.head + row.tail : 0;
        // (these loads overlap the wait, and the next row's token the row)
        const int64_t token = next_token;
        if (ask && k + kLpSelect < n_rows) next_token = a.tokens[r_at + int64_t(kLpSelect) * step];
        const float single = lane < singles ? widen1(row.x[row.single_id(lane, a.vocab)]) : -kInf;
        const float x_token = token >= 0 && token < a.vocab ? widen1(row.x[token]) : 0.0f;
        bar_sync(kBarFull + buf, both);
        const WarpSums ws = lane < n_warps ? sh.warps[buf][lane]
                                           : WarpSums{-kInf, 0.0f, 0.0f, 0.0f, 0.0f, 0};
        Share s;
        s.m = fmaxf(warp_max(ws.m), warp_max(fmaxf(single, -kInf)));
        const float from = s.m == -kInf ? 0.0f : s.m;
        // the warps' sums and the single logits, relative to m
        const float d = fmaxf(ws.m - from, -1e30f) * kLog2e, f = ex2(d);
        const float one_y = max_nan((single - from) * kLog2e, -150.0f), one = ex2(one_y);
        s.c = 0.0f;
        s.r = warp_sum(f * (ws.s + ws.top_s) + one);
        s.t = warp_sum(f * (ws.t + ws.top_t + d * (ws.s + ws.top_s)) + one * one_y) * kLn2;
        bool bad = false;
        if (!(s.r < 1.5f) || s.m == -kInf) {
            // (a sum that lost its row: a NaN, logits beyond kFar either way)
            bad = s.r != s.r || fabsf(s.m) >= kFar;
            if (bad && !(s.m == -kInf && s.r == 0.0f)) s = careful<T>(a, row, rank);
            bad = s.r != s.r;
        } else if (fabsf(s.m) >= kFar) {
            s = careful<T>(a, row, rank);
            bad = s.r != s.r;
        } else {
            // One logit has most of the probability. What the others add to it would drown in
            // the sum, so the sum is taken again without it: its own thread's vectors are read
            // once more, all else is apart already.
            s.c = 1.0f;
            const bool mine = lane < n_warps && ws.m == s.m;
            float r = mine ? ws.s : f * (ws.s + ws.top_s);
            float t = mine ? ws.t : f * (ws.t + ws.top_t + d * (ws.s + ws.top_s));
            if (single != s.m) r += one, t += one * one_y;
            const uint32_t who = __ballot_sync(0xFFFFFFFFu, mine);
            if (who != 0) {
                const int w = __ffs(who) - 1;
                const int v0 = rank * a.stream + w * 32 + __shfl_sync(0xFFFFFFFFu, ws.top_lane, w);
#pragma unroll 1
                for (int i = lane; i < a.iters; i += 32) {
                    if (v0 + i * across >= row.n_vec) break;
                    const Vec16<T> v = load16(row.x + row.head + int64_t(v0 + i * across) * kN);
#pragma unroll
                    for (int j = 0; j < kN; ++j) {
                        if (v.get(j) == s.m) continue;
                        const float y = fmaxf((v.get(j) - s.m) * kLog2e, -150.0f), e = ex2(y);
                        r += e;
                        t += e * y;
                    }
                }
            }
            s.r = warp_sum(r);
            s.t = warp_sum(t) * kLn2;
        }
        Key* best = sh.best[buf];
        if (a.top > 0) {
            if (clustered) best = cg::this_cluster().map_shared_rank(&sh.all_best[rank][0], 0);
            select<T>(a, sh, row, buf, rank, bad, best);
        }
        if (k + kLpBufs < n_rows) bar_arrive(kBarFree + buf, both);
        if (clustered) {
            if (lane == 0) *cg::this_cluster().map_shared_rank(&sh.shares[rank], 0) = s;
            __syncwarp();
            cluster_arrive();
            cluster_wait();
            if (rank != 0) return;
            // the row from its shares
            float M = -kInf;
#pragma unroll 1
            for (int j = 0; j < a.cluster; ++j) M = fmaxf(M, sh.shares[j].m);
            Share all{M, 0.0f, 0.0f, 0.0f};
#pragma unroll 1
            for (int j = 0; j < a.cluster; ++j) {
                const Share o = sh.shares[j];
                if (o.m == M) {
                    all.c += o.c, all.r += o.r, all.t += o.t;
                } else {
                    const float d = fmaxf(o.m - M, -1e30f), e = ex2(d * kLog2e);
                    all.r += e * (o.c + o.r);
                    all.t += e * (o.t + d * (o.c + o.r));
                }
            }
            s = all;
        }
        const RowResult result(s);
        if (lane == 0) result.write(a, r_at, token, x_token);
#pragma unroll 1
        for (int i = lane; i < a.cluster * a.top; i += 32) {
            const Key key = clustered ? sh.all_best[i / a.top][i % a.top] : best[i];
            if (key == 0) continue;
            int place = i;
            if (clustered) {  // each block's list is in order
                place = 0;
#pragma unroll
                for (int j = 0; j < kLpMaxCluster; ++j)
                    if (j < a.cluster) place += count_above(sh.all_best[j], a.top, key);
            }
            if (place < a.top) result.write_top(a, r_at, place, key);
        }
        __syncwarp();
    }
    if (clustered && par >= n_rows) {  // the selecting warps without the cluster's one row
        cluster_arrive();
        cluster_wait();
    }
}

template <typename T>
__global__ void __launch_bounds__(kLpMaxBlock, 2)
    token_logprobs(const __grid_constant__ LogprobArgs a) {
    constexpr int kN = Vec16<T>::kN;
    extern __shared__ __align__(128) uint8_t smem[];
    LogprobShared& sh = *reinterpret_cast<LogprobShared*>(smem);

    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int n_warps = a.stream >> 5, both = a.stream + 32;
    const bool clustered = a.cluster > 1;  // (then a block has one row)
    const int rank = clustered ? static_cast<int>(cg::this_cluster().block_rank()) : 0;
    const int first = blockIdx.x / a.cluster, step = gridDim.x / a.cluster;
    const int n_rows = first < a.rows ? (a.rows - first - 1) / step + 1 : 0;
    const int across = a.stream * a.cluster;
    const T* logits = static_cast<const T*>(a.logits);
    auto plan = [&](int k) {
        return RowPlan<T>(logits + (first + int64_t(k) * step) * a.stride, a.vocab);
    };
    if (clustered) {  // every block of the cluster has started
        cluster_arrive();
        cluster_wait();
    }

    if (warp < n_warps) {
        // ---- streaming ---------------------------------------------------------------
        // The sums are taken relative to a reference of the thread's own: its first batch's
        // largest logit, moved up when a batch passes it by 16, so that no term overflows and
        // none that counts is lost. No thread waits for another within a row.
        using Batch = Vec16<T>[kLpBatch];
        const int w0 = rank * a.stream + warp * 32;  // the warp's first vector
        int l_row = 0, l_w = w0, l_vecs = 0;         // the next batch to load
        const T* l_at = nullptr;
        const int64_t jump = int64_t(across) * kN;
        auto whole = [&](int w, int n_vec) { return w + 32 + (kLpBatch - 1) * across <= n_vec; };
        auto load = [&](Batch& v, int& w, int& n_vec) {
            if (l_w == w0 && l_row < n_rows) {
                const RowPlan<T> p = plan(l_row);
                l_vecs = p.n_vec;
                l_at = p.x + p.head + int64_t(w0 + lane) * kN;
            }
            w = l_w;
            n_vec = l_row < n_rows ? l_vecs : 0;
            if (whole(w, n_vec)) {
#pragma unroll
                for (int j = 0; j < kLpBatch; ++j) v[j] = load16(l_at + j * jump);
            } else {
                constexpr uint32_t kPad = sizeof(T) == 4 ? 0xFF800000u : 0xFF80FF80u;  // -inf
#pragma unroll
                for (int j = 0; j < kLpBatch; ++j) {
                    v[j].u = make_uint4(kPad, kPad, kPad, kPad);
                    if (w + lane + j * across < n_vec) v[j] = load16(l_at + j * jump);
                }
            }
            l_w += kLpBatch * across;
            l_at += kLpBatch * jump;
            if (l_w >= a.iters * across + w0) l_w = w0, ++l_row;
        };

        const Pair log2e = pair(kLog2e, kLog2e);
        float m = -kInf, limit = -kFar, ref = 0.0f;  // ref: minus the reference times log2(e)
        float unit_m = -kInf;                        // the largest of the unit under way
        const int unit_batches = a.unit / kLpBatch;
        int unit_left = unit_batches;
        float* unit_max = reinterpret_cast<float*>(&sh + 1) + tid * kLpUnits;
        float* unit_at = unit_max;
        Pair s2 = pair(0.0f, 0.0f), t2 = s2;
        auto add = [&](const Batch& v, int w, int n_vec) {
            const float big = Vec16<T>::largest_nan(v);
            if (!(big <= limit)) {
                if (big < kFar) {
                    const float up = -big * kLog2e, by = up - ref;
                    const float f = limit == -kFar ? 0.0f : ex2(by);
                    s2 = mul2(s2, pair(f, f));
                    t2 = limit == -kFar ? t2 : fma2(t2, pair(f, f), mul2(s2, pair(by, by)));
                    ref = up;
                    limit = big + 16.0f;
                } else {  // NaN, or too large
                    s2 = pair(NAN, NAN);
                }
            }
            m = fmaxf(m, big);
            unit_m = fmaxf(unit_m, big);
            if (--unit_left == 0) {
                *unit_at++ = unit_m;
                unit_m = -kInf, unit_left = unit_batches;
            }
            const Pair ref2 = pair(ref, ref);
            auto sum = [&](const Vec16<T>& x) {
                // a mask held finite: its exponent times its term is then 0 and not NaN
                const Vec16<T> u = x.held_finite();
#pragma unroll
                for (int q = 0; q < kN; q += 2) {
                    const Pair y = fma2(pair(u.get(q), u.get(q + 1)), log2e, ref2);
                    float y0, y1;
                    split(y, y0, y1);
                    const Pair e = pair(ex2(y0), ex2(y1));
                    s2 = add2(s2, e);
                    t2 = fma2(e, y, t2);
                }
            };
            if (whole(w, n_vec)) {
#pragma unroll
                for (int j = 0; j < kLpBatch; ++j) sum(v[j]);
            } else {
#pragma unroll
                for (int j = 0; j < kLpBatch; ++j)
                    if (w + j * across < n_vec) sum(v[j]);  // (the whole warp's)
            }
        };
        auto finish = [&](int k) {  // the warp's sums of row k, relative to its largest
            const int buf = k % kLpBufs;
            float s, t, hi;
            split(s2, s, hi);
            s += hi;
            split(t2, t, hi);
            t += hi;
            const float wm = warp_max(m);
            const bool top = m == wm;
            const float y = fmaf(wm, kLog2e, ref);  // >= 0 where the lane has a reference
            const float f = s == 0.0f ? 0.0f : ex2(-y);
            t = s == 0.0f ? 0.0f : f * fmaf(-y, s, t);
            s *= f;
            const float rest_s = warp_sum(top ? 0.0f : s), rest_t = warp_sum(top ? 0.0f : t);
            const uint32_t who = __ballot_sync(0xFFFFFFFFu, top);
            const int top_lane = __ffs(who) - 1;
            float top_s = s, top_t = t;  // (on the top lane)
            if (who & (who - 1)) {
                top_s = warp_sum(top ? s : 0.0f);
                top_t = warp_sum(top ? t : 0.0f);
            }
            if (unit_left < unit_batches) *unit_at = unit_m;
            sh.thread_max[buf][tid] = m;
            if (lane == top_lane)
                sh.warps[buf][warp] = WarpSums{wm, rest_s, rest_t, top_s, top_t, top_lane};
            bar_arrive(kBarFull + buf, both);
            m = -kInf, limit = -kFar, ref = 0.0f;
            s2 = t2 = pair(0.0f, 0.0f);
            // the next row's buffer
            unit_m = -kInf, unit_left = unit_batches;
            const int next = (k + 1) % kLpBufs;
            unit_at = unit_max + next * a.stream * kLpUnits;
            if (k + 1 >= kLpBufs && k + 1 < n_rows) bar_sync(kBarFree + next, both);
        };

        Batch v0, v1;
        int at0, at1, n0, n1;
        const int batches = (a.iters + kLpBatch - 1) / kLpBatch;
        int left = batches, k = 0;
        load(v0, at0, n0);
        while (k < n_rows) {
            load(v1, at1, n1);
            add(v0, at0, n0);
            if (--left == 0) {
                finish(k);
                left = batches;
                if (++k == n_rows) break;
            }
            load(v0, at0, n0);
            add(v1, at1, n1);
            if (--left == 0) finish(k), left = batches, ++k;
        }
        if (clustered) {
            __syncwarp();
            cluster_arrive();
            cluster_wait();
        }
        return;
    }

    select_rows<T>(a, sh, warp - n_warps, rank, first, step, n_rows);
}

// ---- rows that fit the registers of a few warps ----------------------------------

constexpr int kLhMaxWarps = 16;  // of a block, which has one row
constexpr int kLhMost = 16;      // vectors per thread
constexpr int kLhFill = 16;      // warps per SM that rows are cut for (8 to 32 measure alike)
constexpr int kLhList = 256;     // candidates a row may have, and vectors with one

struct HeldShared {
    float thread_max[32 * kLhMaxWarps];
    float warp_max[kLhMaxWarps];
    float c[kLhMaxWarps], r[kLhMaxWarps], t[kLhMaxWarps];
    Key key[kLhMaxWarps];
    int n, n_vectors;
    Key list[kLhList];
    uint16_t vectors[kLhList];
};

// NV vectors of a row per thread, loaded at once and kept: the largest logit,
// then the sums relative to it, then the few candidates, which are read once
// more. Other blocks of the SM load meanwhile; what bounds many rows are the
// instructions (8,192 x 4,000 bf16 21 us, 3.1 TB/s; fp32 28 us, 4.8 TB/s).
// Registers for the blocks that are to be resident: 102 of them at NV = 8 cost
// 8,192 x 1,000 fp32 a tenth.
template <typename T, int NV>
__global__ void __maxnreg__(NV <= 4 ? 64 : NV <= 8 ? 80 : 128)
    token_logprobs_held(const __grid_constant__ LogprobArgs a) {
    constexpr int kN = Vec16<T>::kN;
    __shared__ HeldShared sh;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int threads = blockDim.x, warps = threads >> 5;
    const int64_t r_at = blockIdx.x;
    const RowPlan<T> row(static_cast<const T*>(a.logits) + r_at * a.stride, a.vocab);
    const int singles = warp == 0 ? row.head + row.tail : 0;
    auto meet = [&]() {
        if (warps == 1) __syncwarp();
        else __syncthreads();
    };

    const int64_t token = a.logp ? a.tokens[r_at] : -1;
    Vec16<T> v[NV];  // past the end: -inf
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        const int w = i * threads + tid;
        v[i].u = Vec16<T>::nothing();
        if (w < row.n_vec) v[i] = load16(row.x + row.head + w * kN);
    }
    const int single_id = lane < singles ? row.single_id(lane, a.vocab) : 0;
    const float single = lane < singles ? widen1(row.x[single_id]) : -kInf;
    const float x_token = token >= 0 && token < a.vocab ? widen1(row.x[token]) : 0.0f;

    float m = fmaxf(single, -kInf);
#pragma unroll
    for (int i = 0; i < NV; ++i) m = fmaxf(m, v[i].largest());
    m = fmaxf(m, -kInf);
    float M = warp_max(m);
    if (warps > 1) {
        sh.thread_max[tid] = m;
        if (lane == 0) sh.warp_max[warp] = M;
    }
    if (tid == 0) sh.n = sh.n_vectors = 0;
    meet();
    if (warps > 1) {
        M = sh.warp_max[0];
        for (int w = 1; w < warps; ++w) M = fmaxf(M, sh.warp_max[w]);
    }

    // the sums of all warps, in their order
    auto join = [&](Share& s) {
        s.c = warp_sum(s.c), s.r = warp_sum(s.r), s.t = warp_sum(s.t);
        if (warps == 1) {
            __syncwarp();
            return;
        }
        if (lane == 0) sh.c[warp] = s.c, sh.r[warp] = s.r, sh.t[warp] = s.t;
        __syncthreads();
        s.c = s.r = s.t = 0.0f;
        for (int w = 0; w < warps; ++w) s.c += sh.c[w], s.r += sh.r[w], s.t += sh.t[w];
    };
    Share s{M, 0.0f, 0.0f, 0.0f};
    const float from = M == -kInf ? 0.0f : M;
    {
        const Pair less = pair(-from, -from), log2e = pair(kLog2e, kLog2e);
        Pair r2 = pair(0.0f, 0.0f), t2 = r2;
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            // a mask held finite: its exponent times its term is then 0 and not NaN
            const Vec16<T> u = v[i].held_finite();
#pragma unroll
            for (int j = 0; j < kN; j += 2) {
                const Pair d = add2(pair(u.get(j), u.get(j + 1)), less);
                float y0, y1;
                split(mul2(d, log2e), y0, y1);
                const Pair e = pair(ex2(y0), ex2(y1));
                r2 = add2(r2, e);
                t2 = fma2(e, d, t2);
            }
        }
        const float d = max_nan(single - from, -200.0f), e = lane < singles ? ex2(d * kLog2e) : 0.0f;
        float lo, hi;
        split(r2, lo, hi);
        s.r = lo + hi + e;
        split(t2, lo, hi);
        s.t = lo + hi + e * d;
    }

    // a bound that at least `top` logits reach, and the vectors with one that does
    float bound = M;
    if (a.top > 1) {
        float set = m;
        if (warps > 1) {
            set = sh.thread_max[lane];
            for (int w = 1; w < warps; ++w) set = fmaxf(set, sh.thread_max[32 * w + lane]);
        }
        bound = nth_of_warp(set, a.top);
    }
    auto put = [&](float x, int id) {
        const int at = atomicAdd(&sh.n, 1);
        if (at < kLhList) sh.list[at] = make_key(x, static_cast<uint32_t>(id));
    };
    auto mark = [&](auto&& wanted) {
        if (!wanted(m)) return;
        if (wanted(single) && lane < singles) put(single, single_id);
        uint32_t hits = 0;
#pragma unroll
        for (int i = 0; i < NV; ++i) hits |= wanted(v[i].largest()) ? 1u << i : 0u;
        int at = atomicAdd(&sh.n_vectors, __popc(hits));
        for (; hits != 0; hits &= hits - 1, ++at)
            if (at < kLhList)
                sh.vectors[at] = static_cast<uint16_t>((__ffs(hits) - 1) * threads + tid);
    };
    auto look_through = [&](auto&& wanted) {  // a thread to a logit, from the caches
        const int n_vectors = sh.n_vectors;
        if (n_vectors <= kLhList) {
            for (int i = tid; i < n_vectors * kN; i += threads) {
                const int id = row.head + sh.vectors[i / kN] * kN + i % kN;
                const float x = widen1(row.x[id]);
                if (wanted(x)) put(x, id);
            }
        }
        meet();
        return n_vectors <= kLhList && sh.n <= kLhList;
    };
    const auto reaches = [&](float x) { return x >= bound; };
    const auto passes = [&](float x) { return x > bound; };
    const bool list = a.top > 0 && bound > -kInf;
    if (list) mark(reaches);
    join(s);
    bool found = list && look_through(reaches);

    bool bad = false;
    if (s.r != s.r || fabsf(M) >= kHuge) {
        // a NaN, no logit, or logits too large for differences to stay finite
        s = Share{M, 0.0f, 0.0f, 0.0f};
        auto add = [&](float x) {
            if (x != x || x == kInf) s.r = NAN;
            if (x == M) {
                if (M != -kInf) s.c += 1.0f;
            } else {
                const float d = max_nan(x - from, -200.0f), e = ex2(d * kLog2e);
                s.r += e;
                s.t += e * d;
            }
        };
        if (lane < singles) add(single);
#pragma unroll 1
        for (int i = 0; i < NV; ++i) {
            const int w = i * threads + tid;
            if (w >= row.n_vec) break;
            const Vec16<T> u = load16(row.x + row.head + w * kN);
#pragma unroll
            for (int j = 0; j < kN; ++j) add(u.get(j));
        }
        meet();  // (the sums before have been read)
        join(s);
        bad = s.r != s.r;
    } else if (s.r < 1.5f) {
        // One logit has most of the probability, and what the others add to it would drown in
        // the sum: again without it.
        s = Share{M, 0.0f, 0.0f, 0.0f};
        auto add = [&](float x) {
            if (x == M) return;
            const float d = fmaxf(x - M, -200.0f), e = ex2(d * kLog2e);
            s.r += e;
            s.t += e * d;
        };
        if (lane < singles) add(single);
#pragma unroll
        for (int i = 0; i < NV; ++i)
#pragma unroll
            for (int j = 0; j < kN; ++j) add(v[i].get(j));
        meet();
        join(s);
        s.c = 1.0f;
    }
    const RowResult result(s);
    if (tid == 0) result.write(a, r_at, token, x_token);
    if (a.top == 0) return;
    if (!bad && !found) {
        // many logits equal to the bound, or masks where there are too few others: those above
        // it, and of the equal ones the first `top` in the order of ids
        meet();
        if (tid == 0) sh.n = sh.n_vectors = 0;
        meet();
        mark(passes);
        meet();
        found = look_through(passes) && sh.n <= kLhList - 32;
        meet();
        if (found && warp == 0) {
            int left = a.top - sh.n;
            for (int id0 = 0; id0 < a.vocab && left > 0; id0 += 32 * 8) {
                float x[8];
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    const int id = id0 + 32 * j + lane;
                    x[j] = id < a.vocab ? widen1(row.x[id]) : kInf;
                }
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    const uint32_t who = __ballot_sync(0xFFFFFFFFu, x[j] == bound);
                    if (x[j] == bound && __popc(who & ((1u << lane) - 1u)) < left)
                        put(x[j], id0 + 32 * j + lane);
                    left -= __popc(who);
                }
            }
        }
        meet();
    }
    if (found && !bad) {
        // a candidate's place is the number before it
        const int n = sh.n;
        for (int i = tid; i < n; i += threads) {
            const Key key = sh.list[i];
            int place = 0;
#pragma unroll 4
            for (int k = 0; k < n; ++k) place += sh.list[k] > key;
            if (place < a.top) result.write_top(a, r_at, place, key);
        }
        return;
    }
    // a NaN, or more candidates than the list holds: one maximum at a time
    Key last = ~0ull;
    for (int p = 0; p < a.top; ++p) {
        Key key = 0;
        auto look = [&](float x, int id) {
            const Key u = make_key(x, static_cast<uint32_t>(id));
            if (u < last) key = max(key, u);
        };
        if (lane < singles) look(single, single_id);
#pragma unroll 1
        for (int i = 0; i < NV; ++i) {
            const int w = i * threads + tid;
            if (w >= row.n_vec) break;
            const Vec16<T> u = load16(row.x + row.head + w * kN);
#pragma unroll
            for (int j = 0; j < kN; ++j) look(u.get(j), row.head + w * kN + j);
        }
        key = warp_max_key(key);
        if (warps > 1) {
            if (lane == 0) sh.key[warp] = key;
            __syncthreads();
            for (int w = 0; w < warps; ++w) key = max(key, sh.key[w]);
            __syncthreads();
        }
        last = key;
        if (tid == 0) result.write_top(a, r_at, p, key);
    }
}

// ---- backward ----------------------------------------------------------------

constexpr int kLbThreads = 256;
constexpr int kLbBatch = 4;   // vectors per thread in flight
constexpr int kLbBlocks = 5;  // blocks per SM that rows are cut for
constexpr float kOutOfReach = 200.0f;  // (exp(-200) < 2^-149)
// Rows whose |lse| is less go by the fma below: what rounding lse log2(e) leaves out is at most 1,
// and so is lse_lo. 2^it is a factor of their gradients, out of range from |lse| of about 2^31 on.
constexpr float kLbNear = 16777216.0f;

struct LogprobGradArgs {
    const void* logits;
    void* grad;
    int64_t stride, grad_stride;
    const int64_t* tokens;
    const float* lse;
    const float* lse_lo;
    const float* entropy;
    const float* g;
    const float* h;
    int64_t pieces;  // rows * parts
    int32_t vocab;
    int32_t parts;   // pieces per row
};

// The logits may be the gradient's own buffer, so these loads are plain ones.
template <typename T>
__device__ __forceinline__ Vec16<T> load16_rw(const T* p) {
    Vec16<T> v;
    asm volatile("ld.global.L1::no_allocate.v4.b32 {%0,%1,%2,%3}, [%4];"
                 : "=r"(v.u.x), "=r"(v.u.y), "=r"(v.u.z), "=r"(v.u.w)
                 : "l"(p)
                 : "memory");
    return v;
}

__device__ __forceinline__ uint32_t pack2(float lo, float hi) {
    const __nv_bfloat162 v = __floats2bfloat162_rn(lo, hi);
    return *reinterpret_cast<const uint32_t*>(&v);
}

__device__ __forceinline__ void store16(float* p, const float (&v)[4]) {
    *reinterpret_cast<float4*>(p) = make_float4(v[0], v[1], v[2], v[3]);
}

__device__ __forceinline__ void store16(uint16_t* p, const float (&v)[8]) {
    *reinterpret_cast<uint4*>(p) =
        make_uint4(pack2(v[0], v[1]), pack2(v[2], v[3]), pack2(v[4], v[5]), pack2(v[6], v[7]));
}

__device__ __forceinline__ void store1(float* p, float v) { *p = v; }
__device__ __forceinline__ void store1(uint16_t* p, float v) {
    *p = __bfloat16_as_ushort(__float2bfloat16_rn(v));
}

// What a row gives to all its logits.
struct GradRow {
    int64_t token;
    float lse, lse_lo, g, h, H;
};

__device__ __forceinline__ GradRow grad_row(const LogprobGradArgs& a, int64_t row) {
    GradRow r;
    r.token = a.tokens ? a.tokens[row] : -1;
    r.lse = a.lse[row];
    r.lse_lo = a.lse_lo ? a.lse_lo[row] : 0.0f;
    r.g = a.g ? a.g[row] : 0.0f;
    r.h = a.h ? a.h[row] : 0.0f;
    r.H = a.h ? a.entropy[row] : 0.0f;
    return r;
}

// A piece of a row for each TEAM threads of a block; a team has about a batch or
// two of vectors per thread: 256 threads for a long row, 32 for the shortest
// (8,192 x 2,001 bf16 11 us). Blocks that walk over many pieces, with the
// next piece's row values loaded ahead, measured 5 to 8 % slower. With
// y = (x - lse) log2(e), every logit's gradient is
//   -p (g + h (log p + H)) = 2^y (b + k y),  k = -h ln 2,  b = -(g + h H).
// y is one fma, x log2(e) - RN(lse log2(e)); what that rounding (and lse_lo)
// leaves out is the same for all logits of the row, so it goes into b and k.
// Logits more than kOutOfReach below lse, masks among them, have p = 0 in
// binary32; they are held there, because b + k y has to stay finite under any h
// for 0 times it to be 0.
template <typename T, int TEAM>
__global__ void __launch_bounds__(kLbThreads)
    token_logprobs_backward(const __grid_constant__ LogprobGradArgs a) {
    constexpr int kN = Vec16<T>::kN, team = TEAM;
    const int tid = threadIdx.x % team;
    const int64_t piece = int64_t(blockIdx.x) * (kLbThreads / team) + threadIdx.x / team;
    if (piece >= a.pieces) return;
    const int64_t row = piece / a.parts;
    const int part = static_cast<int>(piece - row * a.parts);
    GradRow r = grad_row(a, row);
    const T* x = static_cast<const T*>(a.logits) + row * a.stride;
    T* out = static_cast<T*>(a.grad) + row * a.grad_stride;
    if (r.token < 0) r.g = 0.0f;
    const float g = r.g;
    const bool zeros = (g == 0.0f && r.h == 0.0f) || r.lse == -INFINITY;
    const bool nans = !zeros && (r.lse != r.lse || (g != 0.0f && r.token >= a.vocab));

    // where the two rows are aligned alike, [0, head) and the tail singly, vectors between
    int head = a.vocab;
    if (((reinterpret_cast<uintptr_t>(x) ^ reinterpret_cast<uintptr_t>(out)) & 15) == 0)
        head = RowPlan<T>(x, a.vocab).head;
    const int n_vec = (a.vocab - head) / kN;
    const int tail = a.vocab - head - n_vec * kN;
    const int per = (n_vec + a.parts - 1) / a.parts;
    const int begin = part * per, end = min(n_vec, begin + per);

    // one logit, with care
    auto single = [&](float v) {
        if (zeros) return 0.0f;
        if (nans) return NAN;
        const float d = fmaxf((v - r.lse) - r.lse_lo, -kOutOfReach);
        return -ex2(d * kLog2e) * fmaf(r.h, d + r.H, g);
    };
    if (!zeros && !nans && fabsf(r.lse) < kLbNear) {
        const float base = -r.lse * kLog2e;
        const float off = fmaf(-r.lse, kLog2e, -base) - r.lse_lo * kLog2e;
        const float f = ex2(off);
        const float k = -f * r.h * kLn2;
        const float b = fmaf(k, off, -f * fmaf(r.h, r.H, g));
        const Pair log2e = pair(kLog2e, kLog2e), base2 = pair(base, base);
        const Pair k2 = pair(k, k), b2 = pair(b, b);
        const auto low = Vec16<T>::floor_at(r.lse - kOutOfReach);
        const int hit =  // the token among the vectors' logits
            r.token >= head ? static_cast<int>(min(r.token, int64_t(a.vocab))) - head : -kN;
        for (int v0 = begin + tid; v0 < end; v0 += team * kLbBatch) {
            Vec16<T> in[kLbBatch];
#pragma unroll
            for (int i = 0; i < kLbBatch; ++i)
                if (v0 + i * team < end)
                    in[i] = load16_rw(x + head + int64_t(v0 + i * team) * kN);
#pragma unroll
            for (int i = 0; i < kLbBatch; ++i) {
                const int v = v0 + i * team;
                if (v >= end) break;
                const Vec16<T> u = in[i].held_at(low);
                float y[kN];
#pragma unroll
                for (int j = 0; j < kN; j += 2) {
                    const Pair z = fma2(pair(u.get(j), u.get(j + 1)), log2e, base2);
                    float z0, z1;
                    split(z, z0, z1);
                    split(mul2(pair(ex2(z0), ex2(z1)), fma2(k2, z, b2)), y[j], y[j + 1]);
                }
                const int at = hit - v * kN;
                if (static_cast<unsigned>(at) < static_cast<unsigned>(kN)) {
#pragma unroll
                    for (int j = 0; j < kN; ++j) y[j] = at == j ? y[j] + g : y[j];
                }
                store16(out + head + int64_t(v) * kN, y);
            }
        }
    } else {
        for (int v = begin + tid; v < end; v += team) {
            const int id = head + v * kN;
            Vec16<T> in;
            if (!zeros) in = load16_rw(x + id);
            float y[kN];
#pragma unroll
            for (int j = 0; j < kN; ++j) y[j] = zeros ? 0.0f : single(in.get(j));
#pragma unroll
            for (int j = 0; j < kN; ++j) y[j] += !zeros && r.token == id + j ? g : 0.0f;
            store16(out + id, y);
        }
    }
    const int singles = head + tail;
    for (int i = part * team + tid; i < singles; i += a.parts * team) {
        const int id = i < head ? i : a.vocab - tail + (i - head);
        float y = zeros ? 0.0f : single(widen1(x[id]));
        if (!zeros && r.token == id) y += g;
        store1(out + id, y);
    }
}

template <typename T>
const void* held_kernel(int nv) {
    return nv <= 4   ? reinterpret_cast<const void*>(token_logprobs_held<T, 4>)
           : nv <= 8 ? reinterpret_cast<const void*>(token_logprobs_held<T, 8>)
                     : reinterpret_cast<const void*>(token_logprobs_held<T, kLhMost>);
}

template <typename T>
const void* backward_kernel(int team) {
    return team == 32    ? reinterpret_cast<const void*>(token_logprobs_backward<T, 32>)
           : team == 64  ? reinterpret_cast<const void*>(token_logprobs_backward<T, 64>)
           : team == 128 ? reinterpret_cast<const void*>(token_logprobs_backward<T, 128>)
                         : reinterpret_cast<const void*>(token_logprobs_backward<T, kLbThreads>);
}

int check_logits(const char* fn, int64_t rows, int64_t vocab, const void* logits, int64_t stride,
                 cam_dtype dtype) {
    if (rows < 0 || rows > (int64_t(1) << 27))
        return record_error(CAM_E_ARG, "%s: rows out of range", fn);
    if (vocab < 1 || vocab > CAM_LOGPROBS_MAX_VOCAB)
        return record_error(CAM_E_ARG, "%s: vocab out of range", fn);
    if (dtype != CAM_F32 && dtype != CAM_BF16)
        return record_error(CAM_E_ARG, "%s: unknown dtype %d", fn, static_cast<int>(dtype));
    if (rows > 0 && !logits) return record_error(CAM_E_ARG, "%s: logits is NULL", fn);
    if (stride < vocab || stride > (int64_t(1) << 32))
        return record_error(CAM_E_ARG, "%s: stride out of range", fn);
    if (rows > 0 && stride > (int64_t(1) << 58) / rows)
        return record_error(CAM_E_ARG, "%s: too many logits", fn);
    if (reinterpret_cast<uintptr_t>(logits) % (dtype == CAM_F32 ? 4 : 2) != 0)
        return record_error(CAM_E_ARG, "%s: logits is not aligned to its elements", fn);
    return CAM_OK;
}

}  // namespace
}  // namespace cam

using cam::record_error;

CAM_API int cam_token_logprobs(int64_t rows, int64_t vocab, const void* logits, int64_t stride,
                               cam_dtype dtype, const int64_t* tokens, int32_t top, float* logp,
                               float* entropy, float* lse, float* lse_lo, float* top_logp,
                               int64_t* top_ids, void* stream) {
    using namespace cam;
    const char* fn = "cam_token_logprobs";
    if (const int rc = check_logits(fn, rows, vocab, logits, stride, dtype)) return rc;
    if (top < 0 || top > CAM_LOGPROBS_MAX_TOP || top > vocab)
        return record_error(CAM_E_ARG, "%s: top must be in [0, min(vocab, %d)]", fn,
                            CAM_LOGPROBS_MAX_TOP);
    if (rows > 0 && logp && !tokens)
        return record_error(CAM_E_ARG, "%s: logp needs tokens", fn);
    if (rows == 0) return CAM_OK;
    int dev = 0, sms = 0;
    cudaError_t ce = current_device(&dev, &sms);
    if (ce != cudaSuccess)
        return record_error(CAM_E_CUDA, "%s: no usable CUDA device: %s", fn, cudaGetErrorString(ce));
    LogprobArgs a{logits, stride, tokens, logp, entropy, lse, lse_lo, top_logp, top_ids,
                  static_cast<int32_t>(rows), static_cast<int32_t>(vocab),
                  top_logp || top_ids ? top : 0, 1, 0, 0, 0};
    // Rows that fit the registers of a block are held there. Up to 2,048 vectors that is faster
    // for any number of rows, in us against the streaming form's, without alternatives and with
    // 20: 8,192 x 2,000 fp32 17 and 29 (29 and 66), 8,192 x 16,000 bf16 57 and 84 (70 and 117).
    // Up to 4,096 it is where rows are fewer: 512 x 32,000 bf16 13 and 17 (14 and 23); with many
    // the two are alike: 8,192 x 16,000 fp32 93 to 131 (98 to 133). Up to 8,192 it is where each
    // row has an SM: 1 x 52,000 bf16 8 and 8 (8 and 25), but 512 x 52,000 27 and 33 (19 and 29).
    const int64_t n_vec = std::max<int64_t>(1, vocab / (dtype == CAM_F32 ? 4 : 8));
    const int64_t held = 32 * kLhMaxWarps * kLhMost;
    if (n_vec <= held / 4 || (n_vec <= held / 2 && rows <= int64_t(sms) * 8) ||
        (n_vec <= held && rows <= sms)) {
        // as few warps as hold the row where rows are many, as many as still have four
        // vectors per thread where they are few
        int64_t warps = (n_vec + 32 * kLhMost - 1) / (32 * kLhMost);
        const int64_t most = std::min<int64_t>(kLhMaxWarps, (n_vec + 32 * 4 - 1) / (32 * 4));
        while (warps < most && rows * (warps + 1) <= int64_t(sms) * kLhFill) ++warps;
        const int nv = static_cast<int>((n_vec + 32 * warps - 1) / (32 * warps));
        void* held_args[] = {&a};
        ce = cudaLaunchKernel(dtype == CAM_F32 ? held_kernel<float>(nv) : held_kernel<uint16_t>(nv),
                              dim3(static_cast<unsigned>(rows)),
                              dim3(static_cast<unsigned>(32 * warps)), held_args, 0,
                              static_cast<cudaStream_t>(stream));
        if (ce != cudaSuccess)
            return record_error(CAM_E_CUDA, "%s: launch: %s", fn, cudaGetErrorString(ce));
        return CAM_OK;
    }
    // Streaming threads per block: about 16 vectors each. Where rows are few, a cluster of
    // blocks shares each of them.
    auto threads_for = [&](int64_t share) {
        return static_cast<int32_t>(
            std::min<int64_t>(kLpMaxStream, std::max<int64_t>(64, (share / 16 + 31) / 32 * 32)));
    };
    auto bytes_for = [](int32_t threads) {
        return static_cast<int>(sizeof(LogprobShared)) + kLpBufs * threads * kLpUnits * 4;
    };
    auto blocks_per_sm = [&](int32_t threads) {
        return std::min(228 * 1024 / (bytes_for(threads) + 1024),
                        1024 / (threads + 32 * kLpSelect));
    };
    a.stream = threads_for(n_vec);
    while (a.cluster < kLpMaxCluster && n_vec > int64_t(a.cluster) * 256 &&
           rows * a.cluster * 2 <= int64_t(sms) * blocks_per_sm(kLpMaxStream))
        a.cluster *= 2;
    const int64_t share = (n_vec + a.cluster - 1) / a.cluster;
    if (a.cluster > 1)  // (one row each: all of it at once)
        a.stream = static_cast<int32_t>(
            std::min<int64_t>(kLpMaxStream, std::max<int64_t>(64, (share + 31) / 32 * 32)));
    a.iters = static_cast<int32_t>((share + a.stream - 1) / a.stream);
    a.unit = (a.iters + kLpBatch * kLpUnits - 1) / (kLpBatch * kLpUnits) * kLpBatch;
    const int64_t clusters =
        a.cluster > 1 ? rows : int64_t(sms) * std::max(1, blocks_per_sm(a.stream));
    const void* kern = dtype == CAM_F32 ? reinterpret_cast<const void*>(token_logprobs<float>)
                                        : reinterpret_cast<const void*>(token_logprobs<uint16_t>);
    static std::atomic<uint64_t> shared_ok[2];
    ce = allow_shared(kern, dev, shared_ok[dtype == CAM_F32 ? 0 : 1]);
    if (ce != cudaSuccess)
        return record_error(CAM_E_CUDA, "%s: %s", fn, cudaGetErrorString(ce));
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3(static_cast<unsigned>(std::min(rows, clusters) * a.cluster));
    cfg.blockDim = dim3(a.stream + 32 * kLpSelect);
    cfg.dynamicSmemBytes = bytes_for(a.stream);
    cfg.stream = static_cast<cudaStream_t>(stream);
    cudaLaunchAttribute attr{};
    attr.id = cudaLaunchAttributeClusterDimension;
    attr.val.clusterDim.x = a.cluster;
    attr.val.clusterDim.y = attr.val.clusterDim.z = 1;
    cfg.attrs = &attr;
    cfg.numAttrs = a.cluster > 1 ? 1 : 0;
    void* args[] = {&a};
    ce = cudaLaunchKernelExC(&cfg, kern, args);
    if (ce != cudaSuccess)
        return record_error(CAM_E_CUDA, "%s: launch: %s", fn, cudaGetErrorString(ce));
    return CAM_OK;
}

CAM_API int cam_token_logprobs_backward(int64_t rows, int64_t vocab, const void* logits,
                                        int64_t stride, cam_dtype dtype, const int64_t* tokens,
                                        const float* lse, const float* lse_lo,
                                        const float* entropy,
                                        const float* grad_logp, const float* grad_entropy,
                                        void* grad_logits, int64_t grad_stride, void* stream) {
    using namespace cam;
    const char* fn = "cam_token_logprobs_backward";
    if (const int rc = check_logits(fn, rows, vocab, logits, stride, dtype)) return rc;
    if (grad_stride < vocab || grad_stride > (int64_t(1) << 32))
        return record_error(CAM_E_ARG, "%s: grad_stride out of range", fn);
    if (rows > 0 && !grad_logp && !grad_entropy)
        return record_error(CAM_E_ARG, "%s: grad_logp and grad_entropy are both NULL", fn);
    if (rows > 0 && (!lse || !grad_logits))
        return record_error(CAM_E_ARG, "%s: lse and grad_logits are required", fn);
    if (rows > 0 && grad_logp && !tokens)
        return record_error(CAM_E_ARG, "%s: grad_logp needs tokens", fn);
    if (rows > 0 && grad_entropy && !entropy)
        return record_error(CAM_E_ARG, "%s: grad_entropy needs entropy", fn);
    if (reinterpret_cast<uintptr_t>(grad_logits) % (dtype == CAM_F32 ? 4 : 2) != 0)
        return record_error(CAM_E_ARG, "%s: grad_logits is not aligned to its elements", fn);
    if (logits == grad_logits && stride != grad_stride)
        return record_error(CAM_E_ARG, "%s: in place needs equal strides", fn);
    if (rows == 0) return CAM_OK;
    int dev = 0, sms = 0;
    cudaError_t ce = current_device(&dev, &sms);
    if (ce != cudaSuccess)
        return record_error(CAM_E_CUDA, "%s: no usable CUDA device: %s", fn, cudaGetErrorString(ce));
    // A row in pieces of a few batches: fewer threads for a short row, more pieces where rows
    // are few.
    const int64_t n_vec = vocab / (dtype == CAM_F32 ? 4 : 8);
    int32_t team = kLbThreads;
    while (team > 32 && n_vec <= int64_t(team / 2) * kLbBatch) team /= 2;
    const int64_t slots = int64_t(sms) * kLbBlocks * (kLbThreads / team);
    int64_t parts = std::max<int64_t>(1, n_vec / (int64_t(team) * kLbBatch * 2));
    if (rows * parts < slots)
        parts = std::max(parts, std::min((n_vec + team - 1) / team, slots / rows));
    LogprobGradArgs a{logits, grad_logits, stride, grad_stride, tokens, lse, lse_lo, entropy,
                      grad_logp, grad_entropy, rows * parts, static_cast<int32_t>(vocab),
                      static_cast<int32_t>(parts)};
    const int64_t blocks = (a.pieces + kLbThreads / team - 1) / (kLbThreads / team);
    if (blocks > INT32_MAX) return record_error(CAM_E_ARG, "%s: too many logits", fn);
    void* args[] = {&a};
    const void* kern =
        dtype == CAM_F32 ? backward_kernel<float>(team) : backward_kernel<uint16_t>(team);
    ce = cudaLaunchKernel(kern, dim3(static_cast<unsigned>(blocks)),
                          dim3(kLbThreads), args, 0, static_cast<cudaStream_t>(stream));
    if (ce != cudaSuccess)
        return record_error(CAM_E_CUDA, "%s: launch: %s", fn, cudaGetErrorString(ce));
    return CAM_OK;
}
