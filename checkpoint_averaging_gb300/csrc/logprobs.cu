// logprobs.cu -- cam_token_logprobs and cam_token_logprobs_backward: what a
// model says of given tokens, and its gradient (declarations, definitions and
// the cases without a distribution in include/cam.h).
//
// Forward. With M = max x, r the sum of exp(x - M) over the logits below M, c
// the number of logits equal to M and t the sum of exp(x - M) (x - M):
//   log s = log1p(c - 1 + r),  lse = M + log s,
//   logp = (x_token - M) - log s,  entropy = log s - t / (c + r).
// Keeping c apart from r keeps log s exact where one token takes nearly all
// the probability. The pass reads each logit once (2 or 4 B and one
// exponential each: HBM-bound) and holds it in registers between its two
// steps, the largest logit and the sums; rows too long for a block are split
// over a cluster of up to 8 blocks, each with its own M, joined at the end.
//
// The largest `top` logits. A block has 32 groups of 16 threads, and the
// top-th largest of the groups' largest logits is a bound that at least `top`
// logits reach; the second step collects the few logits that reach it, and
// each candidate counts the candidates before it (larger, or equal with a
// lower id), which is its place. Rows with more candidates than the list
// holds (many equal logits) and rows with a NaN take one maximum at a time.
//
// Backward. One elementwise pass, read and written once (HBM-bound).
#include <cooperative_groups.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <cmath>

#include "cam_internal.h"

#define CAM_API extern "C" __attribute__((visibility("default")))

namespace cam {
namespace {

namespace cg = cooperative_groups;

constexpr int kLpThreads = 512;
constexpr int kLpWarps = kLpThreads / 32;
constexpr int kLpGroups = 32;      // groups of 16 threads
constexpr int kLpList = 1024;      // candidates a block keeps
constexpr int kLpMaxCluster = 8;
constexpr float kLog2e = 1.4426950408889634f;

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
    int32_t vocab;
    int32_t top;
    int32_t cluster;
};

__device__ __forceinline__ float ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
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
};

template <>
struct Vec16<uint16_t> {
    static constexpr int kN = 8;
    uint4 u;
    __device__ __forceinline__ float get(int j) const {
        const uint32_t w = j < 2 ? u.x : j < 4 ? u.y : j < 6 ? u.z : u.w;
        return __uint_as_float((j & 1) ? w & 0xFFFF0000u : w << 16);
    }
};

template <typename T>
__device__ __forceinline__ Vec16<T> load16(const T* p) {
    Vec16<T> v;
    asm volatile("ld.global.nc.L1::no_allocate.v4.b32 {%0,%1,%2,%3}, [%4];"
                 : "=r"(v.u.x), "=r"(v.u.y), "=r"(v.u.z), "=r"(v.u.w)
                 : "l"(p));
    return v;
}

__device__ __forceinline__ float widen1(float v) { return v; }
__device__ __forceinline__ float widen1(uint16_t v) {
    return __uint_as_float(static_cast<uint32_t>(v) << 16);
}

// A logit and its id as one whole number: larger for a larger logit (NaN
// above +inf, -0 as +0) and, among equals, for a lower id. Never 0.
__device__ __forceinline__ unsigned long long make_key(float x, uint32_t id) {
    uint32_t u = __float_as_uint(x + 0.0f);
    if ((u & 0x7FFFFFFFu) > 0x7F800000u) u = 0x7FFFFFFEu;  // (all ones stays free)
    u ^= (u >> 31) ? 0xFFFFFFFFu : 0x80000000u;
    return (static_cast<unsigned long long>(u) << 32) | (0xFFFFFFFFu - id);
}

__device__ __forceinline__ float key_logit(unsigned long long key) {
    const uint32_t u = static_cast<uint32_t>(key >> 32);
    return __uint_as_float(u ^ ((u >> 31) ? 0x80000000u : 0xFFFFFFFFu));
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
    float m;    // largest logit (NaN apart), -inf where there is none
    float c;    // logits equal to m
    float r;    // sum of exp(x - m) over the others
    float t;    // sum of exp(x - m) (x - m)
};

// T: the logits' type. NV: vectors each thread holds in registers; 0 reads
// the share from memory (its second and later readings from L2) instead.
template <typename T, int NV>
__global__ void __launch_bounds__(kLpThreads, NV > 0 && NV <= 8 ? 2 : 1)
    token_logprobs(const __grid_constant__ LogprobArgs a) {
    constexpr int kN = Vec16<T>::kN;
    constexpr float kInf = INFINITY;
    __shared__ float group_max[kLpGroups];
    __shared__ float warp_sums[3][kLpWarps];
    __shared__ unsigned long long list[kLpList];
    __shared__ unsigned long long best[kLpMaxCluster][CAM_LOGPROBS_MAX_TOP];  // the leader's
    __shared__ Share shares[kLpMaxCluster];                                   // the leader's
    __shared__ unsigned long long round_best[kLpWarps];
    __shared__ int n_listed;

    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int rank = a.cluster > 1 ? static_cast<int>(cg::this_cluster().block_rank()) : 0;
    const int64_t row = blockIdx.x / a.cluster;
    const T* x = static_cast<const T*>(a.logits) + row * a.stride;
    // [0, head) and the last `tail` logits singly, by the leader; vectors between
    const int head = min(a.vocab, static_cast<int>((16 - (reinterpret_cast<uintptr_t>(x) & 15)) & 15) /
                                      static_cast<int>(sizeof(T)));
    const int n_vec = (a.vocab - head) / kN;
    const int tail = a.vocab - head - n_vec * kN;
    const T* xv = x + head;
    const int v0 = rank * kLpThreads + tid, v_step = a.cluster * kLpThreads;

    float single = -kInf;  // this thread's single logit
    int single_id = -1;
    if (rank == 0 && tid < head + tail) {
        single_id = tid < head ? tid : a.vocab - tail + (tid - head);
        single = widen1(x[single_id]);
    }
    Vec16<T> held[NV > 0 ? NV : 1];
    if constexpr (NV > 0) {
        const uint32_t pad = sizeof(T) == 4 ? 0xFF800000u : 0xFF80FF80u;  // -inf
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            held[i].u = make_uint4(pad, pad, pad, pad);
            if (v0 + i * v_step < n_vec) held[i] = load16(xv + int64_t(v0 + i * v_step) * kN);
        }
    }
    // f(vector, id of its first logit) over this thread's vectors
    auto each = [&](auto&& f) {
        if constexpr (NV > 0) {
#pragma unroll
            for (int i = 0; i < NV; ++i)
                if (v0 + i * v_step < n_vec) f(held[i], head + (v0 + i * v_step) * kN);
        } else {
            for (int v = v0; v < n_vec; v += v_step) f(load16(xv + int64_t(v) * kN), head + v * kN);
        }
    };

    // the largest logit (fmaxf drops NaN: the sums show it)
    float m = single == single ? single : -kInf;
    each([&](const Vec16<T>& v, int) {
#pragma unroll
        for (int j = 0; j < kN; ++j) m = fmaxf(m, v.get(j));
    });
    const float mine = m;
#pragma unroll
    for (int o = 1; o < 16; o *= 2) m = fmaxf(m, __shfl_xor_sync(0xFFFFFFFFu, m, o));
    if ((lane & 15) == 0) group_max[tid >> 4] = m;
    if (tid == 0) n_listed = 0;
    __syncthreads();
    m = group_max[lane];
    float bound = kInf;
    if (a.top > 1) bound = nth_of_warp(m, a.top);
#pragma unroll
    for (int o = 1; o < 32; o *= 2) m = fmaxf(m, __shfl_xor_sync(0xFFFFFFFFu, m, o));
    if (a.top == 1) bound = m;
    const float zero = m == -kInf ? 0.0f : m;  // what to subtract

    // the sums, and the logits that reach the bound
    float c = 0.0f, r = 0.0f, t = 0.0f;
    auto put = [&](float v, int id) {
        const int at = atomicAdd(&n_listed, 1);
        if (at < kLpList) list[at] = make_key(v, static_cast<uint32_t>(id));
    };
    auto add = [&](float v, bool may_be_largest) {
        const float d = v - zero;
        const float e = ex2(d * kLog2e);
        if (may_be_largest && v == m) {
            if (m != -kInf) c += 1.0f;
        } else {
            r += e;
            t = fmaf(e, fmaxf(d, -1e30f), t);  // 0 for a logit of -inf
        }
    };
    if (mine == m) {
        each([&](const Vec16<T>& v, int) {
#pragma unroll
            for (int j = 0; j < kN; ++j) add(v.get(j), true);
        });
    } else {
        each([&](const Vec16<T>& v, int) {
#pragma unroll
            for (int j = 0; j < kN; ++j) add(v.get(j), false);
        });
    }
    if (single_id >= 0) add(single, true);
    if (a.top > 0 && mine >= bound) {
        each([&](const Vec16<T>& v, int id) {
#pragma unroll
            for (int j = 0; j < kN; ++j)
                if (v.get(j) >= bound) put(v.get(j), id + j);
        });
        if (single_id >= 0 && single >= bound) put(single, single_id);
    }
#pragma unroll
    for (int o = 16; o > 0; o /= 2) {
        c += __shfl_xor_sync(0xFFFFFFFFu, c, o);
        r += __shfl_xor_sync(0xFFFFFFFFu, r, o);
        t += __shfl_xor_sync(0xFFFFFFFFu, t, o);
    }
    if (lane == 0) warp_sums[0][warp] = c, warp_sums[1][warp] = r, warp_sums[2][warp] = t;
    __syncthreads();
    c = r = t = 0.0f;
#pragma unroll
    for (int w = 0; w < kLpWarps; ++w)
        c += warp_sums[0][w], r += warp_sums[1][w], t += warp_sums[2][w];

    cg::cluster_group cluster = cg::this_cluster();
    unsigned long long* places =
        a.cluster > 1 ? cluster.map_shared_rank(&best[rank][0], 0) : &best[0][0];
    if (a.cluster > 1) {
        cluster.sync();  // the leader has started
        if (tid == 0) *cluster.map_shared_rank(&shares[rank], 0) = Share{m, c, r, t};
    } else if (tid == 0) {
        shares[0] = Share{m, c, r, t};
    }

    // the block's own largest, in order
    const int n = n_listed;
    if (a.top > 0) {
        if (n <= kLpList && r == r) {
            if (tid < a.top && tid >= n) places[tid] = 0;
            for (int i = tid; i < n; i += kLpThreads) {
                const unsigned long long key = list[i];
                int place = 0;
                for (int k = 0; k < n; ++k) place += list[k] > key;
                if (place < a.top) places[place] = key;
            }
        } else {
            unsigned long long last = ~0ull;
            for (int k = 0; k < a.top; ++k) {
                unsigned long long key = 0;
                auto look = [&](float v, int id) {
                    const unsigned long long u = make_key(v, static_cast<uint32_t>(id));
                    if (u < last && u > key) key = u;
                };
                each([&](const Vec16<T>& v, int id) {
#pragma unroll
                    for (int j = 0; j < kN; ++j) look(v.get(j), id + j);
                });
                if (single_id >= 0) look(single, single_id);
#pragma unroll
                for (int o = 16; o > 0; o /= 2)
                    key = max(key, __shfl_xor_sync(0xFFFFFFFFu, key, o));
                __syncthreads();
                if (lane == 0) round_best[warp] = key;
                __syncthreads();
#pragma unroll
                for (int w = 0; w < kLpWarps; ++w) key = max(key, round_best[w]);
                if (tid == 0) places[k] = key;
                last = key;
                if (key == 0) last = 1;  // none left: nothing is below 1 but 0
            }
        }
    }
    if (a.cluster > 1) cluster.sync();
    else __syncthreads();
    if (rank != 0) return;

    // the row, from its shares
    float M = -kInf;
    for (int k = 0; k < a.cluster; ++k) M = fmaxf(M, shares[k].m);
    c = r = t = 0.0f;
    for (int k = 0; k < a.cluster; ++k) {
        const Share s = shares[k];
        if (s.m == M) {
            c += s.c, r += s.r, t += s.t;
        } else {
            const float d = fmaxf(s.m - M, -1e30f), e = ex2(d * kLog2e);
            r += e * (s.c + s.r);
            t += e * (s.t + d * (s.c + s.r));
        }
    }
    if (M == kInf) r = NAN;
    // no distribution: c and r are 0; a NaN or +inf: r is NaN
    const bool dead = M == -kInf && r == 0.0f;
    const float log_s = dead ? 0.0f : log1pf((c - 1.0f) + r);
    auto logp_of = [&](float v) { return dead ? -kInf : (v - M) - log_s; };
    if (tid == 0) {
        const float lse = dead ? -kInf : M + log_s;
        if (a.lse) a.lse[row] = lse;
        if (a.lse_lo) {  // what the sum's rounding left out, exactly (no order of the two is needed)
            const float b = __fsub_rn(lse, M);
            const float lo = __fadd_rn(__fsub_rn(M, __fsub_rn(lse, b)), __fsub_rn(log_s, b));
            a.lse_lo[row] = isfinite(lse) ? lo : 0.0f;
        }
        if (a.entropy) a.entropy[row] = dead ? 0.0f : log_s - t / (c + r);
        if (a.logp) {
            const int64_t token = a.tokens[row];
            float p = 0.0f;
            if (token >= a.vocab) p = NAN;
            else if (token >= 0) p = logp_of(widen1(x[token]));
            a.logp[row] = p;
        }
    }
    if (a.top > 0) {
        const unsigned long long* all = &best[0][0];
        for (int i = tid; i < a.cluster * a.top; i += kLpThreads) {
            const unsigned long long key = all[i / a.top * CAM_LOGPROBS_MAX_TOP + i % a.top];
            if (key == 0) continue;
            int place = 0;
            for (int k = 0; k < a.cluster; ++k)
                for (int j = 0; j < a.top; ++j) place += all[k * CAM_LOGPROBS_MAX_TOP + j] > key;
            if (place >= a.top) continue;
            if (a.top_ids)
                a.top_ids[row * a.top + place] = 0xFFFFFFFFu - static_cast<uint32_t>(key);
            if (a.top_logp) a.top_logp[row * a.top + place] = logp_of(key_logit(key));
        }
    }
}

// ---- backward ----------------------------------------------------------------

constexpr int kLbThreads = 256;
constexpr int kLbSteps = 4;  // vectors per thread and block, all in flight

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
    int32_t vocab;
    int32_t parts;  // blocks per row
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

template <typename T>
__global__ void __launch_bounds__(kLbThreads)
    token_logprobs_backward(const __grid_constant__ LogprobGradArgs a) {
    constexpr int kN = Vec16<T>::kN;
    const int64_t row = blockIdx.x / a.parts;
    const int part = static_cast<int>(blockIdx.x % a.parts);
    const T* x = static_cast<const T*>(a.logits) + row * a.stride;
    T* out = static_cast<T*>(a.grad) + row * a.grad_stride;
    const int64_t token = a.tokens ? a.tokens[row] : -1;
    const float lse = a.lse[row], lse_lo = a.lse_lo ? a.lse_lo[row] : 0.0f;
    const float g = a.g && token >= 0 ? a.g[row] : 0.0f;
    const float h = a.h ? a.h[row] : 0.0f;
    const float H = h != 0.0f ? a.entropy[row] : 0.0f;
    const bool zeros = (g == 0.0f && h == 0.0f) || lse == -INFINITY;
    const bool nans = !zeros && (lse != lse || token >= a.vocab);

    // where the two rows are aligned alike, [0, head) and the tail singly and vectors between
    int head = a.vocab;
    if (((reinterpret_cast<uintptr_t>(x) ^ reinterpret_cast<uintptr_t>(out)) & 15) == 0)
        head = min(a.vocab, static_cast<int>((16 - (reinterpret_cast<uintptr_t>(x) & 15)) & 15) /
                                static_cast<int>(sizeof(T)));
    const int n_vec = (a.vocab - head) / kN;
    const int tail = a.vocab - head - n_vec * kN;
    // -p (g + h (log p + H)); log p of a logit of -inf is held finite, p is 0
    auto value = [&](float v) {
        if (zeros) return 0.0f;
        if (nans) return NAN;
        const float d = fmaxf((v - lse) - lse_lo, -1e30f);
        return -ex2(d * kLog2e) * fmaf(h, d + H, g);
    };

    const int per = (n_vec + a.parts - 1) / a.parts;
    const int end = min(n_vec, (part + 1) * per);
    for (int v0 = part * per + threadIdx.x; v0 < end; v0 += kLbThreads * kLbSteps) {
        Vec16<T> in[kLbSteps];
        if (!zeros) {
#pragma unroll
            for (int i = 0; i < kLbSteps; ++i)
                if (v0 + i * kLbThreads < end)
                    in[i] = load16_rw(x + head + int64_t(v0 + i * kLbThreads) * kN);
        }
#pragma unroll
        for (int i = 0; i < kLbSteps; ++i) {
            const int v = v0 + i * kLbThreads;
            if (v >= end) break;
            const int id = head + v * kN;
            float y[kN];
#pragma unroll
            for (int j = 0; j < kN; ++j) y[j] = zeros ? 0.0f : value(in[i].get(j));
            if (!zeros && token >= id && token < id + kN) {
#pragma unroll
                for (int j = 0; j < kN; ++j)
                    if (token == id + j) y[j] += g;
            }
            store16(out + id, y);
        }
    }
    const int singles = head + tail;
    for (int i = part * kLbThreads + threadIdx.x; i < singles; i += a.parts * kLbThreads) {
        const int id = i < head ? i : a.vocab - tail + (i - head);
        float y = zeros ? 0.0f : value(widen1(x[id]));
        if (!zeros && token == id) y += g;
        store1(out + id, y);
    }
}

template <typename T>
const void* forward_kernel(int nv) {
    return nv == 0   ? reinterpret_cast<const void*>(token_logprobs<T, 0>)
           : nv <= 2 ? reinterpret_cast<const void*>(token_logprobs<T, 2>)
           : nv <= 5 ? reinterpret_cast<const void*>(token_logprobs<T, 5>)
                     : reinterpret_cast<const void*>(token_logprobs<T, 8>);
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
    cudaError_t ce = cudaGetDevice(&dev);
    if (ce == cudaSuccess) ce = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
    if (ce != cudaSuccess)
        return record_error(CAM_E_CUDA, "%s: no usable CUDA device: %s", fn, cudaGetErrorString(ce));
    LogprobArgs a{logits, stride, tokens, logp, entropy, lse, lse_lo, top_logp, top_ids,
                  static_cast<int32_t>(vocab), top_logp || top_ids ? top : 0, 1};
    // blocks per row: enough that a share fits the registers, and more while SMs idle
    const int kn = dtype == CAM_F32 ? 4 : 8;
    const int64_t n_vec = vocab / kn;
    while (a.cluster < kLpMaxCluster &&
           (n_vec > int64_t(a.cluster) * kLpThreads * 5 ||
            (rows * a.cluster * 2 <= sms && n_vec > int64_t(a.cluster) * kLpThreads)))
        a.cluster *= 2;
    int64_t nv = (n_vec + int64_t(a.cluster) * kLpThreads - 1) / (int64_t(a.cluster) * kLpThreads);
    if (nv > 8) nv = 0;
    else if (nv == 0) nv = 1;
    const void* kern = dtype == CAM_F32 ? forward_kernel<float>(static_cast<int>(nv))
                                        : forward_kernel<uint16_t>(static_cast<int>(nv));
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3(static_cast<unsigned>(rows * a.cluster));
    cfg.blockDim = dim3(kLpThreads);
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
    const int kn = dtype == CAM_F32 ? 4 : 8;
    const int64_t span = int64_t(kLbThreads) * kLbSteps * kn;
    LogprobGradArgs a{logits, grad_logits, stride, grad_stride, tokens, lse, lse_lo, entropy,
                      grad_logp, grad_entropy, static_cast<int32_t>(vocab),
                      static_cast<int32_t>((vocab + span - 1) / span)};
    if (rows * a.parts > INT32_MAX) return record_error(CAM_E_ARG, "%s: too many logits", fn);
    void* args[] = {&a};
    const void* kern = dtype == CAM_F32
                           ? reinterpret_cast<const void*>(token_logprobs_backward<float>)
                           : reinterpret_cast<const void*>(token_logprobs_backward<uint16_t>);
    const cudaError_t ce =
        cudaLaunchKernel(kern, dim3(static_cast<unsigned>(rows * a.parts)), dim3(kLbThreads), args, 0,
                         static_cast<cudaStream_t>(stream));
    if (ce != cudaSuccess)
        return record_error(CAM_E_CUDA, "%s: launch: %s", fn, cudaGetErrorString(ce));
    return CAM_OK;
}
