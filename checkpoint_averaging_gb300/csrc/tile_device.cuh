// tile_device.cuh -- what the kernels of the operators for whole contexts share on the
// device: issuing by one lane, results through TMA, softmax statistics and gradients of
// logits, and the encoding of tensor maps.
#pragma once

#include <cuda_bf16.h>

#include <climits>
#include <cstdint>

#include "tc_device.cuh"
#include "tile_products.h"

namespace cam {
namespace tc {
namespace {

// A warp's buffer for results: two boxes of 32 rows of 64 bytes, which TMA stores; or, where
// rows do not start on 16 bytes, 32 rows of 16 words and one more between rows, so that a
// column's words lie in as many banks.
constexpr int kBox = 32 * 64;
constexpr int kTurn = 17;
static_assert(32 * kTurn * 4 <= 2 * kBox, "both forms share the buffer");

// One lane of the warp, in a form that the compiler knows for one: what it issues there
// (TMA, MMA) takes its operands from uniform registers without a loop over the lanes
// (2,048 x 38,912 logits of width 2,048: 257 us with a comparison of lanes, 196 with this).
__device__ __forceinline__ bool elect_one() {
    uint32_t p;
    asm volatile(
        "{\n\t.reg .pred q;\n\telect.sync _|q, 0xFFFFFFFF;\n\tselp.u32 %0, 1, 0, q;\n\t}"
        : "=r"(p));
    return p != 0;
}

// 16 consecutive fp32 columns of this thread's TMEM lane.
__device__ __forceinline__ void tmem_ld16(uint32_t taddr, float* v) {
    uint32_t r[16];
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x16.b32 "
        "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]),
          "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]),
          "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
        : "r"(taddr)
        : "memory");
    asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
#pragma unroll
    for (int i = 0; i < 16; ++i) v[i] = __uint_as_float(r[i]);
}

// ---- terms ---------------------------------------------------------------------------

// The nearest bf16, but the largest one where that would be an infinity.
__device__ __forceinline__ __nv_bfloat16 term(float x) {
    __nv_bfloat16 h = __float2bfloat16_rn(x);
    if ((__bfloat16_as_ushort(h) & 0x7FFFu) == 0x7F80u && isfinite(x)) h = __float2bfloat16_rz(x);
    return h;
}

// ---- epilogues -------------------------------------------------------------------------

__device__ __forceinline__ uint32_t bf16x2(float lo, float hi) {
    const __nv_bfloat162 h = __floats2bfloat162_rn(lo, hi);
    return *reinterpret_cast<const uint32_t*>(&h);
}

// 64 bytes of each of 32 rows, this lane's in w, to the box at (x, y, z) by TMA: rows and
// columns past the matrix are left out. (Stored by the threads themselves, a row each, a
// 32-byte store of a warp is 32 passes of the load/store unit.)
__device__ __forceinline__ void store_box(const CUtensorMap* map, uint32_t buf, int& which,
                                          const uint32_t* w, int lane, int x, int y, int z, bool add) {
    if (elect_one()) bulk_wait_read1();  // the box before the last has been read
    __syncwarp();
    const uint32_t box = buf + which * kBox, row = box + lane * 64;
#pragma unroll
    for (int q = 0; q < 4; ++q)
        asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(row + 16 * (q ^ ((lane >> 1) & 3))),
                     "r"(w[4 * q]), "r"(w[4 * q + 1]), "r"(w[4 * q + 2]), "r"(w[4 * q + 3])
                     : "memory");
    fence_async_smem();
    __syncwarp();
    if (elect_one()) {
        if (add)
            asm volatile(
                "cp.reduce.async.bulk.tensor.3d.global.shared::cta.add.tile.bulk_group "
                "[%0, {%2, %3, %4}], [%1];" ::"l"(reinterpret_cast<uint64_t>(map)),
                "r"(box), "r"(x), "r"(y), "r"(z)
                : "memory");
        else
            tma_store(map, box, x, y, z);
        bulk_commit();
    }
    which ^= 1;
}

// 32 columns of 32 rows, this lane's row in v, as bf16 or fp32.
__device__ __forceinline__ void store_bf16(const CUtensorMap* map, uint32_t buf, int& which,
                                           const float* v, int lane, int x, int y, int z) {
    uint32_t w[16];
#pragma unroll
    for (int i = 0; i < 16; ++i) w[i] = bf16x2(v[2 * i], v[2 * i + 1]);
    store_box(map, buf, which, w, lane, x, y, z, false);
}
__device__ __forceinline__ void store_f32(const CUtensorMap* map, uint32_t buf, int& which,
                                          const float* v, int n, int lane, int x, int y, int z,
                                          bool add) {
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        if (16 * h >= n) break;
        uint32_t w[16];
#pragma unroll
        for (int i = 0; i < 16; ++i) w[i] = __float_as_uint(v[16 * h + i]);
        store_box(map, buf, which, w, lane, x + 16 * h, y, z, add);
    }
}

// 32 columns of 32 rows, this lane's row in v, to addresses of any alignment: turned in shared
// memory so that half a warp writes 16 columns of one row (5,003 fp32 columns: a warp's store
// takes 4 sectors of memory instead of 32).
template <typename T>
__device__ __forceinline__ void store_turned(float* buf, T* y, int64_t ldy, const float* v, int rows,
                                             int n, int lane) {
    const int c = lane & 15, odd = lane >> 4;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        __syncwarp();
#pragma unroll
        for (int i = 0; i < 16; ++i) buf[lane * kTurn + i] = v[16 * h + i];
        __syncwarp();
        if (16 * h + c < n) {
#pragma unroll 8
            for (int r = odd; r < 32; r += 2)
                if (r < rows) y[r * ldy + 16 * h + c] = T(buf[r * kTurn + c]);
        }
    }
}

__device__ __forceinline__ float exp2_fast(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// log2(e) in two binary32 numbers.
constexpr double kLog2eExact = 1.4426950408889634074;
constexpr float kLog2e = static_cast<float>(kLog2eExact);
constexpr float kLog2eRest = static_cast<float>(kLog2eExact - static_cast<double>(kLog2e));
constexpr float kLn2 = 0.69314718055994530942f;

// exp(d + rest) = 2^t 2^c: t is d log2(e) rounded, c what rounding that product (an fma gives it),
// log2(e) itself, and `rest` leave of the exponent (all matter in fp32 gradients: 2^-24 of an
// argument of 20 is 1e-6 of the exponential); 2^c is 1 + c ln 2.
__device__ __forceinline__ float exp_exact(float d, float rest) {
    const float t = d * kLog2e;
    const float c = fmaf(d, kLog2e, -t) + fmaf(d, kLog2eRest, rest * kLog2e);
    const float e = exp2_fast(t);
    return fmaf(e, c * kLn2, e);
}

// 1 - exp(d) for d near 0 and below, p = exp(d): the Taylor series of exp(d) - 1 where the
// difference would cancel (its next term is below 2^-30 of the sum there).
__device__ __forceinline__ float one_minus_exp(float d, float p) {
    if (!(d > -0.35f)) return 1.0f - p;
    float s = fmaf(d, 1.0f / 8, 1.0f);
    s = fmaf(d * (1.0f / 7), s, 1.0f);
    s = fmaf(d * (1.0f / 6), s, 1.0f);
    s = fmaf(d * (1.0f / 5), s, 1.0f);
    s = fmaf(d * (1.0f / 4), s, 1.0f);
    s = fmaf(d * (1.0f / 3), s, 1.0f);
    s = fmaf(d * (1.0f / 2), s, 1.0f);
    return -d * s;
}

// What a row of logits brings to its gradient g (1[j = token] - p_j) - h p_j (log p_j + H).
struct GradRow {
    float lse, lo;  // log p = (x - lse) - lo
    float g, h, H;
    float shift;  // the quick form, d = x - lse: p = 2^(d log2(e) - shift), G = -p h d - p base
    float base;
    float far, far_lo;  // what near() takes off the row's logits
    int32_t token;  // its column (the row of D for few rows), or -1
};

// exp_exact takes what is left over as a first-order term, the square of half of which has to be
// below 2^-24: lo is up to 2^-12 for an lse of 2^13, and a half at 2^23. Rows beyond have lse and
// lo taken off their logits first, which then are log p, off by 2^-24 of itself (the logits
// there are rounded by more).
constexpr float kFar = 8192.0f;
__device__ __forceinline__ float near(float x, const GradRow& r) { return (x - r.far) - r.far_lo; }

__device__ __forceinline__ GradRow grad_row(const TileOut& o, int64_t row, int64_t n) {
    GradRow r;
    const int64_t token = o.tokens ? o.tokens[row] : -1;
    r.lse = o.lse[row];
    r.lo = o.lse_lo ? o.lse_lo[row] : 0.0f;
    r.g = o.g && token >= 0 ? o.g[row] : 0.0f;
    r.h = o.h ? o.h[row] : 0.0f;
    r.H = o.h ? o.entropy[row] : 0.0f;
    // (a token that the vocabulary does not have)
    if (r.g != 0.0f && token >= o.vocab) r.lse = __int_as_float(0x7FC00000);
    // no gradient: zeros, whatever lse is (the row's logits are zeros: head.cu)
    if (r.g == 0.0f && r.h == 0.0f) r.lse = r.lo = r.H = 0.0f;
    r.far = r.far_lo = 0.0f;
    if (fabsf(r.lse) > kFar) {
        r.far = r.lse, r.far_lo = r.lo;
        r.lse = r.lo = 0.0f;
    }
    r.shift = r.lo * kLog2e;
    r.base = fmaf(r.h, r.H - r.lo, r.g);
    const int64_t at = token - o.token0;
    r.token = at >= 0 && at < n ? static_cast<int32_t>(at) : -1;
    return r;
}

// log p no lower than where p is 0 (and NaN where it is NaN): a masked logit, the type's lowest
// value, times log2(e) or h is an infinity, and 0 times that a NaN. (1 % of fp32 gradients of 1,023
// rows over 50,304 x 128; selecting 0 for a p of 0 took 5 %.)
__device__ __forceinline__ float held(float d) {
    float y;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(y) : "f"(d), "f"(-8192.0f));
    return y;
}

// The gradient of the logit of the row's own token. Where p is near 1 it is what x and lse
// differ by: x is the sum that lse was taken from, of the same terms in the same order, so that
// what the tensor core lost of it is in both. (An exact x beside that lse: 1 - p of 1e-7 comes
// out as -1e-5 for logits of 25.)
__device__ __forceinline__ float own_grad(float x, const GradRow& r) {
    const float d = held((x - r.lse) - r.lo), p = exp_exact(d, 0.0f);
    return r.g * one_minus_exp(d, p) - r.h * p * (d + r.H);
}

// That of another's. FINE: for fp32 results, with all that matters there of d's rounding.
// Otherwise p is off by 2^-23 of log p, a hundredth of what rounding G to bf16 costs; near
// p = 1, where log p + H is far smaller than lse, d is exact.
template <bool FINE>
__device__ __forceinline__ float other_grad(float x, const GradRow& r) {
    if constexpr (FINE) {
        float d = x - r.lse;
        const float b = x - d;  // (x - lse) - d, exactly: two-sum
        const float rest = ((x - (d + b)) + (b - r.lse)) - r.lo;
        d = held(d);
        const float p = exp_exact(d, rest);
        return -p * fmaf(r.h, (d + rest) + r.H, r.g);
    } else {  // (p h first: h d may be an infinity where p is 0)
        const float d = x - r.lse, p = exp2_fast(fmaf(d, kLog2e, -r.shift));
        return fmaf(-(p * r.h), d, -(p * r.base));
    }
}

// The element of 32 at a place known at run time.
__device__ __forceinline__ float pick(const float* v, int64_t at) {
    float x = v[0];
#pragma unroll
    for (int i = 1; i < 32; ++i) x = at == i ? v[i] : x;
    return x;
}

__device__ __forceinline__ void put(float* v, int at, float x) {
#pragma unroll
    for (int i = 0; i < 32; ++i) v[i] = at == i ? x : v[i];
}

// Two fp32 values in one register pair: one instruction adds or multiplies both.
__device__ __forceinline__ uint64_t two(float x, float y) {
    uint64_t r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(x), "f"(y));
    return r;
}
__device__ __forceinline__ void halves(uint64_t v, float& x, float& y) {
    asm("mov.b64 {%0, %1}, %2;" : "=f"(x), "=f"(y) : "l"(v));
}
__device__ __forceinline__ uint64_t add2(uint64_t x, uint64_t y) {
    uint64_t r;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(x), "l"(y));
    return r;
}
__device__ __forceinline__ uint64_t mul2(uint64_t x, uint64_t y) {
    uint64_t r;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(x), "l"(y));
    return r;
}
__device__ __forceinline__ uint64_t fma2(uint64_t x, uint64_t y, uint64_t z) {
    uint64_t r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(x), "l"(y), "l"(z));
    return r;
}

// A row's statistics over a tile's columns, 32 at a time. The exponentials are relative to
// the largest logit so far, whose own is left out of their sum: where it has nearly all of the
// probability (less than 2^-8 of it elsewhere in its 32) the others are summed again without
// it, so that their share keeps its precision; elsewhere it is subtracted.
struct RowStat {
    float m, a, t;
    __device__ __forceinline__ void add(const float* v, int n, bool first) {
        float top = v[0];
#pragma unroll
        for (int i = 1; i < 32; ++i) top = i < n ? fmaxf(top, v[i]) : top;
        const bool leads = first || top > m;
        float before = 0.0f, t_before = 0.0f;  // what there was, relative to the new largest
        if (!first) {
            before = a;
            t_before = t;
            if (leads) {
                const float d = m - top, f = exp2_fast(d * kLog2e);
                t_before = f * (f > 0.0f ? fmaf(d, 1.0f + a, t) : t);  // (as in join)
                before = (1.0f + a) * f;
            }
        }
        if (leads) m = top;
        float sum, ts;
        if (n == 32) {
            const uint64_t back = two(-m, -m), scale = two(kLog2e, kLog2e);
            uint64_t s2[2] = {0, 0}, t2[2] = {0, 0};
#pragma unroll
            for (int i = 0; i < 32; i += 2) {
                const uint64_t d = add2(two(v[i], v[i + 1]), back), p = mul2(d, scale);
                float x, y;
                halves(p, x, y);
                const uint64_t e = two(exp2_fast(x), exp2_fast(y));
                s2[i >> 1 & 1] = add2(s2[i >> 1 & 1], e);
                // (NaN wherever a logit is NaN or infinite: through t)
                t2[i >> 1 & 1] = fma2(e, d, t2[i >> 1 & 1]);
            }
            float x, y;
            halves(add2(s2[0], s2[1]), x, y);
            sum = x + y;
            halves(add2(t2[0], t2[1]), x, y);
            ts = x + y;
        } else {
            sum = ts = 0.0f;
#pragma unroll
            for (int i = 0; i < 32; ++i) {
                if (i >= n) break;
                const float d = v[i] - m, e = exp2_fast(d * kLog2e);
                sum += e;
                ts = fmaf(e, d, ts);
            }
        }
        if (leads) {
            sum -= 1.0f;
            if (sum < 0x1p-8f) {
                sum = 0.0f;
                bool seen = false;
#pragma unroll
                for (int i = 0; i < 32; ++i) {
                    if (i >= n) break;
                    const float d = v[i] - m;
                    const bool own = !seen && d == 0.0f;
                    seen = seen || own;
                    sum += own ? 0.0f : exp2_fast(d * kLog2e);
                }
            }
        }
        a = before + sum;
        t = t_before + ts;
    }
};

// ---- few rows: the vocabulary along the lanes, the rows along the columns ----------------

// Sums of 32 values over the lanes, value i's in lane i: at each step a lane keeps half of
// its values and adds the other lane's of those.
__device__ __forceinline__ float sums_to_lanes(float* v, int lane) {
#pragma unroll
    for (int by = 16; by >= 1; by /= 2) {
        const bool upper = lane & by;
#pragma unroll
        for (int j = 0; j < by; ++j) {
            const float away = upper ? v[j] : v[j + by], keep = upper ? v[j + by] : v[j];
            v[j] = keep + __shfl_xor_sync(0xFFFFFFFFu, away, by);
        }
    }
    return v[0];
}

// Statistics of up to 32 rows of logits (v: this lane's logit of each) over 32 tokens of the
// vocabulary.
__device__ __forceinline__ void few_stats(const TileOut& o, int64_t M, int64_t N, float* v,
                                          int64_t row0, int64_t col0, bool in, int lane) {
    const int n = N - col0 < 32 ? int(N - col0) : 32;
    // the logits of the rows' tokens: each is met by one warp
    const int64_t token = lane < n && o.tokens ? o.tokens[col0 + lane] - o.token0 - row0 : -1;
    uint32_t here = __ballot_sync(0xFFFFFFFFu, token >= 0 && token < 32 && row0 + token < M);
    while (here) {
        const int i = __ffs(here) - 1;
        here &= here - 1;
        const int at = __shfl_sync(0xFFFFFFFFu, static_cast<int>(token), i);
        const float x = pick(v, i);
        if (lane == at) o.mine[col0 + i] = x;
    }
    float t[32], m = 0.0f, c = 0.0f;
#pragma unroll
    for (int i = 0; i < 32; ++i) {
        t[i] = 0.0f;
        if (i < n) {
            // the largest, by an order of the bits as whole numbers
            const int bits = __float_as_int(v[i]);
            const int key = in ? bits ^ ((bits >> 31) & 0x7FFFFFFF) : INT_MIN;
            const int top_key = __reduce_max_sync(0xFFFFFFFFu, key);
            const float top = __int_as_float(top_key ^ ((top_key >> 31) & 0x7FFFFFFF));
            const float d = v[i] - top, e = exp2_fast(d * kLog2e);
            const bool below = d < 0.0f;
            const uint32_t equal = __ballot_sync(0xFFFFFFFFu, in && !below);
            if (lane == i) {
                m = top;
                c = static_cast<float>(__popc(equal)) - 1.0f;
            }
            t[i] = in ? e * d : 0.0f;
            v[i] = in && below ? e : 0.0f;
        } else {
            v[i] = 0.0f;
        }
    }
    const float a = sums_to_lanes(v, lane), s = sums_to_lanes(t, lane);
    if (lane < n) o.stats[row0 / 32 * N + col0 + lane] = TileStat{m, a + c, s, 1.0f};
}

// The gradient of one token's logits in up to 32 rows.
__device__ __forceinline__ void few_grad(const TileOut& o, int64_t N, const GradRow* rows, float* v,
                                         int64_t token, int64_t col0, bool in) {
    const int n = N - col0 < 32 ? int(N - col0) : 32;
    const int lane = threadIdx.x & 31;
    if (__any_sync(0xFFFFFFFFu, lane < n && rows[lane].far != 0.0f)) {
#pragma unroll
        for (int i = 0; i < 32; ++i)
            if (i < n) v[i] = near(v[i], rows[i]);
    }
    uint32_t own = 0;  // the rows whose token this is
#pragma unroll
    for (int i = 0; i < 32; ++i)
        if (i < n && rows[i].token == int(token)) own |= 1u << i;
    for (uint32_t left = own; left; left &= left - 1) {
        const int i = __ffs(left) - 1;
        put(v, i, own_grad(pick(v, i), rows[i]));
    }
    const bool three = o.planes == 3;
#pragma unroll
    for (int i = 0; i < 32; ++i) {
        if (i >= n) {
            v[i] = 0.0f;
        } else {
            const float w = three ? other_grad<true>(v[i], rows[i]) : other_grad<false>(v[i], rows[i]);
            v[i] = own >> i & 1 ? v[i] : w;
        }
    }
    if (!in) return;
    __nv_bfloat16* y = static_cast<__nv_bfloat16*>(o.y) + token * o.ldy + col0;
    for (int k = 0; k < o.planes; ++k) {
#pragma unroll
        for (int j = 0; j < 32; j += 8) {
            if (j >= n) break;
            uint32_t w[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) w[i] = bf16x2(v[j + 2 * i], v[j + 2 * i + 1]);
            *reinterpret_cast<uint4*>(y + k * o.plane_stride + j) = make_uint4(w[0], w[1], w[2], w[3]);
        }
#pragma unroll
        for (int i = 0; i < 32; ++i) v[i] -= __bfloat162float(__float2bfloat16_rn(v[i]));
    }
}

// ---- host side ----

inline bool encode(CUtensorMap* map, CUtensorMapDataType type, const void* base, int64_t x, int64_t y,
            int64_t z, int64_t y_bytes, int64_t z_bytes, int box_x, int box_y,
            CUtensorMapSwizzle swizzle, int box_z = 1) {
    const auto enc = encoder();
    if (!enc) return false;
    if (z == 1) z_bytes = y_bytes;  // (of no use, but below the limit)
    const cuuint64_t dims[3] = {cuuint64_t(x), cuuint64_t(y), cuuint64_t(z)};
    const cuuint64_t strides[2] = {cuuint64_t(y_bytes), cuuint64_t(z_bytes)};
    const cuuint32_t box[3] = {cuuint32_t(box_x), cuuint32_t(box_y), cuuint32_t(box_z)};
    const cuuint32_t unit[3] = {1, 1, 1};
    return enc(map, type, 3, const_cast<void*>(base), dims, strides, box, unit,
               CU_TENSOR_MAP_INTERLEAVE_NONE, swizzle, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
               CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

}  // namespace
}  // namespace tc
}  // namespace cam
