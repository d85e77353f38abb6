// tile_products.h -- products of long rows on the fifth-generation tensor
// cores with an epilogue of the caller's choice, for the operators beside the
// merge: ragged extents, operands in one to three bf16 terms or in e4m3 with
// scales, either majorness, products split along K.
//
//     D[i][j] = sum over term pairs (a, b), sum_k A_a[i][k] * B_b[j][k]
#pragma once

#include <cuda_runtime.h>

#include <cstdint>

namespace cam {

// The terms of a matrix: planes of rows x k elements (k contiguous) or, MN-major, of
// k x rows (rows contiguous). bf16 by default; e4m3 operands have one plane of
// bytes and `scales` (see pack8_layout.h).
struct TileOperand {
    const void* base;
    int64_t rows, k;
    int64_t ld;            // elements between rows of the stored matrix (16-byte multiples)
    int64_t plane_stride;  // elements between terms (16-byte multiple)
    int32_t planes;
    bool mn_major;
    const void* scales;
};

enum TileEpilogue : int {
    kTileOut = 0,    // D stored in fp32 or bf16, or added into fp32 partials
    kTileStats = 1,  // softmax statistics of D's rows (logits)
    kTileGrad = 2,   // the logits' gradient, in bf16 terms
    // The same for few rows of logits, which are D's columns (at most kTileFew), the
    // vocabulary its rows: D^T's statistics by 32 tokens of the vocabulary, and G^T.
    kTileStatsFew = 3,
    kTileGradFew = 4,
};

// What kTileStats leaves of a row and a tile of columns: the largest logit m,
// the sum a of exp(x - m) over the others, and t = sum exp(x - m) (x - m). `any` is 1 (0: of no
// logits at all).
struct alignas(16) TileStat {
    float m, a, t, any;
};

// The statistics of both's logits.
__device__ __forceinline__ void join(TileStat& s, const TileStat& o) {
    if (o.any == 0.0f) return;
    if (s.any == 0.0f) {
        s = o;
        return;
    }
    const bool mine = s.m >= o.m;
    const TileStat hi = mine ? s : o, lo = mine ? o : s;
    const float d = lo.m - hi.m, f = exp2f(d * 1.4426950408889634f), sum = 1.0f + lo.a;
    // (masks of the type's lowest value: d times their number is beyond binary32, and 0 times that
    // a NaN; a part of NaN has it in t)
    const float t = f > 0.0f ? fmaf(d, sum, lo.t) : lo.t;
    s = TileStat{hi.m, fmaf(f, sum, hi.a), fmaf(f, t, hi.t), 1.0f};
}

struct TileOut {
    // kTileOut: y, or (part != null) fp32 partials, part[split][M][part_ld], written or,
    // with `add`, added to
    void* y;
    int64_t ldy;
    int32_t y_bf16;
    int32_t add;
    float* part;
    int64_t part_ld;
    // kTileStats: stats[tile of columns][M]; `mine` [M] takes the logit of each
    // row's token. kTileGrad: G into `planes` terms of y (bf16, row stride ldy). Few rows:
    // stats[row of D / 32][N], and G^T (rows of a multiple of eight elements).
    TileStat* stats;
    float* mine;
    const int64_t* tokens;
    int64_t token0;  // the id of column 0
    int64_t vocab;
    const float *lse, *lse_lo, *entropy, *g, *h;
    int32_t planes;
    int64_t plane_stride;
};

struct TileProduct {
    TileOperand a, b;
    int32_t splits;  // kTileOut with partials: ranges of K
    TileOut out;
};

constexpr int kTileCols = 256;   // columns of a bf16 tile
constexpr int kTileNarrow = 128;  // of products with so few columns
constexpr int kTileCols8 = 192;  // of an e4m3 tile
constexpr int kTileFew = 64;     // rows of logits that take the forms for few rows

// Rows of a tile: a pair of SMs takes 256, one SM 128 (for few rows).
inline int tile_rows(bool pair) { return pair ? 256 : 128; }

// Enqueues n (1 or 2) products as one launch whose tiles share the SMs, the first's
// first. Both take pairs of SMs or neither. Errors: CAM_E_CUDA.
int tile_products(const char* fn, const TileProduct* p, int n, bool e4m3, bool pair,
                  TileEpilogue epilogue, int sms, cudaStream_t stream);

// A product of an fp32 matrix w [w_rows][width] with few rows (at most kFew32) in three
// bf16 terms, whose own terms the kernel makes as it reads it:
//     turned = false:  D[v][r] = sum_k w[v][k] b[r][k]    (b.rows = r, b.k = width)
//     turned = true:   D[d][r] = sum_v w[v][d] b[r][v]    (b MN-major, b.k = w_rows)
// with kTileStatsFew or kTileGradFew of the first, kTileOut into partials of the second.
struct Few32Product {
    const float* w;
    int64_t w_rows, width, w_stride;
    bool turned;
    TileOperand b;
    int32_t splits;
    TileOut out;
};
constexpr int kFew32 = 128;

// Enqueues it (f32_products.cu). Errors: CAM_E_CUDA.
int few32_product(const char* fn, const Few32Product& p, TileEpilogue epilogue, int sms,
                  cudaStream_t stream);

// The status word of these kernels on device `dev`, the current one.
cudaError_t operators_status(int dev, int32_t** at);

}  // namespace cam
