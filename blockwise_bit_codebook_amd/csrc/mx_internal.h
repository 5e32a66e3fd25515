// Internal launcher interface of the microscaled 4-bit layers and the layer
// norm (include/kbit_mx.h), between mx_api.cpp and the HIP translation units.
// No HIP types cross this boundary; arguments are already validated.
#pragma once

#include <stdint.h>

#include <tuple>

#include "kbit_internal.h"
#include "mx_choice.h"

namespace kbit {

constexpr int kMxBlock = 32;       // values a scale
constexpr int kMxBlockBytes = 16;  // of codes

// Longest row: its codes' bytes and their steps count in 32 bits.
constexpr int64_t kMxMaxDepth = int64_t(1) << 26;

// Most columns that are quantized as such.
constexpr int64_t kMxMaxColumns = int64_t(1) << 30;

inline int64_t mx_blocks(int64_t d) { return (d + kMxBlock - 1) / kMxBlock; }

// Rows of codes and scales.  paired: the scales stand in the order of pairs of
// steps of the product, 16 blocks of all rows after each other, lds bytes from
// pair to pair, 16 bytes a row (pair_place), for tiles of kPairedRows rows.
struct MxCoded {
    uint8_t *codes, *scales;  // both or neither null
    int64_t ldc, lds;
    bool paired;
};

int launch_mx_quantize(Dtype t, const void* X, int64_t rows, int d, int64_t ldx, const MxCoded& c, void* stream);

// Columns of X [rows][cols], a column a row of codes, and its rows where
// by_rows is there, in one reading of X.  sums: null, or mx_sum_groups(rows)
// rows of cols floats, the columns' sums over kMxSumRows rows each; with
// columns null they are all that is written.  Up to kMxColumnJobs matrices in one
// launch, by_rows for the first alone.
constexpr int64_t kMxSumRows = 256;
inline int64_t mx_sum_groups(int64_t rows) { return (rows + kMxSumRows - 1) / kMxSumRows; }
constexpr int kMxColumnJobs = 3;
struct MxColumns {
    const void* X;
    int64_t rows, ldx;
    int cols;
    MxCoded columns, by_rows;
    float* sums;
};
int launch_mx_quantize_columns(Dtype t, const MxColumns* jobs, int count, void* stream);

// out[c] = sum over groups of sums[group][c], in order.
int launch_mx_add_sums(const float* sums, int64_t groups, int cols, float* out, void* stream);

// Zeros to rows of cols floats.
int launch_mx_zero(float* out, int64_t rows, int cols, int64_t ldo, void* stream);

int launch_mx_dequantize(Dtype t, const uint8_t* codes, int64_t ldc, const uint8_t* scales, int64_t lds, int64_t rows,
                         int d, void* out, int64_t ldo, void* stream);

struct MxProduct {
    const uint8_t *x, *xs, *w, *ws;
    const void* bias;
    void* out;
    int64_t M, ldx, ldxs, ldw, ldws, ldo;
    int N, K;                 // K: bytes of a row of codes, a multiple of 16
    bool x_paired, w_paired;  // see MxCoded; only where mx_paired(M, N, K)
};

// workspace: of mx_product_workspace bytes, 16-byte aligned.
int launch_mx_product(Dtype t, const MxProduct& p, void* workspace, void* stream);

// Tokens quantized inside the product's kernel: their codes stay in LDS.
constexpr int kMxTokenItems = 4;   // pieces of 512 values a wave
constexpr int kMxTokenBytes = 20 * 1024;
constexpr int kMxTokenPad = 16;
constexpr int kMxMaxTokens = 8;
inline bool mx_tokens_fit(int64_t M, int N, int64_t d, int64_t ldw, int64_t ldws) {
    if (M > kMxMaxTokens || N > kMaxChannels || (N > 1 && (ldw >= kFarRows || ldws >= kFarRows))) return false;
    const int64_t per_row = (d + 511) / 512, bytes = mx_blocks(d) * kMxBlockBytes;
    const int64_t steps = (bytes + kDepth - 1) / kDepth;
    return M * (steps * kDepth + kMxTokenPad) <= kMxTokenBytes && M * per_row <= 8 * kMxTokenItems;
}

// Rows of quantized operands in a workspace: their codes start at whole cache
// lines, so that no step of kDepth bytes lies across two.
struct MxRows {
    int64_t ldc, lds, scales, bytes;  // scales: where they start
};
inline MxRows mx_rows(int64_t rows, int64_t d) {
    MxRows r;
    r.ldc = (mx_blocks(d) * kMxBlockBytes + kDepth - 1) / kDepth * kDepth;
    r.lds = (mx_blocks(d) + 15) / 16 * 16;
    r.scales = rows * r.ldc;
    r.bytes = r.scales + rows * r.lds;
    return r;
}

// Bytes of a row of codes.
inline int mx_depth(int64_t d) { return static_cast<int>(mx_blocks(d) * kMxBlockBytes); }

// Workspace of the backward pass, of the gradients that are wanted: for dX dout's
// rows and W's columns (along N), for dW dout's and X's columns (along M), for db
// the partial sums; then the products' own.
struct MxBackParts {
    MxRows g_rows, w_cols, g_cols, x_cols;
    int64_t w_at, gc_at, x_at, sums_at, product_at;
};
inline MxBackParts mx_back_parts(int64_t M, int N, int K, bool dX, bool dW, bool db) {
    MxBackParts b{};
    if (dX) b.g_rows = mx_rows(M, N);
    if (dX) b.w_cols = mx_rows(K, N);
    if (dW) b.g_cols = mx_rows(N, M);
    if (dW) b.x_cols = mx_rows(K, M);
    const auto up = [](int64_t n) { return (n + kDepth - 1) / kDepth * kDepth; };
    b.w_at = up(b.g_rows.bytes);
    b.gc_at = b.w_at + up(b.w_cols.bytes);
    b.x_at = b.gc_at + up(b.g_cols.bytes);
    b.sums_at = b.x_at + up(b.x_cols.bytes);
    b.product_at = b.sums_at + (db ? up(4 * mx_sum_groups(M) * N) : 0);
    return b;
}

// Bytes of it that a call needs.
inline int64_t mx_back_workspace(int64_t M, int N, int K, bool dX, bool dW, bool db) {
    int64_t own = 0;
    for (const auto& [rows, depth, wanted] : {std::make_tuple(M, mx_depth(N), dX), std::make_tuple(int64_t(N), mx_depth(M), dW)}) {
        if (!wanted) continue;
        const bool paired = mx_paired(rows, K, depth);
        const int64_t need = mx_product_workspace(rows, K, depth, paired, paired);
        if (need > own) own = need;
    }
    return mx_back_parts(M, N, K, dX, dW, db).product_at + own;
}

// p.x and p.xs are not looked at.
int launch_mx_tokens(Dtype t, const MxProduct& p, int d, const void* X, int64_t ldX, void* stream);

// ---------------------------------------------------------------------------
// layer norm
// ---------------------------------------------------------------------------
// Longest row: 64 threads a column add up the gradients, counted in 32 bits.
constexpr int kLayerNormMax = 1 << 25;

struct LayerNormArgs {
    const void *x, *weight, *bias;  // bias may be null
    void* out;
    int64_t rows, ldx, ldo;
    int d;
    float eps;
    bool weight_fp32;
};

int launch_layer_norm(Dtype t, const LayerNormArgs& p, void* stream);

// Rows of partial sums of the weights' gradients, each 2 d floats.
constexpr int kLayerNormPartials = 512;
// Longest row whose sums stay in registers; above it the rows' statistics go
// to the workspace and a second pass sums over rows.
constexpr int kLayerNormKept = 16384;
constexpr int kLayerNormStats = 8;  // floats a row

// Rows of partial sums: of long rows, whose columns fill the device by
// themselves, as many as keep 2048 workgroups of kLayerNormColumns at work.
constexpr int kLayerNormColumns = 2048;
inline int64_t layer_norm_groups(int64_t rows, int d) {
    int64_t most = kLayerNormPartials;
    if (d > kLayerNormKept) most = 2048 / ((d + kLayerNormColumns - 1) / kLayerNormColumns);
    if (most < 1) most = 1;
    return rows < most ? rows : most;
}

inline int64_t layer_norm_backward_bytes(int64_t rows, int d) {
    return 4 * (layer_norm_groups(rows, d) * 2 * d + (d > kLayerNormKept ? kLayerNormStats * rows : 0));
}

struct LayerNormBackArgs {
    const void *g, *x, *weight;
    void* dx;
    float *dweight, *dbias, *workspace;
    int64_t rows, ldg, ldx, lddx;
    int d;
    float eps;
    bool weight_fp32;
};

int launch_layer_norm_back(Dtype t, const LayerNormBackArgs& p, void* stream);

}  // namespace kbit
