/*
 * kbit_mx.h -- microscaled 4-bit (MXFP4) linear layers of libkbit.so, forward
 * and backward, and the layer norm in front of them.
 *
 * The conventions of kbit.h hold: kbit_status results, validation before
 * anything is launched, device pointers, caller-owned buffers, asynchronous
 * work on `stream`, no allocation and no synchronisation.  T stands for the
 * element type (fp32, fp16, bf16; the 16-bit types are raw bits).  Distances of
 * rows count elements, for codes and scales bytes.  No pass writes what it does not own.
 * An output may be its input (same address and distance) where that is said;
 * other overlaps are undefined (the torch binding refuses them).
 */
#ifndef KBIT_MX_H
#define KBIT_MX_H

#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

/* ------------------------------------------------------------------------
 * MXFP4: blocks of 32 neighbouring values of a row share a power of two.
 *   e = max(floor(log2(max |x|)) - 2, -127), scale byte e + 127;
 *   code = x / 2^e rounded to the nearest of 0, 1/2, 1, 3/2, 2, 3, 4, 6 (codes
 *   0 .. 7, ties to the even code, at most 6), plus 8 for a negative sign.
 * A block of zeros has byte 0; a block with a NaN or an infinity byte 255, which
 * is NaN, and codes 0 (every output that it meets is NaN).  Values past a
 * row's end count as 0.  This is the OCP Microscaling Formats (MX) v1.0
 * specification's MXFP4 with its suggested scale.
 * codes: two a byte, the first in the low half; a row has 16 bytes a block, also
 *   for the last, partly filled one: ceil(d / 32) * 16.  Rows of codes start at
 *   multiples of 16 bytes (ldc a multiple of 16).
 * scales: ceil(d / 32) bytes a row, any alignment, lds bytes apart.
 * d is at most 2^26.
 * --------------------------------------------------------------------- */

/* Rows of X [rows][d] to codes and scales.  rows = 0 is a no-op. */
#define KBIT_DECLARE_QUANTIZE_MXFP4(T, CTYPE)                                                                  \
    int quantize_mxfp4_##T(const CTYPE* X, int64_t rows, int32_t d, int64_t ldx, uint8_t* codes, int64_t ldc,    \
                           uint8_t* scales, int64_t lds, void* stream);

/* Columns of X [rows][cols] to codes and scales: row c of both is column c of
 * X, in blocks along its rows (the rows of X transposed, without transposing
 * it).  rows is at most 2^26, cols at most 2^30.  cols = 0 is a no-op. */
#define KBIT_DECLARE_QUANTIZE_MXFP4_COLUMNS(T, CTYPE)                                                          \
    int quantize_mxfp4_columns_##T(const CTYPE* X, int64_t rows, int32_t cols, int64_t ldx, uint8_t* codes,      \
                                   int64_t ldc, uint8_t* scales, int64_t lds, void* stream);

/* out[r][i] = RN_T(code * 2^(scale - 127)) for i < d; exact where T holds the
 * value (it does for codes of values of T).  rows = 0 is a no-op. */
#define KBIT_DECLARE_DEQUANTIZE_MXFP4(T, CTYPE)                                                                \
    int dequantize_mxfp4_##T(const uint8_t* codes, int64_t ldc, const uint8_t* scales, int64_t lds, int64_t rows, \
                             int32_t d, CTYPE* out, int64_t ldo, void* stream);

/* out[m][n] = RN_T(sum over k of x[m][k] w[n][k] + bias[n]), both operands
 * MXFP4 rows of K values, sums in fp32 (in an order that is fixed for given
 * sizes and device).  bias: N values of T, or null.  Rows of codes and of scales
 * are less than 2^22 bytes apart (one row may be any distance from the next
 * where there is no next).  Values of the last block past K have to be codes
 * 0 in one of the operands at least, as the quantizers leave them.  workspace: at least linear_mxfp4_workspace_bytes(M, N, K)
 * bytes, 16-byte aligned (may be null where that is 0).  M = 0 is a no-op. */
#define KBIT_DECLARE_LINEAR_MXFP4(T, CTYPE)                                                                    \
    int linear_mxfp4_##T(const uint8_t* codes, const uint8_t* scales, int64_t M, int32_t K, int64_t ldx,         \
                         int64_t ldxs, const uint8_t* w_codes, const uint8_t* w_scales, int32_t N, int64_t ldw,  \
                         int64_t ldws, const CTYPE* bias, CTYPE* out, int64_t ldo, void* workspace,              \
                         int64_t workspace_bytes, void* stream);

/* Bytes of workspace on the current device; -1 for arguments out of range, and
 * where several rows of x or w would be 2^22 bytes of codes and more, K about
 * 2^23, apart.  It does not fall with M: one workspace for the largest batch
 * serves every smaller one. */
int64_t linear_mxfp4_workspace_bytes(int64_t M, int32_t N, int32_t K);

/* quantize_mxfp4 of X, then linear_mxfp4: the same values as the two calls up
 * to the order of sums.  workspace: linear_mxfp4_dynamic_workspace_bytes(M, N, K)
 * bytes (not falling with M; -1 as there), 16-byte aligned.  Several rows of X
 * have at most 2^23 - 256 values: their codes stand in the workspace, in whole
 * 128 bytes a row, less than 2^22 apart.  A few tokens are quantized
 * inside the product's kernel: where linear_mxfp4_dynamic_fused(M, N, K, ldw,
 * ldws) is 1 no workspace is needed and it may be null. */
#define KBIT_DECLARE_LINEAR_MXFP4_DYNAMIC(T, CTYPE)                                                            \
    int linear_mxfp4_dynamic_##T(const CTYPE* X, int64_t M, int32_t K, int64_t ldx, const uint8_t* w_codes,      \
                                 const uint8_t* w_scales, int32_t N, int64_t ldw, int64_t ldws,                  \
                                 const CTYPE* bias, CTYPE* out, int64_t ldo, void* workspace,                    \
                                 int64_t workspace_bytes, void* stream);

int64_t linear_mxfp4_dynamic_workspace_bytes(int64_t M, int32_t N, int32_t K);
int linear_mxfp4_dynamic_fused(int64_t M, int32_t N, int32_t K, int64_t ldw, int64_t ldws);

/* Gradients of out = X W^T + b with X [M][K], W [N][K] and dout [M][N] given as
 * values, each product taken in MXFP4 along the axis that it sums over:
 *   dX[m][k] = sum over n of q(dout[m][.])[n] q(W[.][k])[n]   (T)
 *   dW[n][k] = sum over m of q(dout[.][n])[m] q(X[.][k])[m]   (fp32)
 *   db[n]    = sum over m of dout[m][n]                        (fp32, not quantized)
 * where q quantizes that row or column in blocks of 32.  Each of dX, dW and db
 * may be null and is not computed then; W is read for dX only, X for dW only
 * (null otherwise).  Sums are in a fixed order.  M = 0 gives zeros for dW and db.
 * M, N and K are at most 2^26, and what a product sums over, in several rows of
 * codes in the workspace, at most 2^23 - 256: N for dX unless M = K = 1, M for dW
 * unless N = K = 1.
 * workspace: linear_mxfp4_backward_workspace_bytes(M, N, K) bytes (not falling
 * with M), 16-byte aligned, serve every choice of gradients; a call looks for no
 * more than it uses. */
#define KBIT_DECLARE_LINEAR_MXFP4_BACKWARD(T, CTYPE)                                                           \
    int linear_mxfp4_backward_##T(const CTYPE* dout, int64_t lddo, const CTYPE* X, int64_t ldx, const CTYPE* W,  \
                                  int64_t ldw, int64_t M, int32_t N, int32_t K, CTYPE* dX, int64_t lddx,         \
                                  float* dW, int64_t lddw, float* db, void* workspace,                           \
                                  int64_t workspace_bytes, void* stream);

int64_t linear_mxfp4_backward_workspace_bytes(int64_t M, int32_t N, int32_t K);

/* ------------------------------------------------------------------------
 * Layer norm of rows of d values: y = (x - mean) / sqrt(var + eps) * weight +
 * bias with var the mean square of x - mean, fp32 inside, one rounding to T.
 * weight, bias: d values of T, or fp32 with weight_fp32 != 0; bias may be null.
 * eps >= 0, finite; d at most 2^25.  out may be x.  rows = 0 is a no-op.
 * --------------------------------------------------------------------- */
#define KBIT_DECLARE_LAYER_NORM(T, CTYPE)                                                                      \
    int layer_norm_##T(const CTYPE* x, int64_t rows, int32_t d, int64_t ldx, const void* weight,                 \
                       const void* bias, int32_t weight_fp32, float eps, CTYPE* out, int64_t ldo, void* stream);

/* Its gradients, from that of the output and the input:
 *   dx = r (h - mean(h) - xh mean(h xh)), h = dout weight, xh = (x - mean) r;
 *   dweight = sum over rows of dout xh, dbias = sum over rows of dout: d fp32
 *   values each, in an order that is fixed for given sizes (zeros without rows).
 * dx may be dout.  workspace: layer_norm_backward_workspace_bytes(rows, d)
 * bytes (not falling with rows), 16-byte aligned. */
#define KBIT_DECLARE_LAYER_NORM_BACKWARD(T, CTYPE)                                                             \
    int layer_norm_backward_##T(const CTYPE* dout, int64_t lddo, const CTYPE* x, int64_t ldx, int64_t rows,      \
                                int32_t d, const void* weight, int32_t weight_fp32, float eps, CTYPE* dx,        \
                                int64_t lddx, float* dweight, float* dbias, void* workspace,                     \
                                int64_t workspace_bytes, void* stream);

int64_t layer_norm_backward_workspace_bytes(int64_t rows, int32_t d);

#define KBIT_DECLARE_MX(T, CTYPE)                 \
    KBIT_DECLARE_QUANTIZE_MXFP4(T, CTYPE)         \
    KBIT_DECLARE_QUANTIZE_MXFP4_COLUMNS(T, CTYPE) \
    KBIT_DECLARE_DEQUANTIZE_MXFP4(T, CTYPE)       \
    KBIT_DECLARE_LINEAR_MXFP4(T, CTYPE)           \
    KBIT_DECLARE_LINEAR_MXFP4_DYNAMIC(T, CTYPE)   \
    KBIT_DECLARE_LINEAR_MXFP4_BACKWARD(T, CTYPE)  \
    KBIT_DECLARE_LAYER_NORM(T, CTYPE)             \
    KBIT_DECLARE_LAYER_NORM_BACKWARD(T, CTYPE)
KBIT_DECLARE_MX(fp32, float)
KBIT_DECLARE_MX(fp16, uint16_t)
KBIT_DECLARE_MX(bf16, uint16_t)

#ifdef __cplusplus
}
#endif
#endif /* KBIT_MX_H */
