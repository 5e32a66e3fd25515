/*
 * kbit_layer.h -- the operators of libkbit.so around a quantized layer:
 * 8-bit integer linear layers, rotary positions, norms of query and key
 * heads with the rotation in the same pass, and the append to a paged cache.
 *
 * The conventions of kbit.h hold: kbit_status results, validation before
 * anything is launched, device pointers, caller-owned buffers, asynchronous
 * work on `stream`, no allocation and no synchronisation.  T stands for the
 * element type (fp32, fp16, bf16; the 16-bit types are raw bits).  Strides
 * count elements.  No pass writes what it does not own: strided outputs leave
 * the elements between their rows alone.  Outputs may be their input (same
 * address and strides) where that is said; other overlaps are undefined (the
 * torch binding refuses them).
 */
#ifndef KBIT_LAYER_H
#define KBIT_LAYER_H

#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

/* ------------------------------------------------------------------------
 * int8 linear layer.
 *
 * Codes of a row x of d values, one fp32 scale a row:
 *   amax = max |x|, scale = RN(amax / 127), q = rint(RN(x * RN(127 * RN(1 / amax))))
 *   (half to even), |q| <= 127.  The step is rounded twice, as where a program
 *   divides a scalar by a tensor through its reciprocal; RN(127 / amax) would
 *   give another code, by one, for some values within a rounding of a tie.
 *   amax < 2^-100: scale 0 and codes 0.  A row
 *   with a NaN or an infinity: scale NaN and codes 0 (its outputs are NaN).
 * codes: row r starts at codes + r * ldc, 16-byte aligned (ldc a multiple of
 *   16, at least d rounded up to 16); the bytes from d up to that multiple of
 *   16 are set to zero, any further ones are left alone.
 * Used for activations (a row is a token) and for weights (a row is an output
 * channel).  d is at most 2^31 - 16.  rows = 0 is a no-op.
 * --------------------------------------------------------------------- */
#define KBIT_DECLARE_QUANTIZE_ROWS(T, CTYPE)                                                                   \
    int quantize_rows_int8_##T(const CTYPE* X, int64_t rows, int32_t d, int64_t ldx, int8_t* codes, int64_t ldc, \
                               float* scale, void* stream);

/* out[m][n] = RN_T( RN(RN(RN(acc) * scale[m]) * w_scale[n]) + bias[n] ),
 * acc = sum over k of codes[m][k] * w_codes[n][k], exact in int32 (K at most
 * 131071, codes any int8 value).  bias: N values of T, or null.  ldx, ldw,
 * ldo: distance of rows.  Any alignment and any K >= 1 give the same values;
 * rows of codes that all start at multiples of 16 bytes take the fast path.
 * workspace: at least linear_int8_workspace_bytes(M, N, K) bytes, 16-byte
 * aligned (may be null where that is 0): where rows and channels are too few
 * to fill the device and the depth is long, the parts' sums.  M = 0 is a
 * no-op. */
#define KBIT_DECLARE_LINEAR_INT8(T, CTYPE)                                                                     \
    int linear_int8_##T(const int8_t* codes, const float* scale, int64_t M, int32_t K, int64_t ldx,              \
                        const int8_t* w_codes, const float* w_scale, int32_t N, int64_t ldw, const CTYPE* bias,  \
                        CTYPE* out, int64_t ldo, void* workspace, int64_t workspace_bytes, void* stream);

/* Bytes of workspace on the current device (-1 for arguments out of range).
 * It does not fall with M: one workspace for the largest batch serves every
 * smaller one.  At most 128 KB a compute unit. */
int64_t linear_int8_workspace_bytes(int64_t M, int32_t N, int32_t K);

/* quantize_rows_int8 of X, then linear_int8: the same values as the two
 * calls.  workspace: linear_int8_dynamic_workspace_bytes(M, N, K) bytes (again
 * not falling with M), 16-byte aligned.  A few tokens are quantized inside the product's kernel:
 * where linear_int8_dynamic_fused(M, N, K, ldw) is 1 and w_codes is 16-byte
 * aligned no workspace is needed and it may be null. */
#define KBIT_DECLARE_LINEAR_INT8_DYNAMIC(T, CTYPE)                                                             \
    int linear_int8_dynamic_##T(const CTYPE* X, int64_t M, int32_t K, int64_t ldx, const int8_t* w_codes,        \
                                const float* w_scale, int32_t N, int64_t ldw, const CTYPE* bias, CTYPE* out,     \
                                int64_t ldo, void* workspace, int64_t workspace_bytes, void* stream);

int64_t linear_int8_dynamic_workspace_bytes(int64_t M, int32_t N, int32_t K);
int linear_int8_dynamic_fused(int64_t M, int32_t N, int32_t K, int64_t ldw);

/* ------------------------------------------------------------------------
 * Rotary positions.
 *
 * Frequencies of the rot / 2 pairs (host arrays, fp64): f_i = base^(-2i/rot),
 *   KBIT_ROPE_LINEAR  f_i / factor (positions interpolated);
 *   KBIT_ROPE_NTK     base * factor^(rot / (rot - 2)) as the base: the lowest
 *                     frequency divided by factor, the highest kept;
 *   KBIT_ROPE_YARN    with t_i = original_length * f_i / (2 pi) turns over the
 *                     original length: pairs of at most slow_turns are divided
 *                     by factor, pairs of at least fast_turns kept, a line in
 *                     t_i between; amplitude 0.1 ln(factor) + 1 (Peng et al.,
 *                     "YaRN: Efficient Context Window Extension of Large
 *                     Language Models").
 * factor >= 1.  amplitude is 1 but for YARN.  Any other frequencies can be
 * given to rope_table as well.
 * --------------------------------------------------------------------- */
enum { KBIT_ROPE_UNSCALED = 0, KBIT_ROPE_LINEAR = 1, KBIT_ROPE_NTK = 2, KBIT_ROPE_YARN = 3 };
enum { KBIT_ROPE_HALF = 0, KBIT_ROPE_INTERLEAVED = 1 };

int rope_frequencies(int32_t rot, double base, int32_t scaling, double factor, double original_length,
                     double slow_turns, double fast_turns, double* freq_host, double* amplitude_host);

/* table[p][i] = RN(amplitude cos(p freq[i])), table[p][rot/2 + i] =
 * RN(amplitude sin(p freq[i])) for p < max_pos, fp64 inside.  freq: device.
 * table: device, max_pos * rot floats, 16-byte aligned. */
int rope_table(const double* freq, int32_t rot, int64_t max_pos, double amplitude, float* table, void* stream);

/* Rotates the first rot elements (even, at most dim) of every head of
 * x[batch][tokens][heads][dim] (dim at most 1024, unit stride in dim):
 *   (a, b) -> (RN(RN(a c) - RN(b s)), RN(RN(b c) + RN(a s))) rounded to T,
 * pairs (i, i + rot/2) in the half layout, (2i, 2i + 1) interleaved; the other
 * elements are copied.  c, s: the table's row of the token's position,
 * positions[batch][tokens] (contiguous, int32 or int64: position_bytes 4 or
 * 8).  A position outside [0, max_pos) gives NaN in the rotated elements.
 * inverse != 0 negates s: the transposed rotation, which takes the output's
 * gradient to the input's.  out may be x.  batch is at most 65535 unless tokens
 * is 1 or the batches follow one another at tokens times the tokens' distance
 * (in x and out), so that they count as one; the same holds for qk_norm_rope. */
#define KBIT_DECLARE_ROPE(T, CTYPE)                                                                            \
    int rope_##T(const CTYPE* x, int64_t x_batch, int64_t x_token, int64_t x_head, CTYPE* out, int64_t out_batch, \
                 int64_t out_token, int64_t out_head, int64_t batch, int64_t tokens, int32_t heads, int32_t dim, \
                 const void* positions, int32_t position_bytes, const float* table, int32_t rot, int64_t max_pos, \
                 int32_t layout, int32_t inverse, void* stream);

/* ------------------------------------------------------------------------
 * Norms of queries and keys with the rotation in the same pass:
 *   y = rotation( x / sqrt(mean(x^2) + eps) * weight ), per head, fp32 inside,
 * one rounding to T.  q and k share batch, tokens, dim, positions and table;
 * weights: dim values of T, or fp32 with weight_fp32 != 0.  eps >= 0, finite.
 * q_out may be q and k_out may be k.
 * --------------------------------------------------------------------- */
#define KBIT_DECLARE_QK_NORM_ROPE(T, CTYPE)                                                                    \
    int qk_norm_rope_##T(const CTYPE* q, int64_t q_batch, int64_t q_token, int64_t q_head, const CTYPE* k,       \
                         int64_t k_batch, int64_t k_token, int64_t k_head, CTYPE* q_out, int64_t qo_batch,       \
                         int64_t qo_token, int64_t qo_head, CTYPE* k_out, int64_t ko_batch, int64_t ko_token,    \
                         int64_t ko_head, int64_t batch, int64_t tokens, int32_t q_heads, int32_t k_heads,       \
                         int32_t dim, const void* q_weight, const void* k_weight, int32_t weight_fp32, float eps, \
                         const void* positions, int32_t position_bytes, const float* table, int32_t rot,         \
                         int64_t max_pos, int32_t layout, void* stream);

/* Its gradient.  gq, gk: gradients of the outputs; q, k: the inputs of the
 * forward pass; dq, dk: gradients of the inputs (dq may be gq, dk may be gk);
 * dq_weight, dk_weight: dim fp32 sums over batch, tokens and heads, in an
 * order that is fixed for given sizes (zeros without tokens).  workspace: qk_norm_rope_backward_
 * workspace_bytes(dim) bytes, 16-byte aligned. */
#define KBIT_DECLARE_QK_NORM_ROPE_BACKWARD(T, CTYPE)                                                           \
    int qk_norm_rope_backward_##T(                                                                               \
        const CTYPE* gq, int64_t gq_batch, int64_t gq_token, int64_t gq_head, const CTYPE* gk, int64_t gk_batch, \
        int64_t gk_token, int64_t gk_head, const CTYPE* q, int64_t q_batch, int64_t q_token, int64_t q_head,     \
        const CTYPE* k, int64_t k_batch, int64_t k_token, int64_t k_head, CTYPE* dq, int64_t dq_batch,           \
        int64_t dq_token, int64_t dq_head, CTYPE* dk, int64_t dk_batch, int64_t dk_token, int64_t dk_head,       \
        int64_t batch, int64_t tokens, int32_t q_heads, int32_t k_heads, int32_t dim, const void* q_weight,      \
        const void* k_weight, int32_t weight_fp32, float* dq_weight, float* dk_weight, float eps,                \
        const void* positions, int32_t position_bytes, const float* table, int32_t rot, int64_t max_pos,         \
        int32_t layout, void* workspace, int64_t workspace_bytes, void* stream);

int64_t qk_norm_rope_backward_workspace_bytes(int32_t dim);

/* ------------------------------------------------------------------------
 * Append to a paged cache: token t's keys (rotated as by rope_T when rot is
 * not 0) and values go to slot slots[t] = page * page_size + place, that is to
 *   k_cache + page * kc_page + place * kc_slot + head * kc_head (dim elements),
 * so that both orders of heads and places inside a page are covered.  Keys
 * and values have the same heads; k_dim and v_dim may differ.  slots: int32 or
 * int64 (slot_bytes).  A slot below 0 (padding) or beyond the cache writes
 * nothing; the slots of a call have to be distinct.  rot = 0: keys are copied,
 * positions, table, max_pos and layout are not looked at.
 * --------------------------------------------------------------------- */
#define KBIT_DECLARE_APPEND_KV_PAGED(T, CTYPE)                                                                 \
    int append_kv_paged_##T(const CTYPE* k, int64_t k_token, int64_t k_head, const CTYPE* v, int64_t v_token,    \
                            int64_t v_head, int64_t tokens, int32_t heads, int32_t k_dim, int32_t v_dim,         \
                            const void* slots, int32_t slot_bytes, CTYPE* k_cache, int64_t kc_page,              \
                            int64_t kc_slot, int64_t kc_head, CTYPE* v_cache, int64_t vc_page, int64_t vc_slot,  \
                            int64_t vc_head, int64_t pages, int32_t page_size, const void* positions,            \
                            int32_t position_bytes, const float* table, int32_t rot, int64_t max_pos,            \
                            int32_t layout, void* stream);

#define KBIT_DECLARE_LAYER(T, CTYPE)             \
    KBIT_DECLARE_QUANTIZE_ROWS(T, CTYPE)         \
    KBIT_DECLARE_LINEAR_INT8(T, CTYPE)           \
    KBIT_DECLARE_LINEAR_INT8_DYNAMIC(T, CTYPE)   \
    KBIT_DECLARE_ROPE(T, CTYPE)                  \
    KBIT_DECLARE_QK_NORM_ROPE(T, CTYPE)          \
    KBIT_DECLARE_QK_NORM_ROPE_BACKWARD(T, CTYPE) \
    KBIT_DECLARE_APPEND_KV_PAGED(T, CTYPE)
KBIT_DECLARE_LAYER(fp32, float)
KBIT_DECLARE_LAYER(fp16, uint16_t)
KBIT_DECLARE_LAYER(bf16, uint16_t)

#ifdef __cplusplus
}
#endif
#endif /* KBIT_LAYER_H */
