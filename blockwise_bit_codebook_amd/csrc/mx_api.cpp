// C ABI of include/kbit_mx.h: argument validation, device checks and dispatch
// to the HIP launchers.  As in api.cpp every entry point validates before it
// launches and reports errors as kbit_status codes; nothing aborts, allocates
// or synchronises.
#include <cmath>
#include <cstdint>

#include "kbit.h"
#include "kbit_mx.h"
#include "mx_internal.h"

namespace kbit {
namespace {

constexpr int64_t kMaxElems = int64_t(1) << 40;
constexpr int64_t kMaxRows = (int64_t(1) << 31) - 1;

bool aligned(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }
int64_t elem_size(Dtype t) { return t == Dtype::fp32 ? 4 : 2; }
int map_launch(int hip_status) { return hip_status == 0 ? KBIT_OK : KBIT_ELAUNCH; }

// Rows of d elements ld apart (one row may carry any distance).
bool rows_ok(int64_t rows, int64_t d, int64_t ld) {
    return rows >= 0 && rows <= kMaxRows && d >= 1 && d <= kMaxElems && (rows <= 1 || (ld >= d && ld <= kMaxElems / rows));
}
bool depth_ok(int64_t d) { return d >= 1 && d <= kMxMaxDepth; }
bool codes_aligned(const void* p, int64_t rows, int64_t ld) { return aligned(p, 16) && (rows <= 1 || ld % 16 == 0); }

// Codes and scales of rows of d values.
bool coded_rows_ok(int64_t rows, int64_t d, int64_t ldc, int64_t lds) {
    return rows_ok(rows, mx_depth(d), ldc) && rows_ok(rows, mx_blocks(d), lds);
}

int do_quantize(Dtype t, const void* X, int64_t rows, int32_t d, int64_t ldx, uint8_t* codes, int64_t ldc,
                uint8_t* scales, int64_t lds, void* stream) {
    if (!depth_ok(d) || !rows_ok(rows, d, ldx) || !coded_rows_ok(rows, d, ldc, lds)) return KBIT_EINVAL;
    if (rows == 0) return KBIT_OK;
    if (!X || !codes || !scales) return KBIT_EINVAL;
    if (!aligned(X, elem_size(t)) || !codes_aligned(codes, rows, ldc)) return KBIT_EALIGN;
    if (!device_usable()) return KBIT_EDEVICE;
    return map_launch(launch_mx_quantize(t, X, rows, d, ldx, MxCoded{codes, scales, ldc, lds, false}, stream));
}

int do_quantize_columns(Dtype t, const void* X, int64_t rows, int32_t cols, int64_t ldx, uint8_t* codes, int64_t ldc,
                        uint8_t* scales, int64_t lds, void* stream) {
    if (!depth_ok(rows) || cols < 0 || cols > kMxMaxColumns || (cols > 0 && !rows_ok(rows, cols, ldx)) || !coded_rows_ok(cols, rows, ldc, lds))
        return KBIT_EINVAL;
    if (cols == 0) return KBIT_OK;
    if (!X || !codes || !scales) return KBIT_EINVAL;
    if (!aligned(X, elem_size(t)) || !codes_aligned(codes, cols, ldc)) return KBIT_EALIGN;
    if (!device_usable()) return KBIT_EDEVICE;
    const MxColumns job{X, rows, ldx, cols, MxCoded{codes, scales, ldc, lds, false}, MxCoded{}, nullptr};
    return map_launch(launch_mx_quantize_columns(t, &job, 1, stream));
}

int do_dequantize(Dtype t, const uint8_t* codes, int64_t ldc, const uint8_t* scales, int64_t lds, int64_t rows, int32_t d,
                  void* out, int64_t ldo, void* stream) {
    if (!depth_ok(d) || !rows_ok(rows, d, ldo) || !coded_rows_ok(rows, d, ldc, lds)) return KBIT_EINVAL;
    if (rows == 0) return KBIT_OK;
    if (!out || !codes || !scales) return KBIT_EINVAL;
    if (!aligned(out, elem_size(t)) || !codes_aligned(codes, rows, ldc)) return KBIT_EALIGN;
    if (!device_usable()) return KBIT_EDEVICE;
    return map_launch(launch_mx_dequantize(t, codes, ldc, scales, lds, rows, d, out, ldo, stream));
}

// Rows of an operand in reach of the kernels' 32-bit offsets.
bool near_rows(int64_t rows, int64_t ld) { return rows <= 1 || ld < kFarRows; }

// Shared checks of the product: 1 = go on.
int check_product(Dtype t, const MxProduct& p, int64_t d) {
    if (!depth_ok(d) || p.N < 1 || !coded_rows_ok(p.M, d, p.ldx, p.ldxs) || !coded_rows_ok(p.N, d, p.ldw, p.ldws) ||
        !rows_ok(p.M, p.N, p.ldo) || !near_rows(p.M, p.ldx) || !near_rows(p.M, p.ldxs) || !near_rows(p.N, p.ldw) ||
        !near_rows(p.N, p.ldws))
        return KBIT_EINVAL;
    if (p.M == 0) return KBIT_OK;
    if (!p.w || !p.ws || !p.out) return KBIT_EINVAL;
    if (!codes_aligned(p.w, p.N, p.ldw) || !aligned(p.out, elem_size(t)) || !aligned(p.bias, elem_size(t))) return KBIT_EALIGN;
    return 1;
}

int do_linear(Dtype t, MxProduct p, int64_t d, void* workspace, int64_t workspace_bytes, void* stream) {
    const int c = check_product(t, p, d);
    if (c != 1) return c;
    if (!p.x || !p.xs) return KBIT_EINVAL;
    if (!codes_aligned(p.x, p.M, p.ldx) || !aligned(workspace, 16)) return KBIT_EALIGN;
    p.K = mx_depth(d);
    const int64_t need = mx_product_workspace(p.M, p.N, p.K);
    if (workspace_bytes < need || (need > 0 && !workspace)) return KBIT_EINVAL;
    if (!device_usable()) return KBIT_EDEVICE;
    return map_launch(launch_mx_product(t, p, workspace, stream));
}

// Rows in a workspace; paired: the order of their scales.
MxCoded coded_in(uint8_t* at, const MxRows& r, int64_t rows, bool paired) {
    return MxCoded{at, at + r.scales, r.ldc, paired ? rows * 16 : r.lds, paired};
}

int do_linear_dynamic(Dtype t, const void* X, int64_t ldX, MxProduct p, int64_t d, void* workspace,
                      int64_t workspace_bytes, void* stream) {
    if (!depth_ok(d) || !rows_ok(p.M, d, ldX)) return KBIT_EINVAL;
    const MxRows r = mx_rows(p.M, d);
    p.ldx = r.ldc;
    p.ldxs = r.lds;
    const int c = check_product(t, p, d);
    if (c != 1) return c;
    if (!X) return KBIT_EINVAL;
    if (!aligned(X, elem_size(t)) || !aligned(workspace, 16)) return KBIT_EALIGN;
    p.K = mx_depth(d);
    if (mx_tokens_fit(p.M, p.N, d, p.ldw, p.ldws)) {
        if (!device_usable()) return KBIT_EDEVICE;
        return map_launch(launch_mx_tokens(t, p, static_cast<int>(d), X, ldX, stream));
    }
    const int64_t at = (r.bytes + 15) / 16 * 16;
    p.x_paired = mx_paired(p.M, p.N, p.K);
    if (!workspace || workspace_bytes < at + mx_product_workspace(p.M, p.N, p.K, p.x_paired)) return KBIT_EINVAL;
    if (!device_usable()) return KBIT_EDEVICE;
    uint8_t* w = static_cast<uint8_t*>(workspace);
    const MxCoded c_x = coded_in(w, r, p.M, p.x_paired);
    if (launch_mx_quantize(t, X, p.M, static_cast<int>(d), ldX, c_x, stream) != 0) return KBIT_ELAUNCH;
    p.x = w;
    p.xs = c_x.scales;
    p.ldxs = c_x.lds;
    return map_launch(launch_mx_product(t, p, w + at, stream));
}

MxProduct product_of(const MxCoded& a, int64_t M, const MxCoded& b, int N, int64_t depth, void* out, int64_t ldo) {
    return MxProduct{a.codes, a.scales, b.codes, b.scales, nullptr, out,           M,       a.ldc,
                     a.lds,   b.ldc,    b.lds,   ldo,      N,       mx_depth(depth), a.paired, b.paired};
}

int do_linear_backward(Dtype t, const void* g, int64_t ldg, const void* X, int64_t ldx, const void* W, int64_t ldw, int64_t M,
                       int32_t N, int32_t K, void* dX, int64_t lddx, float* dW, int64_t lddw, float* db, void* workspace,
                       int64_t workspace_bytes, void* stream) {
    if (!depth_ok(N) || !depth_ok(K) || M < 0 || M > kMxMaxDepth || !rows_ok(M, N, ldg)) return KBIT_EINVAL;
    if (dX && (!rows_ok(N, K, ldw) || !rows_ok(M, K, lddx))) return KBIT_EINVAL;
    if (dW && (!rows_ok(M, K, ldx) || !rows_ok(N, K, lddw))) return KBIT_EINVAL;
    if (!dX && !dW && !db) return KBIT_OK;
    if (M == 0 && !dW && !db) return KBIT_OK;
    if (M > 0 && (!g || (dX && !W) || (dW && !X))) return KBIT_EINVAL;
    const int64_t es = elem_size(t);
    if (!aligned(g, es) || !aligned(X, es) || !aligned(W, es) || !aligned(dX, es) || !aligned(dW, 4) || !aligned(db, 4) ||
        !aligned(workspace, 16))
        return KBIT_EALIGN;
    const MxBackParts b = mx_back_parts(M, N, K, dX != nullptr, dW != nullptr, db != nullptr);
    if (M > 0 && (!workspace || workspace_bytes < mx_back_workspace(M, N, K, dX != nullptr, dW != nullptr, db != nullptr)))
        return KBIT_EINVAL;
    // the operands' rows in the workspace, as the products need them
    if (M > 0 && ((dX && (!near_rows(M, b.g_rows.ldc) || !near_rows(K, b.w_cols.ldc))) ||
                  (dW && (!near_rows(N, b.g_cols.ldc) || !near_rows(K, b.x_cols.ldc)))))
        return KBIT_EINVAL;
    if (!device_usable()) return KBIT_EDEVICE;
    if (M == 0) {
        if (dW && launch_mx_zero(dW, N, K, lddw, stream) != 0) return KBIT_ELAUNCH;
        return db ? map_launch(launch_mx_add_sums(nullptr, 0, N, db, stream)) : KBIT_OK;
    }
    uint8_t* w = static_cast<uint8_t*>(workspace);
    float* sums = reinterpret_cast<float*>(w + b.sums_at);
    const bool pair_x = dX && mx_paired(M, K, mx_depth(N)), pair_w = dW && mx_paired(N, K, mx_depth(M));
    const MxCoded g_rows = coded_in(w, b.g_rows, M, pair_x), w_cols = coded_in(w + b.w_at, b.w_cols, K, pair_x),
                  g_cols = coded_in(w + b.gc_at, b.g_cols, N, pair_w), x_cols = coded_in(w + b.x_at, b.x_cols, K, pair_w);
    // dout's columns and their sums with its rows, W's and X's in one launch; dout's rows alone where nothing else needs it
    MxColumns jobs[kMxColumnJobs];
    int count = 0;
    if (dW || db) jobs[count++] = MxColumns{g, M, ldg, N, dW ? g_cols : MxCoded{}, dX ? g_rows : MxCoded{}, db ? sums : nullptr};
    else if (launch_mx_quantize(t, g, M, N, ldg, g_rows, stream) != 0) return KBIT_ELAUNCH;
    if (dX) jobs[count++] = MxColumns{W, N, ldw, K, w_cols, MxCoded{}, nullptr};
    if (dW) jobs[count++] = MxColumns{X, M, ldx, K, x_cols, MxCoded{}, nullptr};
    if (launch_mx_quantize_columns(t, jobs, count, stream) != 0) return KBIT_ELAUNCH;
    if (db && launch_mx_add_sums(sums, mx_sum_groups(M), N, db, stream) != 0) return KBIT_ELAUNCH;
    if (dX && launch_mx_product(t, product_of(g_rows, M, w_cols, K, N, dX, lddx), w + b.product_at, stream) != 0) return KBIT_ELAUNCH;
    if (dW && launch_mx_product(Dtype::fp32, product_of(g_cols, N, x_cols, K, M, dW, lddw), w + b.product_at, stream) != 0)
        return KBIT_ELAUNCH;
    return KBIT_OK;
}

bool eps_ok(float eps) { return eps >= 0.0f && !std::isinf(eps); }

int do_layer_norm(Dtype t, const LayerNormArgs& p, void* stream) {
    if (p.d < 1 || p.d > kLayerNormMax || !rows_ok(p.rows, p.d, p.ldx) || !rows_ok(p.rows, p.d, p.ldo) || !eps_ok(p.eps)) return KBIT_EINVAL;
    if (p.rows == 0) return KBIT_OK;
    if (!p.x || !p.weight || !p.out) return KBIT_EINVAL;
    const int64_t es = elem_size(t), ws = p.weight_fp32 ? 4 : es;
    if (!aligned(p.x, es) || !aligned(p.out, es) || !aligned(p.weight, ws) || !aligned(p.bias, ws)) return KBIT_EALIGN;
    if (!device_usable()) return KBIT_EDEVICE;
    return map_launch(launch_layer_norm(t, p, stream));
}

int do_layer_norm_backward(Dtype t, const LayerNormBackArgs& p, int64_t workspace_bytes, void* stream) {
    if (p.d < 1 || p.d > kLayerNormMax || !rows_ok(p.rows, p.d, p.ldg) || !rows_ok(p.rows, p.d, p.ldx) || !rows_ok(p.rows, p.d, p.lddx) ||
        !eps_ok(p.eps))
        return KBIT_EINVAL;
    const int64_t need = layer_norm_backward_bytes(p.rows, p.d);
    if (!p.dweight || !p.dbias || workspace_bytes < need || (need > 0 && !p.workspace)) return KBIT_EINVAL;
    if (p.rows > 0 && (!p.g || !p.x || !p.weight || !p.dx)) return KBIT_EINVAL;
    const int64_t es = elem_size(t), ws = p.weight_fp32 ? 4 : es;
    if (!aligned(p.g, es) || !aligned(p.x, es) || !aligned(p.dx, es) || !aligned(p.weight, ws) || !aligned(p.dweight, 4) ||
        !aligned(p.dbias, 4) || !aligned(p.workspace, 16))
        return KBIT_EALIGN;
    if (!device_usable()) return KBIT_EDEVICE;
    return map_launch(launch_layer_norm_back(t, p, stream));
}

// Sizes for which there is a product: several rows have to be in the kernels'
// reach at the least distance that they can have, `row` and a weight's own row.
bool product_sizes_ok(int64_t M, int32_t N, int32_t K, int64_t row) {
    return M >= 0 && M <= kMaxRows && N >= 1 && depth_ok(K) && near_rows(M, row) && near_rows(N, mx_depth(K));
}
bool codes_sizes_ok(int64_t M, int32_t N, int32_t K) { return product_sizes_ok(M, N, K, mx_depth(K)); }
bool values_sizes_ok(int64_t M, int32_t N, int32_t K) { return product_sizes_ok(M, N, K, mx_rows(1, K).ldc); }

}  // namespace
}  // namespace kbit

using kbit::Dtype;
using kbit::LayerNormArgs;
using kbit::LayerNormBackArgs;
using kbit::MxProduct;

extern "C" {

int64_t linear_mxfp4_workspace_bytes(int64_t M, int32_t N, int32_t K) {
    if (!kbit::codes_sizes_ok(M, N, K)) return -1;
    return kbit::mx_product_workspace_up_to(M, N, kbit::mx_depth(K));
}

int64_t linear_mxfp4_dynamic_workspace_bytes(int64_t M, int32_t N, int32_t K) {
    if (!kbit::values_sizes_ok(M, N, K)) return -1;
    return (kbit::mx_rows(M, K).bytes + 15) / 16 * 16 + kbit::mx_product_workspace_up_to(M, N, kbit::mx_depth(K));
}

int linear_mxfp4_dynamic_fused(int64_t M, int32_t N, int32_t K, int64_t ldw, int64_t ldws) {
    return M >= 1 && kbit::values_sizes_ok(M, N, K) && kbit::mx_tokens_fit(M, N, K, ldw, ldws);
}

int64_t linear_mxfp4_backward_workspace_bytes(int64_t M, int32_t N, int32_t K) {
    if (M < 0 || M > kbit::kMxMaxDepth || !kbit::depth_ok(N) || !kbit::depth_ok(K)) return -1;
    if (M == 0) return 0;
    const int64_t a = kbit::mx_product_workspace_up_to(M, K, kbit::mx_depth(N));
    const int64_t b = kbit::mx_product_workspace_up_to(N, K, kbit::mx_depth(M));
    return kbit::mx_back_parts(M, N, K, true, true, true).product_at + (a > b ? a : b);
}

int64_t layer_norm_backward_workspace_bytes(int64_t rows, int32_t d) {
    if (rows < 0 || rows > kbit::kMaxRows || d < 1 || d > kbit::kLayerNormMax) return -1;
    return kbit::layer_norm_backward_bytes(rows, d);
}

#define KBIT_DEFINE_MX(TNAME, CTYPE)                                                                                  \
    int quantize_mxfp4_##TNAME(const CTYPE* X, int64_t rows, int32_t d, int64_t ldx, uint8_t* codes, int64_t ldc,     \
                               uint8_t* scales, int64_t lds, void* stream) {                                          \
        return kbit::do_quantize(Dtype::TNAME, X, rows, d, ldx, codes, ldc, scales, lds, stream);                     \
    }                                                                                                                 \
    int quantize_mxfp4_columns_##TNAME(const CTYPE* X, int64_t rows, int32_t cols, int64_t ldx, uint8_t* codes,       \
                                       int64_t ldc, uint8_t* scales, int64_t lds, void* stream) {                     \
        return kbit::do_quantize_columns(Dtype::TNAME, X, rows, cols, ldx, codes, ldc, scales, lds, stream);          \
    }                                                                                                                 \
    int dequantize_mxfp4_##TNAME(const uint8_t* codes, int64_t ldc, const uint8_t* scales, int64_t lds, int64_t rows, \
                                 int32_t d, CTYPE* out, int64_t ldo, void* stream) {                                  \
        return kbit::do_dequantize(Dtype::TNAME, codes, ldc, scales, lds, rows, d, out, ldo, stream);                 \
    }                                                                                                                 \
    int linear_mxfp4_##TNAME(const uint8_t* codes, const uint8_t* scales, int64_t M, int32_t K, int64_t ldx,          \
                             int64_t ldxs, const uint8_t* w_codes, const uint8_t* w_scales, int32_t N, int64_t ldw,   \
                             int64_t ldws, const CTYPE* bias, CTYPE* out, int64_t ldo, void* workspace,               \
                             int64_t workspace_bytes, void* stream) {                                                 \
        return kbit::do_linear(Dtype::TNAME,                                                                          \
                               MxProduct{codes, scales, w_codes, w_scales, bias, out, M, ldx, ldxs, ldw, ldws, ldo, N, 0, false, false}, \
                               K, workspace, workspace_bytes, stream);                                                \
    }                                                                                                                 \
    int linear_mxfp4_dynamic_##TNAME(const CTYPE* X, int64_t M, int32_t K, int64_t ldx, const uint8_t* w_codes,       \
                                     const uint8_t* w_scales, int32_t N, int64_t ldw, int64_t ldws,                   \
                                     const CTYPE* bias, CTYPE* out, int64_t ldo, void* workspace,                     \
                                     int64_t workspace_bytes, void* stream) {                                         \
        return kbit::do_linear_dynamic(                                                                               \
            Dtype::TNAME, X, ldx, MxProduct{nullptr, nullptr, w_codes, w_scales, bias, out, M, 0, 0, ldw, ldws, ldo, N, 0, false, false}, \
            K, workspace, workspace_bytes, stream);                                                                   \
    }                                                                                                                 \
    int linear_mxfp4_backward_##TNAME(const CTYPE* dout, int64_t lddo, const CTYPE* X, int64_t ldx, const CTYPE* W,   \
                                      int64_t ldw, int64_t M, int32_t N, int32_t K, CTYPE* dX, int64_t lddx,          \
                                      float* dW, int64_t lddw, float* db, void* workspace,                            \
                                      int64_t workspace_bytes, void* stream) {                                        \
        return kbit::do_linear_backward(Dtype::TNAME, dout, lddo, X, ldx, W, ldw, M, N, K, dX, lddx, dW, lddw, db,    \
                                        workspace, workspace_bytes, stream);                                          \
    }                                                                                                                 \
    int layer_norm_##TNAME(const CTYPE* x, int64_t rows, int32_t d, int64_t ldx, const void* weight,                  \
                           const void* bias, int32_t weight_fp32, float eps, CTYPE* out, int64_t ldo, void* stream) { \
        return kbit::do_layer_norm(Dtype::TNAME,                                                                      \
                                   LayerNormArgs{x, weight, bias, out, rows, ldx, ldo, d, eps, weight_fp32 != 0}, stream); \
    }                                                                                                                 \
    int layer_norm_backward_##TNAME(const CTYPE* dout, int64_t lddo, const CTYPE* x, int64_t ldx, int64_t rows,       \
                                    int32_t d, const void* weight, int32_t weight_fp32, float eps, CTYPE* dx,         \
                                    int64_t lddx, float* dweight, float* dbias, void* workspace,                      \
                                    int64_t workspace_bytes, void* stream) {                                          \
        return kbit::do_layer_norm_backward(                                                                          \
            Dtype::TNAME,                                                                                             \
            LayerNormBackArgs{dout, x, weight, dx, dweight, dbias, static_cast<float*>(workspace), rows, lddo, ldx,   \
                              lddx, d, eps, weight_fp32 != 0},                                                        \
            workspace_bytes, stream);                                                                                 \
    }

KBIT_DEFINE_MX(fp32, float)
KBIT_DEFINE_MX(fp16, uint16_t)
KBIT_DEFINE_MX(bf16, uint16_t)

}  // extern "C"
