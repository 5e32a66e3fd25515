// C ABI of include/kbit_layer.h: argument validation, device checks and
// dispatch to the HIP launchers.  As in api.cpp every entry point validates
// before it launches and reports errors as kbit_status codes; nothing aborts,
// allocates or synchronises.
#include <cmath>
#include <cstdint>

#include "int8_choice.h"
#include "kbit.h"
#include "kbit_layer.h"
#include "layer_internal.h"

namespace kbit {
namespace {

constexpr int64_t kMaxElems = int64_t(1) << 40;
constexpr int64_t kMaxRows = (int64_t(1) << 31) - 1;  // rows of heads, slots
constexpr int64_t kMaxStride = int64_t(1) << 40;
constexpr int64_t kMaxBatch = 65535;

bool aligned(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }
int64_t elem_size(Dtype t) { return t == Dtype::fp32 ? 4 : 2; }
int map_launch(int hip_status) { return hip_status == 0 ? KBIT_OK : KBIT_ELAUNCH; }
int64_t round_up(int64_t n, int64_t a) { return (n + a - 1) / a * a; }
bool stride_ok(int64_t s) { return s >= -kMaxStride && s <= kMaxStride; }

// ---------------------------------------------------------------------------
// int8 linear
// ---------------------------------------------------------------------------
bool rows_shape_ok(int64_t rows, int64_t d, int64_t ld) {
    return rows >= 0 && d >= 1 && ld >= d && ld <= kMaxElems && rows <= kMaxElems / ld;
}

// Longest row of codes: rounded up to 16 it still counts in 32 bits.
constexpr int32_t kMaxCodes = INT32_MAX - 15;

int do_quantize_rows(Dtype t, const void* X, int64_t rows, int32_t d, int64_t ldx, int8_t* codes, int64_t ldc,
                     float* scale, void* stream) {
    if (d > kMaxCodes) return KBIT_EINVAL;
    if (!rows_shape_ok(rows, d, ldx) || ldc < round_up(d, 16) || !rows_shape_ok(rows, d, ldc)) return KBIT_EINVAL;
    if (rows == 0) return KBIT_OK;
    if (!X || !codes || !scale) return KBIT_EINVAL;
    if (!aligned(X, elem_size(t)) || !aligned(codes, 16) || ldc % 16 != 0 || !aligned(scale, 4)) return KBIT_EALIGN;
    if (!device_usable()) return KBIT_EDEVICE;
    const bool vec = aligned(X, 16) && (rows == 1 || ldx * elem_size(t) % 16 == 0);
    return map_launch(launch_quantize_rows(t, X, rows, d, ldx, codes, ldc, scale, vec, stream));
}

// Shared checks of the product: 1 = go on.
int check_product(Dtype t, const Int8Product& p) {
    if (p.K < 1 || p.K > kMaxInt8Depth || p.N < 1 || !rows_shape_ok(p.M, p.K, p.ldx) ||
        !rows_shape_ok(p.N, p.K, p.ldw) || !rows_shape_ok(p.M, p.N, p.ldo) || p.M > kMaxRows)
        return KBIT_EINVAL;
    if (p.M == 0) return KBIT_OK;
    if (!p.w || !p.ws || !p.out) return KBIT_EINVAL;
    if (!aligned(p.ws, 4) || !aligned(p.out, elem_size(t)) || !aligned(p.bias, elem_size(t))) return KBIT_EALIGN;
    return 1;
}

// Both operands' rows start at multiples of 16 bytes (a single row has no
// second one to reach, whatever its distance).
bool product_aligned(const Int8Product& p) {
    return aligned(p.x, 16) && aligned(p.w, 16) && (p.M == 1 || p.ldx % 16 == 0) && (p.N == 1 || p.ldw % 16 == 0);
}

int do_linear_int8(Dtype t, const Int8Product& p, void* workspace, int64_t workspace_bytes, void* stream) {
    const int c = check_product(t, p);
    if (c != 1) return c;
    if (!p.x || !p.xs) return KBIT_EINVAL;
    const int64_t need = int8_product_workspace(p.M, p.N, p.K);
    if (workspace_bytes < need || (need > 0 && !workspace)) return KBIT_EINVAL;
    if (!aligned(p.xs, 4) || !aligned(workspace, 16)) return KBIT_EALIGN;
    if (!device_usable()) return KBIT_EDEVICE;
    return map_launch(launch_int8_product(t, p, product_aligned(p), workspace, stream));
}

int do_linear_int8_dynamic(Dtype t, const void* X, int64_t ldX, Int8Product p, void* workspace,
                           int64_t workspace_bytes, void* stream) {
    p.ldx = p.K >= 1 ? dynamic_ld(p.K) : 0;
    const int c = check_product(t, p);
    if (c != 1) return c;
    if (!X || !rows_shape_ok(p.M, p.K, ldX)) return KBIT_EINVAL;
    if (!aligned(X, elem_size(t)) || !aligned(workspace, 16)) return KBIT_EALIGN;
    const bool one_kernel = aligned(p.w, 16) && linear_int8_dynamic_fused(p.M, p.N, p.K, p.ldw);
    const DynamicParts w = dynamic_parts(p.M, p.K);
    if (!one_kernel && (!workspace || workspace_bytes < w.product + int8_product_workspace(p.M, p.N, p.K)))
        return KBIT_EINVAL;
    if (!device_usable()) return KBIT_EDEVICE;
    const bool vec = aligned(X, 16) && (p.M == 1 || ldX * elem_size(t) % 16 == 0);
    if (one_kernel) return map_launch(launch_int8_tokens(t, p, X, ldX, vec, stream));
    int8_t* codes = static_cast<int8_t*>(workspace);
    float* scale = reinterpret_cast<float*>(codes + w.scale);
    const int q = launch_quantize_rows(t, X, p.M, p.K, ldX, codes, p.ldx, scale, vec, stream);
    if (q != 0) return KBIT_ELAUNCH;
    p.x = codes;
    p.xs = scale;
    return map_launch(launch_int8_product(t, p, product_aligned(p), codes + w.product, stream));
}

// ---------------------------------------------------------------------------
// heads
// ---------------------------------------------------------------------------
struct View {  // [batch, tokens, heads, dim] with unit stride in dim
    const void* p;
    int64_t b, s, h;
};

// The vector form needs 16-byte pieces everywhere: see heads.hip.
bool vec_sizes(int dim, int rot, int layout) { return dim % 8 == 0 && rot % (layout == KBIT_ROPE_HALF ? 16 : 8) == 0; }

bool vec_view(const View& v, int64_t B, int64_t S, int64_t H, int64_t esize) {
    return aligned(v.p, 16) && (B <= 1 || v.b * esize % 16 == 0) && (S <= 1 || v.s * esize % 16 == 0) &&
           (H <= 1 || v.h * esize % 16 == 0);
}

int lanes_log2(int dim, int rot, int layout) {
    const int lanes = layout == KBIT_ROPE_HALF ? rot / 16 + (dim - rot + 15) / 16 : (dim + 15) / 16;
    int l = 0;
    while ((1 << l) < lanes) ++l;
    return l;
}

bool head_shape_ok(int64_t B, int64_t S, int32_t H, int32_t D) {
    return B >= 0 && S >= 0 && H >= 1 && D >= 1 && D <= kMaxHeadDim && B <= kMaxRows && S <= kMaxRows &&
           (B == 0 || S <= kMaxRows / B) && (B * S == 0 || H <= kMaxRows / (B * S));
}

bool view_ok(const View& v) { return stride_ok(v.b) && stride_ok(v.s) && stride_ok(v.h); }

bool rot_ok(int32_t rot, int32_t D, int64_t max_pos, int32_t layout) {
    return rot >= 2 && rot <= D && rot % 2 == 0 && max_pos >= 1 && max_pos <= kMaxElems / rot &&
           (layout == KBIT_ROPE_HALF || layout == KBIT_ROPE_INTERLEAVED);
}

bool index_bytes_ok(int32_t n) { return n == 4 || n == 8; }

// One token axis instead of batch and tokens where every view allows it: the
// batch axis is then the grid's, and is limited.
template <int N>
bool merge_batch(View* const (&v)[N], int64_t& B, int64_t& S) {
    if (S == 1) {
        for (View* x : v) x->s = x->b;
        S = B;
        B = 1;
    }
    if (B > 1) {
        bool one = true;
        for (View* x : v) one = one && x->b == S * x->s;
        if (one) {
            S *= B;
            B = 1;
        }
    }
    return B <= kMaxBatch;
}

HeadSet head_set(const View& in, const View& out, const void* weight, int heads, int dim, int rot) {
    return HeadSet{in.p, const_cast<void*>(out.p), weight, in.b, in.s, in.h, out.b, out.s, out.h, heads, dim, rot, 0};
}

int do_rope(Dtype t, View x, View out, int64_t B, int64_t S, int32_t H, int32_t D, const void* positions,
            int32_t pos_bytes, const float* table, int32_t rot, int64_t max_pos, int32_t layout, int32_t inverse,
            void* stream) {
    if (!head_shape_ok(B, S, H, D) || !rot_ok(rot, D, max_pos, layout) || !index_bytes_ok(pos_bytes) ||
        !view_ok(x) || !view_ok(out))
        return KBIT_EINVAL;
    if (B * S == 0) return KBIT_OK;
    if (!x.p || !out.p || !positions || !table) return KBIT_EINVAL;
    const int64_t es = elem_size(t);
    if (!aligned(x.p, es) || !aligned(out.p, es) || !aligned(positions, pos_bytes) || !aligned(table, 16))
        return KBIT_EALIGN;
    if (!merge_batch({&x, &out}, B, S)) return KBIT_EINVAL;
    if (!device_usable()) return KBIT_EDEVICE;
    HeadsArgs a{};
    a.set[0] = head_set(x, out, nullptr, H, D, rot);
    a.positions = positions;
    a.positions_wide = pos_bytes == 8;
    a.table = table;
    a.tokens = S;
    a.max_pos = max_pos;
    a.sign = inverse ? -1.0f : 1.0f;
    a.log2_lanes = lanes_log2(D, rot, layout);
    const bool vec = vec_sizes(D, rot, layout) && vec_view(x, B, S, H, es) && vec_view(out, B, S, H, es);
    return map_launch(launch_heads(t, a, B, HeadsKind::rope, layout, vec, stream));
}

int do_norm(Dtype t, View q, View k, View qo, View ko, int64_t B, int64_t S, int32_t Hq, int32_t Hk, int32_t D,
            const void* qw, const void* kw, int32_t weight_fp32, float eps, const void* positions, int32_t pos_bytes,
            const float* table, int32_t rot, int64_t max_pos, int32_t layout, void* stream) {
    if (!head_shape_ok(B, S, Hq, D) || !head_shape_ok(B, S, Hk, D) ||
        (B * S > 0 && static_cast<int64_t>(Hq) + Hk > kMaxRows / (B * S)) || !rot_ok(rot, D, max_pos, layout) ||
        !index_bytes_ok(pos_bytes) || !view_ok(q) || !view_ok(k) || !view_ok(qo) || !view_ok(ko) || !(eps >= 0.0f) ||
        std::isinf(eps))
        return KBIT_EINVAL;
    if (B * S == 0) return KBIT_OK;
    if (!q.p || !k.p || !qo.p || !ko.p || !qw || !kw || !positions || !table) return KBIT_EINVAL;
    const int64_t es = elem_size(t), ws = weight_fp32 ? 4 : es;
    if (!aligned(q.p, es) || !aligned(k.p, es) || !aligned(qo.p, es) || !aligned(ko.p, es) || !aligned(qw, ws) ||
        !aligned(kw, ws) || !aligned(positions, pos_bytes) || !aligned(table, 16))
        return KBIT_EALIGN;
    if (!merge_batch({&q, &k, &qo, &ko}, B, S)) return KBIT_EINVAL;
    if (!device_usable()) return KBIT_EDEVICE;
    HeadsArgs a{};
    a.set[0] = head_set(q, qo, qw, Hq, D, rot);
    a.set[1] = head_set(k, ko, kw, Hk, D, rot);
    a.positions = positions;
    a.positions_wide = pos_bytes == 8;
    a.table = table;
    a.tokens = S;
    a.max_pos = max_pos;
    a.sign = 1.0f;
    a.eps = eps;
    a.inv_dim = 1.0f / static_cast<float>(D);
    a.weight_fp32 = weight_fp32 != 0 || t == Dtype::fp32;
    a.log2_lanes = lanes_log2(D, rot, layout);
    const bool vec = vec_sizes(D, rot, layout) && vec_view(q, B, S, Hq, es) && vec_view(k, B, S, Hk, es) &&
                     vec_view(qo, B, S, Hq, es) && vec_view(ko, B, S, Hk, es) && aligned(qw, 16) && aligned(kw, 16);
    return map_launch(launch_heads(t, a, B, HeadsKind::norm, layout, vec, stream));
}

BackSet back_set(const View& x, const View& g, const View& dx, const void* w, int heads, int64_t tokens) {
    return BackSet{x.p, g.p, w, const_cast<void*>(dx.p), x.b, x.s, x.h, g.b, g.s, g.h, dx.b, dx.s, dx.h, heads,
                   static_cast<uint32_t>(tokens * heads)};
}

int do_norm_back(Dtype t, View gq, View gk, View q, View k, View dq, View dk, int64_t B, int64_t S, int32_t Hq,
                 int32_t Hk, int32_t D, const void* qw, const void* kw, int32_t weight_fp32, float* dqw, float* dkw,
                 float eps, const void* positions, int32_t pos_bytes, const float* table, int32_t rot,
                 int64_t max_pos, int32_t layout, void* workspace, int64_t workspace_bytes, void* stream) {
    if (!head_shape_ok(B, S, Hq, D) || !head_shape_ok(B, S, Hk, D) || !rot_ok(rot, D, max_pos, layout) ||
        !index_bytes_ok(pos_bytes) || !view_ok(gq) || !view_ok(gk) || !view_ok(q) || !view_ok(k) || !view_ok(dq) ||
        !view_ok(dk) || !(eps >= 0.0f) || std::isinf(eps))
        return KBIT_EINVAL;
    if (!dqw || !dkw || !workspace || workspace_bytes < qk_norm_rope_backward_workspace_bytes(D)) return KBIT_EINVAL;
    const bool any = B * S > 0;  // without tokens the weights' gradients are still written, as zeros
    if (!qw || !kw || (any && (!gq.p || !gk.p || !q.p || !k.p || !dq.p || !dk.p || !positions || !table)))
        return KBIT_EINVAL;
    const int64_t es = elem_size(t), ws = weight_fp32 ? 4 : es;
    if (!aligned(qw, ws) || !aligned(kw, ws) || !aligned(dqw, 4) || !aligned(dkw, 4) || !aligned(workspace, 16) ||
        !aligned(gq.p, es) || !aligned(gk.p, es) || !aligned(q.p, es) || !aligned(k.p, es) || !aligned(dq.p, es) ||
        !aligned(dk.p, es) || !aligned(positions, pos_bytes) || !aligned(table, 16))
        return KBIT_EALIGN;
    if (!device_usable()) return KBIT_EDEVICE;
    NormBackArgs a{};
    a.set[0] = back_set(q, gq, dq, qw, Hq, B * S);
    a.set[1] = back_set(k, gk, dk, kw, Hk, B * S);
    a.positions = positions;
    a.positions_wide = pos_bytes == 8;
    a.table = table;
    a.partial = static_cast<float*>(workspace);
    a.max_pos = max_pos;
    a.tokens = S > 0 ? S : 1;
    a.dim = D;
    a.rot = rot;
    a.eps = eps;
    a.inv_dim = 1.0f / static_cast<float>(D);
    a.weight_fp32 = weight_fp32 != 0 || t == Dtype::fp32;
    a.log2_lanes = lanes_log2(D, rot, layout);
    const bool vec = vec_sizes(D, rot, layout) && vec_view(gq, B, S, Hq, es) && vec_view(gk, B, S, Hk, es) &&
                     vec_view(q, B, S, Hq, es) && vec_view(k, B, S, Hk, es) && vec_view(dq, B, S, Hq, es) &&
                     vec_view(dk, B, S, Hk, es) && aligned(qw, 16) && aligned(kw, 16);
    return map_launch(launch_norm_back(t, a, layout, vec, dqw, dkw, stream));
}

int do_append(Dtype t, View k, View v, int64_t T, int32_t H, int32_t D, int32_t Dv, const void* slots,
              int32_t slot_bytes, View kc, View vc, int64_t pages, int32_t page_size, const void* positions,
              int32_t pos_bytes, const float* table, int32_t rot, int64_t max_pos, int32_t layout, void* stream) {
    if (!head_shape_ok(1, T, H, D) || !head_shape_ok(1, T, H, Dv) || (T > 0 && 2 * static_cast<int64_t>(H) > kMaxRows / T) ||
        !index_bytes_ok(slot_bytes) || pages < 0 || page_size < 1 || pages > kMaxRows / page_size || !view_ok(k) ||
        !view_ok(v) || !view_ok(kc) || !view_ok(vc))
        return KBIT_EINVAL;
    if (rot == 0) layout = KBIT_ROPE_HALF;  // no rotation: keys are copied like values
    if (rot != 0 && (!rot_ok(rot, D, max_pos, layout) || !index_bytes_ok(pos_bytes))) return KBIT_EINVAL;
    if (T == 0 || pages == 0) return KBIT_OK;
    if (!k.p || !v.p || !kc.p || !vc.p || !slots || (rot != 0 && (!positions || !table))) return KBIT_EINVAL;
    const int64_t es = elem_size(t);
    if (!aligned(k.p, es) || !aligned(v.p, es) || !aligned(kc.p, es) || !aligned(vc.p, es) ||
        !aligned(slots, slot_bytes) || (rot != 0 && (!aligned(positions, pos_bytes) || !aligned(table, 16))))
        return KBIT_EALIGN;
    if (!device_usable()) return KBIT_EDEVICE;
    HeadsArgs a{};
    a.set[0] = head_set(k, kc, nullptr, H, D, rot);
    a.set[1] = head_set(v, vc, nullptr, H, Dv, 0);
    a.positions = positions;
    a.positions_wide = pos_bytes == 8;
    a.slots = slots;
    a.slots_wide = slot_bytes == 8;
    a.n_slots = pages * page_size;
    a.page_size = page_size;
    a.table = table;
    a.tokens = T;
    a.max_pos = max_pos;
    a.sign = 1.0f;
    const int lk = lanes_log2(D, rot, layout), lv = lanes_log2(Dv, 0, layout);
    a.log2_lanes = lk > lv ? lk : lv;
    const bool vec = vec_sizes(D, rot, layout) && vec_sizes(Dv, 0, layout) && vec_view(k, 1, T, H, es) &&
                     vec_view(v, 1, T, H, es) && vec_view(kc, pages, page_size, H, es) &&
                     vec_view(vc, pages, page_size, H, es);
    return map_launch(launch_heads(t, a, 1, HeadsKind::append, layout, vec, stream));
}

}  // namespace
}  // namespace kbit

using kbit::Dtype;
using kbit::Int8Product;
using kbit::View;

extern "C" {

int64_t linear_int8_workspace_bytes(int64_t M, int32_t N, int32_t K) {
    if (M < 0 || M > kbit::kMaxRows || N < 1 || K < 1 || K > kbit::kMaxInt8Depth) return -1;
    return kbit::int8_product_workspace_up_to(M, N, K);
}

int64_t linear_int8_dynamic_workspace_bytes(int64_t M, int32_t N, int32_t K) {
    if (M < 0 || M > kbit::kMaxRows || N < 1 || K < 1 || K > kbit::kMaxInt8Depth) return -1;
    return kbit::dynamic_parts(M, K).product + kbit::int8_product_workspace_up_to(M, N, K);
}

int linear_int8_dynamic_fused(int64_t M, int32_t N, int32_t K, int64_t ldw) {
    return M >= 1 && M <= kbit::kMaxRows && N >= 1 && K >= 1 && K <= kbit::kMaxInt8Depth &&
           (N == 1 || ldw % 16 == 0) && kbit::int8_tokens_fit(M, N, K, ldw);
}

int64_t qk_norm_rope_backward_workspace_bytes(int32_t D) {
    if (D < 1 || D > kbit::kMaxHeadDim) return -1;
    return static_cast<int64_t>(kbit::kNormBackGroups + 2) * D * 4;
}

int rope_frequencies(int32_t rot, double base, int32_t scaling, double factor, double original_length,
                     double slow_turns, double fast_turns, double* freq, double* amplitude) {
    if (rot < 2 || rot % 2 != 0 || rot > kbit::kMaxHeadDim || !(base > 1.0) || std::isinf(base) || !freq || !amplitude)
        return KBIT_EINVAL;
    if (scaling < KBIT_ROPE_UNSCALED || scaling > KBIT_ROPE_YARN) return KBIT_EINVAL;
    if (scaling != KBIT_ROPE_UNSCALED && (!(factor >= 1.0) || std::isinf(factor))) return KBIT_EINVAL;
    if (scaling == KBIT_ROPE_YARN &&
        (!(original_length >= 1.0) || std::isinf(original_length) || !(slow_turns >= 0.0) ||
         !(fast_turns > slow_turns) || std::isinf(fast_turns)))
        return KBIT_EINVAL;
    const double pi = 3.14159265358979323846;
    if (scaling == KBIT_ROPE_NTK && rot > 2) base *= std::pow(factor, rot / (rot - 2.0));
    for (int i = 0; i < rot / 2; ++i) {
        double f = std::pow(base, -2.0 * i / rot);
        if (scaling == KBIT_ROPE_LINEAR) f /= factor;
        if (scaling == KBIT_ROPE_YARN) {
            const double turns = original_length * f / (2.0 * pi);
            double keep = (turns - slow_turns) / (fast_turns - slow_turns);
            keep = keep < 0.0 ? 0.0 : keep > 1.0 ? 1.0 : keep;
            f = keep * f + (1.0 - keep) * f / factor;
        }
        freq[i] = f;
    }
    *amplitude = scaling == KBIT_ROPE_YARN ? 0.1 * std::log(factor) + 1.0 : 1.0;
    return KBIT_OK;
}

int rope_table(const double* freq, int32_t rot, int64_t max_pos, double amplitude, float* table, void* stream) {
    if (rot < 2 || rot % 2 != 0 || rot > kbit::kMaxHeadDim || max_pos < 1 || max_pos > kbit::kMaxElems / rot ||
        !std::isfinite(amplitude) || !freq || !table)
        return KBIT_EINVAL;
    if (!kbit::aligned(freq, 8) || !kbit::aligned(table, 16)) return KBIT_EALIGN;
    if (!kbit::device_usable()) return KBIT_EDEVICE;
    return kbit::map_launch(kbit::launch_rope_table(freq, rot, max_pos, amplitude, table, stream));
}

#define KBIT_DEFINE_LAYER(TNAME, CTYPE)                                                                               \
    int quantize_rows_int8_##TNAME(const CTYPE* X, int64_t rows, int32_t d, int64_t ldx, int8_t* codes, int64_t ldc,  \
                                   float* scale, void* stream) {                                                      \
        return kbit::do_quantize_rows(Dtype::TNAME, X, rows, d, ldx, codes, ldc, scale, stream);                      \
    }                                                                                                                 \
    int linear_int8_##TNAME(const int8_t* codes, const float* scale, int64_t M, int32_t K, int64_t ldx,               \
                            const int8_t* w_codes, const float* w_scale, int32_t N, int64_t ldw, const CTYPE* bias,   \
                            CTYPE* out, int64_t ldo, void* workspace, int64_t workspace_bytes, void* stream) {        \
        return kbit::do_linear_int8(Dtype::TNAME,                                                                     \
                                    Int8Product{codes, scale, w_codes, w_scale, bias, out, M, ldx, ldw, ldo, N, K},   \
                                    workspace, workspace_bytes, stream);                                              \
    }                                                                                                                 \
    int linear_int8_dynamic_##TNAME(const CTYPE* X, int64_t M, int32_t K, int64_t ldx, const int8_t* w_codes,         \
                                    const float* w_scale, int32_t N, int64_t ldw, const CTYPE* bias, CTYPE* out,      \
                                    int64_t ldo, void* workspace, int64_t workspace_bytes, void* stream) {            \
        return kbit::do_linear_int8_dynamic(                                                                          \
            Dtype::TNAME, X, ldx, Int8Product{nullptr, nullptr, w_codes, w_scale, bias, out, M, 0, ldw, ldo, N, K},   \
            workspace, workspace_bytes, stream);                                                                      \
    }                                                                                                                 \
    int rope_##TNAME(const CTYPE* x, int64_t x_batch, int64_t x_token, int64_t x_head, CTYPE* out, int64_t out_batch, \
                     int64_t out_token, int64_t out_head, int64_t batch, int64_t tokens, int32_t heads, int32_t dim,  \
                     const void* positions, int32_t position_bytes, const float* table, int32_t rot,                  \
                     int64_t max_pos, int32_t layout, int32_t inverse, void* stream) {                                \
        return kbit::do_rope(Dtype::TNAME, View{x, x_batch, x_token, x_head},                                         \
                             View{out, out_batch, out_token, out_head}, batch, tokens, heads, dim, positions,         \
                             position_bytes, table, rot, max_pos, layout, inverse, stream);                           \
    }                                                                                                                 \
    int qk_norm_rope_##TNAME(const CTYPE* q, int64_t q_batch, int64_t q_token, int64_t q_head, const CTYPE* k,        \
                             int64_t k_batch, int64_t k_token, int64_t k_head, CTYPE* q_out, int64_t qo_batch,        \
                             int64_t qo_token, int64_t qo_head, CTYPE* k_out, int64_t ko_batch, int64_t ko_token,     \
                             int64_t ko_head, int64_t batch, int64_t tokens, int32_t q_heads, int32_t k_heads,        \
                             int32_t dim, const void* q_weight, const void* k_weight, int32_t weight_fp32, float eps, \
                             const void* positions, int32_t position_bytes, const float* table, int32_t rot,          \
                             int64_t max_pos, int32_t layout, void* stream) {                                         \
        return kbit::do_norm(Dtype::TNAME, View{q, q_batch, q_token, q_head}, View{k, k_batch, k_token, k_head},      \
                             View{q_out, qo_batch, qo_token, qo_head}, View{k_out, ko_batch, ko_token, ko_head},      \
                             batch, tokens, q_heads, k_heads, dim, q_weight, k_weight, weight_fp32, eps, positions,   \
                             position_bytes, table, rot, max_pos, layout, stream);                                    \
    }                                                                                                                 \
    int qk_norm_rope_backward_##TNAME(                                                                                \
        const CTYPE* gq, int64_t gq_batch, int64_t gq_token, int64_t gq_head, const CTYPE* gk, int64_t gk_batch,      \
        int64_t gk_token, int64_t gk_head, const CTYPE* q, int64_t q_batch, int64_t q_token, int64_t q_head,          \
        const CTYPE* k, int64_t k_batch, int64_t k_token, int64_t k_head, CTYPE* dq, int64_t dq_batch,                \
        int64_t dq_token, int64_t dq_head, CTYPE* dk, int64_t dk_batch, int64_t dk_token, int64_t dk_head,            \
        int64_t batch, int64_t tokens, int32_t q_heads, int32_t k_heads, int32_t dim, const void* q_weight,           \
        const void* k_weight, int32_t weight_fp32, float* dq_weight, float* dk_weight, float eps,                     \
        const void* positions, int32_t position_bytes, const float* table, int32_t rot, int64_t max_pos,              \
        int32_t layout, void* workspace, int64_t workspace_bytes, void* stream) {                                     \
        return kbit::do_norm_back(                                                                                    \
            Dtype::TNAME, View{gq, gq_batch, gq_token, gq_head}, View{gk, gk_batch, gk_token, gk_head},               \
            View{q, q_batch, q_token, q_head}, View{k, k_batch, k_token, k_head},                                     \
            View{dq, dq_batch, dq_token, dq_head}, View{dk, dk_batch, dk_token, dk_head}, batch, tokens, q_heads,     \
            k_heads, dim, q_weight, k_weight, weight_fp32, dq_weight, dk_weight, eps, positions, position_bytes,      \
            table, rot, max_pos, layout, workspace, workspace_bytes, stream);                                         \
    }                                                                                                                 \
    int append_kv_paged_##TNAME(const CTYPE* k, int64_t k_token, int64_t k_head, const CTYPE* v, int64_t v_token,     \
                                int64_t v_head, int64_t tokens, int32_t heads, int32_t k_dim, int32_t v_dim,          \
                                const void* slots, int32_t slot_bytes, CTYPE* k_cache, int64_t kc_page,               \
                                int64_t kc_slot, int64_t kc_head, CTYPE* v_cache, int64_t vc_page, int64_t vc_slot,   \
                                int64_t vc_head, int64_t pages, int32_t page_size, const void* positions,             \
                                int32_t position_bytes, const float* table, int32_t rot, int64_t max_pos,             \
                                int32_t layout, void* stream) {                                                       \
        return kbit::do_append(Dtype::TNAME, View{k, 0, k_token, k_head}, View{v, 0, v_token, v_head}, tokens, heads, \
                               k_dim, v_dim, slots, slot_bytes, View{k_cache, kc_page, kc_slot, kc_head},             \
                               View{v_cache, vc_page, vc_slot, vc_head}, pages, page_size, positions, position_bytes, \
                               table, rot, max_pos, layout, stream);                                                  \
    }

KBIT_DEFINE_LAYER(fp32, float)
KBIT_DEFINE_LAYER(fp16, uint16_t)
KBIT_DEFINE_LAYER(bf16, uint16_t)

}  // extern "C"
