// The Python binding of include/kbit_layer.h for torch tensors: checks,
// output allocation and the C calls, on torch's current stream of the
// inputs' device.  It is C++ because the smallest calls last a few
// microseconds on the GPU: through ctypes and checks in Python a call cost
// 9 us (rotation) to 27 us (norm gradient) of host time, more than its
// kernels; layer.py holds the functions' documented signatures.
//
// Every function checks all it passes on (the C ABI sees raw addresses):
// types and shapes raise TypeError and ValueError, a status of the library
// KbitError.  No C++ exception leaves a function.
//
// Nothing is recorded for autograd, but it is not left in the dark: whatever
// was written counts as modified in place, and a call that cuts a gradient
// off says so.
#include "bind.h"
#include "int8_choice.h"
#include "kbit_layer.h"

namespace {

// ---------------------------------------------------------------------------
// int8 linear
// ---------------------------------------------------------------------------
int64_t up16(int64_t n) { return (n + 15) / 16 * 16; }

PyObject* quantize_rows(PyObject* const* a) {
    const Tensor& X = tensor(a[0], "X");
    const int64_t ldx = rows_of(X, "X", is_float(X.scalar_type()), kFloats);
    const int64_t rows = X.size(0), d = X.size(1), whole = up16(d);
    if (d < 1) value_error("X must have at least one column");
    Tensor codes, scale;
    int64_t ldc = whole;
    if (a[1] == Py_None) {
        codes = at::empty({rows, whole}, X.options().dtype(at::kChar)).narrow(1, 0, d);
    } else {
        codes = tensor(a[1], "codes");
        ldc = rows_of(codes, "codes", codes.scalar_type() == at::kChar, "int8");
        same_shape(codes, "codes", X.sizes());
        same_device(codes, "codes", X);
        if (rows <= 1 && ldc < whole) ldc = whole;
        const int64_t room = static_cast<int64_t>(codes.storage().nbytes()) - codes.storage_offset();
        if (rows > 0 && room < (rows - 1) * ldc + whole)
            value_error("codes: every row needs room up to the next multiple of 16 bytes");
    }
    if (a[2] == Py_None) scale = at::empty({rows}, X.options().dtype(at::kFloat));
    else vector(a[2], "scale", at::kFloat, rows, X), scale = THPVariable_Unpack(a[2]);
    const int di = fits_int(d, "the number of columns");
    KBIT_BY_TYPE(X.scalar_type(), quantize_rows_int8, run("quantize_rows_int8", X, {&codes, &scale}, [&](void* stream) {
        return fn(static_cast<const T*>(X.data_ptr()), rows, di, ldx, static_cast<int8_t*>(codes.data_ptr()), ldc,
                  static_cast<float*>(scale.data_ptr()), stream);
    }))
    return wrap({codes, scale});
}

// The weight's side of a product, and its output.
struct Weight {
    const int8_t* codes;
    const float* scale;
    const void* bias;
    int64_t ldw, ldo;
    int N, K;
    Tensor out;
};

Weight weight(const Tensor& x, PyObject* codes, PyObject* scale, PyObject* bias, PyObject* out, at::ScalarType type,
              const char* what) {
    Weight w;
    const Tensor& c = tensor(codes, "w_codes");
    w.ldw = rows_of(c, "w_codes", c.scalar_type() == at::kChar, "int8");
    const int64_t M = x.size(0), K = x.size(1), N = c.size(0);
    if (c.size(1) != K) value_error(cat("w_codes: rows of ", c.size(1), " codes, ", what, " has ", K));
    if (N < 1 || K < 1) value_error("the weight must have at least one row and one column");
    same_device(c, "w_codes", x);
    w.N = fits_int(N, "the number of output channels");
    w.K = fits_int(K, "the depth");
    w.codes = static_cast<const int8_t*>(c.data_ptr());
    w.scale = static_cast<const float*>(channel_vector(scale, "w_scale", at::kFloat, N, x));
    w.bias = bias == Py_None ? nullptr : channel_vector(bias, "bias", type, N, x);
    if (out == Py_None) {
        w.out = at::empty({M, N}, x.options().dtype(type));
        w.ldo = N;
    } else {
        w.out = tensor(out, "out");
        w.ldo = rows_of(w.out, "out", w.out.scalar_type() == type, at::toString(type));
        same_shape(w.out, "out", {M, N});
        same_device(w.out, "out", x);
    }
    return w;
}

PyObject* linear(PyObject* const* a) {  // codes, scale, w_codes, w_scale, bias, dtype, out, workspace
    const Tensor& x = tensor(a[0], "codes");
    const int64_t ldx = rows_of(x, "codes", x.scalar_type() == at::kChar, "int8"), M = x.size(0);
    if (!THPDtype_Check(a[5])) type_error("dtype must be a torch.dtype");
    const at::ScalarType type = reinterpret_cast<THPDtype*>(a[5])->scalar_type;
    if (!is_float(type)) type_error(cat("unsupported element dtype ", type));
    const Weight w = weight(x, a[2], a[3], a[4], a[6], type, "codes");
    const float* scale = static_cast<const float*>(vector(a[1], "scale", at::kFloat, M, x));
    const int64_t need = linear_int8_workspace_bytes(M, w.N, w.K);
    const Space ws = workspace(need, need > 0 ? kbit::int8_product_workspace(M, w.N, w.K) : 0, a[7], "linear_int8", x);
    KBIT_BY_TYPE(type, linear_int8, run("linear_int8", x, {&w.out}, [&](void* stream) {
        return fn(static_cast<const int8_t*>(x.data_ptr()), scale, M, w.K, ldx, w.codes, w.scale, w.N, w.ldw,
                  static_cast<const T*>(w.bias), static_cast<T*>(w.out.data_ptr()), w.ldo, ws.p, ws.bytes, stream);
    }))
    return wrap(w.out);
}

PyObject* linear_dynamic(PyObject* const* a) {  // X, w_codes, w_scale, bias, out, workspace
    const Tensor& x = tensor(a[0], "X");
    const at::ScalarType type = x.scalar_type();
    const int64_t ldx = rows_of(x, "X", is_float(type), kFloats), M = x.size(0);
    const Weight w = weight(x, a[1], a[2], a[3], a[4], type, "X");
    no_overlap(w.out, "out", x, "X", false);
    if (M == 0) return wrap(w.out);
    const bool fused = reinterpret_cast<uintptr_t>(w.codes) % 16 == 0 && linear_int8_dynamic_fused(M, w.N, w.K, w.ldw);
    const int64_t need = fused ? 0 : linear_int8_dynamic_workspace_bytes(M, w.N, w.K);
    const int64_t take = need <= 0 ? 0 : kbit::dynamic_parts(M, w.K).product + kbit::int8_product_workspace(M, w.N, w.K);
    const Space ws = workspace(need, take, a[5], "linear_int8_dynamic", x);
    KBIT_BY_TYPE(type, linear_int8_dynamic, run("linear_int8_dynamic", x, {&w.out}, [&](void* stream) {
        return fn(static_cast<const T*>(x.data_ptr()), M, w.K, ldx, w.codes, w.scale, w.N, w.ldw,
                  static_cast<const T*>(w.bias), static_cast<T*>(w.out.data_ptr()), w.ldo, ws.p, ws.bytes, stream);
    }))
    return wrap(w.out);
}

// ---------------------------------------------------------------------------
// heads
// ---------------------------------------------------------------------------
// [.., tokens, heads, dim] with contiguous heads.
struct View {
    void* p;
    int64_t batch, token, head;
};

View view(const Tensor& t) {
    const auto st = t.strides();
    return t.dim() == 3 ? View{t.data_ptr(), 0, st[0], st[1]} : View{t.data_ptr(), st[0], st[1], st[2]};
}

const Tensor& heads(PyObject* o, const char* what, const Tensor* like) {
    const Tensor& t = tensor(o, what);
    const at::ScalarType type = t.scalar_type();
    if (like ? type != like->scalar_type() : !is_float(type))
        type_error(cat(what, ": element type ", type, ", expected ", like ? at::toString(like->scalar_type()) : kFloats));
    if (t.dim() != 3 && t.dim() != 4)
        value_error(cat(what, " must be [tokens, heads, dim] or [batch, tokens, heads, dim]"));
    on_gpu(t, what);
    if (t.size(-1) > 1 && t.stride(-1) != 1) value_error(cat(what, ": the elements of a head must be contiguous"));
    if (like) same_device(t, what, *like);
    return t;
}

// An output shaped like x: new, in x's layout where that is dense, or given
// (it may be x).
Tensor out_like(const Tensor& x, PyObject* given, const char* what, const char* name) {
    if (given == Py_None) {
        Tensor out = at::empty_like(x);
        if (out.size(-1) > 1 && out.stride(-1) != 1) out = at::empty(x.sizes(), x.options());
        return out;
    }
    const Tensor& out = heads(given, what, &x);
    same_shape(out, what, x.sizes());
    no_overlap(out, what);
    no_overlap(out, what, x, name, true);
    return out;
}

// A contiguous int32 or int64 tensor of a shape.
struct Index {
    const void* p = nullptr;
    int bytes = 0;
};

Index index(PyObject* o, const char* what, at::IntArrayRef shape, const Tensor& ref) {
    const bool is = THPVariable_Check(o);
    const at::ScalarType type = is ? THPVariable_Unpack(o).scalar_type() : at::kFloat;
    if (type != at::kInt && type != at::kLong) type_error(cat(what, " must be an int32 or int64 tensor"));
    const Tensor& t = THPVariable_Unpack(o);
    same_shape(t, what, shape);
    same_device(t, what, ref);
    if (!t.is_contiguous()) value_error(cat(what, ": tensor must be contiguous"));
    return Index{t.data_ptr(), type == at::kLong ? 8 : 4};
}

struct Turn {
    Index positions;
    const float* table = nullptr;
    int rot = 0, layout = 0;
    int64_t max_pos = 0;
};

Turn turn(PyObject* positions, PyObject* table, PyObject* layout, const Tensor& x) {
    Turn r;
    if (PyUnicode_Check(layout) && PyUnicode_CompareWithASCIIString(layout, "half") == 0) r.layout = KBIT_ROPE_HALF;
    else if (PyUnicode_Check(layout) && PyUnicode_CompareWithASCIIString(layout, "interleaved") == 0)
        r.layout = KBIT_ROPE_INTERLEAVED;
    else value_error("layout must be 'half' or 'interleaved'");
    if (!THPVariable_Check(table) || THPVariable_Unpack(table).scalar_type() != at::kFloat ||
        THPVariable_Unpack(table).dim() != 2)
        type_error("table must be the 2-D float32 tensor of rope_table");
    const Tensor& t = THPVariable_Unpack(table);
    if (t.size(1) > x.size(-1)) value_error(cat("table rotates ", t.size(1), " elements, a head has ", x.size(-1)));
    if (!t.is_contiguous()) value_error("table: tensor must be contiguous");
    same_device(t, "table", x);
    r.table = static_cast<const float*>(t.data_ptr());
    r.max_pos = t.size(0);
    r.rot = fits_int(t.size(1), "table");
    r.positions = index(positions, "positions", x.sizes().slice(0, x.dim() - 2), x);
    return r;
}

#define KBIT_VIEW(T, v) static_cast<T*>((v).p), (v).batch, (v).token, (v).head

PyObject* rope(PyObject* const* a) {  // x, positions, table, layout, inverse, out
    const Tensor& x = heads(a[0], "x", nullptr);
    const Turn t = turn(a[1], a[2], a[3], x);
    const int inverse = PyObject_IsTrue(a[4]);
    if (inverse < 0) throw Raise{nullptr, ""};
    const Tensor out = out_like(x, a[5], "out", "x");
    const View vx = view(x), vo = view(out);
    const int64_t batch = x.dim() == 4 ? x.size(0) : 1, tokens = x.size(-3);
    const int h = fits_int(x.size(-2), "the number of heads"), dim = fits_int(x.size(-1), "the head's size");
    KBIT_BY_TYPE(x.scalar_type(), rope, run("rope", x, {&out}, [&](void* stream) {
        return fn(KBIT_VIEW(const T, vx), KBIT_VIEW(T, vo), batch, tokens, h, dim, t.positions.p, t.positions.bytes,
                  t.table, t.rot, t.max_pos, t.layout, inverse, stream);
    }))
    return wrap(out);
}

struct Norm {
    const Tensor &q, &k;
    int64_t batch, tokens;
    int q_heads, k_heads, dim, weight_fp32;
    const void *qw, *kw;
};

Norm norm_inputs(PyObject* qo, PyObject* ko, PyObject* qw, PyObject* kw) {
    const Tensor& q = heads(qo, "q", nullptr);
    const Tensor& k = heads(ko, "k", &q);
    const int64_t n = q.dim();
    if (k.dim() != n || k.sizes().slice(0, n - 2) != q.sizes().slice(0, n - 2) || k.size(-1) != q.size(-1))
        value_error(cat("q ", q.sizes(), " and k ", k.sizes(), " may differ in their heads only"));
    const at::ScalarType wt = THPVariable_Check(qw) ? THPVariable_Unpack(qw).scalar_type() : at::kByte;
    if (wt != q.scalar_type() && wt != at::kFloat)
        type_error(cat("q_weight must be a ", q.scalar_type(), " or float32 tensor"));
    const int dim = fits_int(q.size(-1), "the head's size");
    const void* pq = vector(qw, "q_weight", wt, dim, q);
    const void* pk = vector(kw, "k_weight", wt, dim, q);
    if (THPVariable_Unpack(qw).numel() != dim || THPVariable_Unpack(kw).numel() != dim)
        value_error(cat("q_weight and k_weight must have ", dim, " elements"));
    return Norm{q, k, n == 4 ? q.size(0) : 1, q.size(-3), fits_int(q.size(-2), "the number of heads"),
                fits_int(k.size(-2), "the number of heads"), dim, wt == at::kFloat ? 1 : 0, pq, pk};
}

PyObject* norm_rope(PyObject* const* a) {  // q, k, q_weight, k_weight, positions, table, eps, layout, q_out, k_out
    const Norm n = norm_inputs(a[0], a[1], a[2], a[3]);
    const Turn t = turn(a[4], a[5], a[7], n.q);
    const float eps = number(a[6], "eps");
    const Tensor qo = out_like(n.q, a[8], "q_out", "q"), ko = out_like(n.k, a[9], "k_out", "k");
    no_overlap(qo, "q_out", n.k, "k", false);
    no_overlap(ko, "k_out", n.q, "q", false);
    no_overlap(qo, "q_out", ko, "k_out", false);
    const View vq = view(n.q), vk = view(n.k), vqo = view(qo), vko = view(ko);
    KBIT_BY_TYPE(n.q.scalar_type(), qk_norm_rope, run("qk_norm_rope", n.q, {&qo, &ko}, [&](void* stream) {
        return fn(KBIT_VIEW(const T, vq), KBIT_VIEW(const T, vk), KBIT_VIEW(T, vqo), KBIT_VIEW(T, vko), n.batch, n.tokens,
                  n.q_heads, n.k_heads, n.dim, n.qw, n.kw, n.weight_fp32, eps, t.positions.p, t.positions.bytes, t.table,
                  t.rot, t.max_pos, t.layout, stream);
    }))
    return wrap({qo, ko});
}

// dq_out, dk_out, q, k, q_weight, k_weight, positions, table, eps, layout, dq, dk, workspace
PyObject* norm_rope_backward(PyObject* const* a) {
    const Norm n = norm_inputs(a[2], a[3], a[4], a[5]);
    const Turn t = turn(a[6], a[7], a[9], n.q);
    const float eps = number(a[8], "eps");
    const Tensor& gq = heads(a[0], "dq_out", &n.q);
    const Tensor& gk = heads(a[1], "dk_out", &n.q);
    same_shape(gq, "dq_out", n.q.sizes());
    same_shape(gk, "dk_out", n.k.sizes());
    const Tensor dq = out_like(n.q, a[10], "dq", "q"), dk = out_like(n.k, a[11], "dk", "k");
    no_overlap(dq, "dq", gq, "dq_out", true);
    no_overlap(dk, "dk", gk, "dk_out", true);
    for (const auto& [t, name] : {std::pair<const Tensor&, const char*>{n.k, "k"}, {gk, "dk_out"}, {dk, "dk"}})
        no_overlap(dq, "dq", t, name, false);
    no_overlap(dk, "dk", n.q, "q", false);
    no_overlap(dk, "dk", gq, "dq_out", false);
    const Tensor dqw = at::empty({n.dim}, n.q.options().dtype(at::kFloat)), dkw = at::empty_like(dqw);
    const int64_t need = qk_norm_rope_backward_workspace_bytes(n.dim);
    const Space ws = workspace(need, need, a[12], "qk_norm_rope_backward", n.q);
    const View vgq = view(gq), vgk = view(gk), vq = view(n.q), vk = view(n.k), vdq = view(dq), vdk = view(dk);
    KBIT_BY_TYPE(n.q.scalar_type(), qk_norm_rope_backward, run("qk_norm_rope_backward", n.q, {&dq, &dk}, [&](void* stream) {
        return fn(KBIT_VIEW(const T, vgq), KBIT_VIEW(const T, vgk), KBIT_VIEW(const T, vq), KBIT_VIEW(const T, vk),
                  KBIT_VIEW(T, vdq), KBIT_VIEW(T, vdk), n.batch, n.tokens, n.q_heads, n.k_heads, n.dim, n.qw, n.kw,
                  n.weight_fp32, static_cast<float*>(dqw.data_ptr()), static_cast<float*>(dkw.data_ptr()), eps,
                  t.positions.p, t.positions.bytes, t.table, t.rot, t.max_pos, t.layout, ws.p, ws.bytes, stream);
    }))
    return wrap({dq, dk, dqw, dkw});
}

PyObject* append(PyObject* const* a) {  // k, v, slots, k_cache, v_cache, positions, table, layout
    const Tensor& k = heads(a[0], "k", nullptr);
    const Tensor& v = heads(a[1], "v", &k);
    const Tensor& kc = heads(a[3], "k_cache", &k);
    const Tensor& vc = heads(a[4], "v_cache", &k);
    if (k.dim() != 3 || v.dim() != 3 || v.size(0) != k.size(0) || v.size(1) != k.size(1))
        value_error(cat("k ", k.sizes(), " and v ", v.sizes(),
                        " must be [tokens, heads, dim], and differ in dim at most"));
    if (kc.dim() != 4 || kc.size(2) != k.size(1) || kc.size(3) != k.size(2))
        value_error(cat("k_cache: shape ", kc.sizes(), ", expected [pages, page_size, ", k.size(1), ", ", k.size(2), "]"));
    if (vc.dim() != 4 || vc.size(0) != kc.size(0) || vc.size(1) != kc.size(1) || vc.size(2) != k.size(1) ||
        vc.size(3) != v.size(2))
        value_error(cat("v_cache: shape ", vc.sizes(), ", expected [", kc.size(0), ", ", kc.size(1), ", ", k.size(1), ", ",
                        v.size(2), "]"));
    const Index slots = index(a[2], "slots", k.sizes().slice(0, 1), k);
    if ((a[5] == Py_None) != (a[6] == Py_None)) type_error("give both positions and table, or neither");
    const Turn t = a[6] == Py_None ? Turn{} : turn(a[5], a[6], a[7], k);
    const int h = fits_int(k.size(1), "the number of heads"), dim = fits_int(k.size(2), "the head's size"),
              v_dim = fits_int(v.size(2), "the head's size"), page = fits_int(kc.size(1), "page_size");
    const View vk = view(k), vv = view(v), ck = view(kc), cv = view(vc);
    KBIT_BY_TYPE(k.scalar_type(), append_kv_paged, run("append_kv_paged", k, {&kc, &vc}, [&](void* stream) {
        return fn(static_cast<const T*>(vk.p), vk.token, vk.head, static_cast<const T*>(vv.p), vv.token, vv.head,
                  k.size(0), h, dim, v_dim, slots.p, slots.bytes, KBIT_VIEW(T, ck), KBIT_VIEW(T, cv), kc.size(0), page,
                  t.positions.p, t.positions.bytes, t.table, t.rot, t.max_pos, t.layout, stream);
    }))
    return PyTuple_Pack(2, a[3], a[4]);
}

// ---------------------------------------------------------------------------
// module
// ---------------------------------------------------------------------------
PyMethodDef methods[] = {
    method<quantize_rows, 3>("quantize_rows_int8"),
    method<linear, 8>("linear_int8"),
    method<linear_dynamic, 6>("linear_int8_dynamic"),
    method<rope, 6>("rope"),
    method<norm_rope, 10>("qk_norm_rope"),
    method<norm_rope_backward, 13>("qk_norm_rope_backward"),
    method<append, 8>("append_kv_paged"),
    {nullptr, nullptr, 0, nullptr},
};

PyModuleDef module = {PyModuleDef_HEAD_INIT, "_layer", "Binding of include/kbit_layer.h and kbit_mx.h for torch tensors.", -1,
                      methods};

}  // namespace

extern PyMethodDef mx_methods[];  // mx_bind.cpp

PyMODINIT_FUNC PyInit__layer() {
    PyObject* m = PyModule_Create(&module);
    if (m != nullptr && PyModule_AddFunctions(m, mx_methods) != 0) {
        Py_DECREF(m);
        return nullptr;
    }
    return m;
}
