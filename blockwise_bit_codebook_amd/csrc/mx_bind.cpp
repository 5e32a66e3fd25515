// The Python binding of include/kbit_mx.h for torch tensors, a part of the
// module _layer: checks, output allocation and the C calls; mx.py holds the
// functions' documented signatures.
#include "bind.h"
#include "kbit_mx.h"
#include "mx_internal.h"

namespace {

constexpr at::ScalarType kByte = at::kByte;

// A tensor's rows in bytes; a contiguous one, of any shape, is one row.
Rows byte_rows(const Tensor& t) {
    const int64_t size = static_cast<int64_t>(t.element_size());
    if (t.is_contiguous()) return Rows{{1, 1, 1}, {0, 0, 0}, t.numel() * size, 0};
    Rows r = rows_in(t);
    for (int64_t& s : r.stride) s *= size;
    r.length *= size;
    r.last *= size;
    return r;
}

// Refuses an output that shares bytes with a tensor of another type; rows that
// lie between each other's are apart.
void apart(const Tensor& out, const char* what, const Tensor& other, const char* name) {
    if (!out.is_alias_of(other) || out.numel() == 0 || other.numel() == 0) return;
    const int64_t bytes = static_cast<char*>(other.data_ptr()) - static_cast<char*>(out.data_ptr());
    if (rows_meet(byte_rows(out), byte_rows(other), bytes, false, true)) value_error(cat(what, " overlaps ", name));
}

// Refuses a given workspace whose first `used` bytes, which are all that the call
// writes of it, are shared with one of the call's tensors.
struct Named {
    const Tensor& t;
    const char* name;
};
void clear_of(const Space& ws, PyObject* given, int64_t used, std::initializer_list<Named> tensors) {
    if (given == Py_None || used <= 0) return;
    const Rows space{{1, 1, 1}, {0, 0, 0}, used, 0};
    for (const auto& [t, name] : tensors) {
        if (!t.defined() || t.numel() == 0 || !t.is_alias_of(THPVariable_Unpack(given))) continue;
        const int64_t bytes = static_cast<char*>(t.data_ptr()) - static_cast<char*>(ws.p);
        if (rows_meet(space, byte_rows(t), bytes, false, true)) value_error(cat("the workspace overlaps ", name));
    }
}
Tensor or_none(PyObject* o) { return o == Py_None ? Tensor() : THPVariable_Unpack(o); }

// Codes and scales of rows of d values.
struct Coded {
    uint8_t *codes, *scales;
    int64_t rows, ldc, lds;
};

Coded coded(const Tensor& c, const char* codes, const Tensor& s, const char* scales, int64_t d, const Tensor& ref) {
    Coded r;
    r.ldc = rows_of(c, codes, c.scalar_type() == kByte, "uint8");
    r.lds = rows_of(s, scales, s.scalar_type() == kByte, "uint8");
    const int64_t blocks = kbit::mx_blocks(d);
    if (c.size(1) != blocks * kbit::kMxBlockBytes)
        value_error(cat(codes, ": rows of ", c.size(1), " bytes, ", d, " values take ", blocks * kbit::kMxBlockBytes));
    r.rows = c.size(0);
    same_shape(s, scales, {r.rows, blocks});
    same_device(c, codes, ref);
    same_device(s, scales, ref);
    r.codes = static_cast<uint8_t*>(c.data_ptr());
    r.scales = static_cast<uint8_t*>(s.data_ptr());
    return r;
}

int depth(int64_t n, const char* what) {
    if (n < 1 || n > kbit::kMxMaxDepth) value_error(cat(what, " must be between 1 and ", kbit::kMxMaxDepth, ", got ", n));
    return static_cast<int>(n);
}

PyObject* quantize(PyObject* const* a) {  // X, codes, scales
    const Tensor& X = tensor(a[0], "X");
    if (!is_float(X.scalar_type()) || X.dim() != 2)
        type_error(cat("X must be a 2-D tensor of ", kFloats, ", got ", X.dim(), "-D ", X.scalar_type()));
    on_gpu(X, "X");
    // rows as they stand, else the columns of the transposed matrix
    const int64_t rows = X.size(0), d = X.size(1);
    const bool by_rows = d <= 1 || X.stride(1) == 1;
    if (!by_rows && rows > 1 && X.stride(0) != 1) value_error("X: the rows or the columns must be contiguous");
    int64_t ldx;
    if (by_rows) {
        ldx = rows > 1 ? X.stride(0) : d;
        if (ldx < d) value_error("X: the rows overlap");
    } else {
        ldx = X.stride(1);
        if (ldx < rows) value_error("X: the columns overlap");
    }
    const int di = depth(d, "the number of columns");
    fits_int(rows, "the number of rows");
    const int64_t blocks = kbit::mx_blocks(d);
    const Tensor codes = a[1] == Py_None ? at::empty({rows, blocks * kbit::kMxBlockBytes}, X.options().dtype(kByte))
                                         : tensor(a[1], "codes");
    const Tensor scales = a[2] == Py_None ? at::empty({rows, blocks}, X.options().dtype(kByte)) : tensor(a[2], "scales");
    const Coded c = coded(codes, "codes", scales, "scales", d, X);
    if (c.rows != rows) value_error(cat("codes: ", c.rows, " rows, X has ", rows));
    if (codes.is_alias_of(X) || scales.is_alias_of(X)) {
        const Tensor lines = by_rows ? X : X.t();  // what is contiguous of X as rows
        apart(codes, "codes", lines, "X");
        apart(scales, "scales", lines, "X");
    }
    no_overlap(codes, "codes", scales, "scales", false);
    if (by_rows) {
        KBIT_BY_TYPE(X.scalar_type(), quantize_mxfp4, run("quantize_mxfp4", X, {&codes, &scales}, [&](void* stream) {
            return fn(static_cast<const T*>(X.data_ptr()), rows, di, ldx, c.codes, c.ldc, c.scales, c.lds, stream);
        }))
    } else {
        KBIT_BY_TYPE(X.scalar_type(), quantize_mxfp4_columns, run("quantize_mxfp4", X, {&codes, &scales}, [&](void* stream) {
            return fn(static_cast<const T*>(X.data_ptr()), di, static_cast<int>(rows), ldx, c.codes, c.ldc, c.scales, c.lds,
                      stream);
        }))
    }
    return wrap({codes, scales});
}

at::ScalarType dtype_of(PyObject* o) {
    if (!THPDtype_Check(o)) type_error("dtype must be a torch.dtype");
    const at::ScalarType type = reinterpret_cast<THPDtype*>(o)->scalar_type;
    if (!is_float(type)) type_error(cat("unsupported element dtype ", type));
    return type;
}

int64_t whole_number(PyObject* o, const char* what) {
    const int64_t v = PyLong_AsLongLong(o);
    if (v == -1 && PyErr_Occurred()) {
        PyErr_Clear();
        type_error(cat(what, " must be an integer"));
    }
    return v;
}

// A given output of a shape, or a new one; its rows' distance.
struct Out {
    Tensor t;
    int64_t ld;
};

Out output(PyObject* given, const char* what, at::IntArrayRef shape, at::ScalarType type, const Tensor& ref) {
    Out o;
    if (given == Py_None) {
        o.t = at::empty(shape, ref.options().dtype(type));
        o.ld = shape[1];
    } else {
        o.t = tensor(given, what);
        o.ld = rows_of(o.t, what, o.t.scalar_type() == type, at::toString(type));
        same_shape(o.t, what, shape);
        same_device(o.t, what, ref);
    }
    return o;
}

PyObject* dequantize(PyObject* const* a) {  // codes, scales, d, dtype, out
    const Tensor& codes = tensor(a[0], "codes");
    const Tensor& scales = tensor(a[1], "scales");
    const int d = depth(whole_number(a[2], "d"), "d");
    const at::ScalarType type = dtype_of(a[3]);
    const Coded c = coded(codes, "codes", scales, "scales", d, codes);
    const Out out = output(a[4], "out", {c.rows, d}, type, codes);
    apart(out.t, "out", codes, "codes");
    apart(out.t, "out", scales, "scales");
    KBIT_BY_TYPE(type, dequantize_mxfp4, run("dequantize_mxfp4", codes, {&out.t}, [&](void* stream) {
        return fn(c.codes, c.ldc, c.scales, c.lds, c.rows, d, static_cast<T*>(out.t.data_ptr()), out.ld, stream);
    }))
    return wrap(out.t);
}

// The weight's side of a product, and its output.
struct Weight {
    Coded c;
    const void* bias;
    int N;
    Out out;
};

Weight weight(const Tensor& x, int64_t M, int64_t K, PyObject* codes, PyObject* scales, PyObject* bias, PyObject* out,
              at::ScalarType type) {
    Weight w;
    const Tensor& c = tensor(codes, "w_codes");
    const Tensor& s = tensor(scales, "w_scales");
    w.c = coded(c, "w_codes", s, "w_scales", K, x);
    if (w.c.rows < 1) value_error("the weight must have at least one row");
    w.N = fits_int(w.c.rows, "the number of output channels");
    w.bias = bias == Py_None ? nullptr : channel_vector(bias, "bias", type, w.N, x);
    w.out = output(out, "out", {M, w.N}, type, x);
    apart(w.out.t, "out", c, "w_codes");
    apart(w.out.t, "out", s, "w_scales");
    if (bias != Py_None) apart(w.out.t, "out", THPVariable_Unpack(bias), "bias");
    return w;
}

PyObject* linear(PyObject* const* a) {  // codes, scales, w_codes, w_scales, bias, dtype, out, workspace
    const Tensor& x = tensor(a[0], "codes");
    const Tensor& xs = tensor(a[1], "scales");
    const at::ScalarType type = dtype_of(a[5]);
    if (x.scalar_type() != kByte || x.dim() != 2)
        type_error(cat("codes must be a 2-D tensor of uint8, got ", x.dim(), "-D ", x.scalar_type()));
    on_gpu(x, "codes");
    if (x.size(1) < kbit::kMxBlockBytes || x.size(1) % kbit::kMxBlockBytes != 0)
        value_error(cat("codes: rows of ", x.size(1), " bytes, expected whole blocks of ", kbit::kMxBlockBytes));
    const int K = depth(x.size(1) * 2, "the depth");  // whole blocks: the last one's zeros add nothing
    const Coded c = coded(x, "codes", xs, "scales", K, x);
    const Weight w = weight(x, c.rows, K, a[2], a[3], a[4], a[6], type);
    apart(w.out.t, "out", x, "codes");
    apart(w.out.t, "out", xs, "scales");
    const int64_t need = linear_mxfp4_workspace_bytes(c.rows, w.N, K);
    const int64_t take = need > 0 ? kbit::mx_product_workspace(c.rows, w.N, kbit::mx_depth(K)) : 0;
    const Space ws = workspace(need, take, a[7], "linear_mxfp4", x);
    clear_of(ws, a[7], take, {{x, "codes"}, {xs, "scales"}, {THPVariable_Unpack(a[2]), "w_codes"},
                              {THPVariable_Unpack(a[3]), "w_scales"}, {or_none(a[4]), "bias"}, {w.out.t, "out"}});
    KBIT_BY_TYPE(type, linear_mxfp4, run("linear_mxfp4", x, {&w.out.t}, [&](void* stream) {
        return fn(c.codes, c.scales, c.rows, K, c.ldc, c.lds, w.c.codes, w.c.scales, w.N, w.c.ldc, w.c.lds,
                  static_cast<const T*>(w.bias), static_cast<T*>(w.out.t.data_ptr()), w.out.ld, ws.p, ws.bytes, stream);
    }))
    return wrap(w.out.t);
}

PyObject* linear_dynamic(PyObject* const* a) {  // X, w_codes, w_scales, bias, out, workspace
    const Tensor& x = tensor(a[0], "X");
    const at::ScalarType type = x.scalar_type();
    const int64_t ldx = rows_of(x, "X", is_float(type), kFloats), M = x.size(0);
    const int K = depth(x.size(1), "the depth");
    const Weight w = weight(x, M, K, a[1], a[2], a[3], a[4], type);
    no_overlap(w.out.t, "out", x, "X", false);
    if (M == 0) return wrap(w.out.t);
    const bool fused = linear_mxfp4_dynamic_fused(M, w.N, K, w.c.ldc, w.c.lds);
    const int64_t need = fused ? 0 : linear_mxfp4_dynamic_workspace_bytes(M, w.N, K);
    const int64_t take = need <= 0 ? 0
                                   : (kbit::mx_rows(M, K).bytes + 15) / 16 * 16 +
                                         kbit::mx_product_workspace(M, w.N, kbit::mx_depth(K),
                                                                    kbit::mx_paired(M, w.N, kbit::mx_depth(K)));
    const Space ws = workspace(need, take, a[5], "linear_mxfp4_dynamic", x);
    clear_of(ws, a[5], take, {{x, "X"}, {THPVariable_Unpack(a[1]), "w_codes"}, {THPVariable_Unpack(a[2]), "w_scales"},
                              {or_none(a[3]), "bias"}, {w.out.t, "out"}});
    KBIT_BY_TYPE(type, linear_mxfp4_dynamic, run("linear_mxfp4_dynamic", x, {&w.out.t}, [&](void* stream) {
        return fn(static_cast<const T*>(x.data_ptr()), M, K, ldx, w.c.codes, w.c.scales, w.N, w.c.ldc, w.c.lds,
                  static_cast<const T*>(w.bias), static_cast<T*>(w.out.t.data_ptr()), w.out.ld, ws.p, ws.bytes, stream);
    }))
    return wrap(w.out.t);
}

bool flag(PyObject* o) {
    const int v = PyObject_IsTrue(o);
    if (v < 0) throw Raise{nullptr, ""};
    return v != 0;
}

// dout, X, weight, input_grad, weight_grad, bias_grad, dX, dweight, workspace
PyObject* linear_backward(PyObject* const* a) {
    const Tensor& g = tensor(a[0], "dout");
    const at::ScalarType type = g.scalar_type();
    const int64_t ldg = rows_of(g, "dout", is_float(type), kFloats), M = g.size(0);
    const int N = depth(g.size(1), "the number of output channels");
    const Tensor& x = tensor(a[1], "X");
    const Tensor& w = tensor(a[2], "weight");
    const int64_t ldx = rows_of(x, "X", x.scalar_type() == type, at::toString(type));
    const int64_t ldw = rows_of(w, "weight", w.scalar_type() == type, at::toString(type));
    const int K = depth(x.size(1), "the depth");
    same_shape(x, "X", {M, K});
    same_shape(w, "weight", {N, K});
    same_device(x, "X", g);
    same_device(w, "weight", g);
    const bool input = flag(a[3]), weights = flag(a[4]), bias = flag(a[5]);
    if ((!input && a[6] != Py_None) || (!weights && a[7] != Py_None))
        value_error("an output is given for a gradient that is not asked for");
    Out dx, dw;
    Tensor db;
    if (input) {
        dx = output(a[6], "dX", {M, K}, type, g);
        no_overlap(dx.t, "dX", g, "dout", false);
        no_overlap(dx.t, "dX", x, "X", false);
        no_overlap(dx.t, "dX", w, "weight", false);
    }
    if (weights) {
        dw = output(a[7], "dweight", {N, K}, at::kFloat, g);
        for (const auto& [t, name] : {std::pair<const Tensor&, const char*>{g, "dout"}, {x, "X"}, {w, "weight"}})
            apart(dw.t, "dweight", t, name);
        if (input) apart(dw.t, "dweight", dx.t, "dX");
    }
    if (bias) db = at::empty({N}, g.options().dtype(at::kFloat));
    Space ws;
    if (M > 0) {
        const int64_t need = linear_mxfp4_backward_workspace_bytes(M, N, K);
        const int64_t take = need < 0 ? need : kbit::mx_back_workspace(M, N, K, input, weights, bias);
        ws = workspace(need, take, a[8], "linear_mxfp4_backward", g);
        clear_of(ws, a[8], take, {{g, "dout"}, {x, "X"}, {w, "weight"}, {dx.t, "dX"}, {dw.t, "dweight"}});
    }
    const auto ptr = [](const Tensor& t) { return t.defined() ? t.data_ptr() : nullptr; };
    KBIT_BY_TYPE(type, linear_mxfp4_backward, run("linear_mxfp4_backward", g, {}, [&](void* stream) {
        return fn(static_cast<const T*>(g.data_ptr()), ldg, static_cast<const T*>(x.data_ptr()), ldx,
                  static_cast<const T*>(w.data_ptr()), ldw, M, N, K, static_cast<T*>(ptr(dx.t)), dx.ld,
                  static_cast<float*>(ptr(dw.t)), dw.ld, static_cast<float*>(ptr(db)), ws.p, ws.bytes, stream);
    }))
    if (input) written(dx.t);
    if (weights) written(dw.t);
    PyObject* tuple = PyTuple_New(3);
    if (tuple == nullptr) throw Raise{nullptr, ""};
    const Tensor* outs[3] = {input ? &dx.t : nullptr, weights ? &dw.t : nullptr, bias ? &db : nullptr};
    for (int i = 0; i < 3; ++i) {
        PyObject* o = outs[i] ? wrap(*outs[i]) : (Py_INCREF(Py_None), Py_None);
        if (o == nullptr) {
            Py_DECREF(tuple);
            throw Raise{nullptr, ""};
        }
        PyTuple_SET_ITEM(tuple, i, o);
    }
    return tuple;
}

// ---------------------------------------------------------------------------
// layer norm
// ---------------------------------------------------------------------------
struct NormWeights {
    const void *weight, *bias;
    int fp32;
};

NormWeights norm_weights(PyObject* w, PyObject* b, const Tensor& x) {
    const at::ScalarType wt = THPVariable_Check(w) ? THPVariable_Unpack(w).scalar_type() : at::kByte;
    if (wt != x.scalar_type() && wt != at::kFloat) type_error(cat("weight must be a ", x.scalar_type(), " or float32 tensor"));
    const int64_t d = x.size(1);
    NormWeights n;
    n.weight = vector(w, "weight", wt, d, x);
    n.bias = b == nullptr || b == Py_None ? nullptr : vector(b, "bias", wt, d, x);
    if (THPVariable_Unpack(w).numel() != d || (n.bias && THPVariable_Unpack(b).numel() != d))
        value_error(cat("weight and bias must have ", d, " elements"));
    n.fp32 = wt == at::kFloat;
    return n;
}

PyObject* layer_norm(PyObject* const* a) {  // x, weight, bias, eps, out
    const Tensor& x = tensor(a[0], "x");
    const at::ScalarType type = x.scalar_type();
    const int64_t ldx = rows_of(x, "x", is_float(type), kFloats), rows = x.size(0);
    if (x.size(1) < 1) value_error("x must have at least one column");
    const int d = fits_int(x.size(1), "the number of columns");
    const NormWeights n = norm_weights(a[1], a[2], x);
    const float eps = number(a[3], "eps");
    const Out out = output(a[4], "out", {rows, d}, type, x);
    no_overlap(out.t, "out", x, "x", true);
    apart(out.t, "out", THPVariable_Unpack(a[1]), "weight");
    if (n.bias) apart(out.t, "out", THPVariable_Unpack(a[2]), "bias");
    KBIT_BY_TYPE(type, layer_norm, run("layer_norm", x, {&out.t}, [&](void* stream) {
        return fn(static_cast<const T*>(x.data_ptr()), rows, d, ldx, n.weight, n.bias, n.fp32, eps,
                  static_cast<T*>(out.t.data_ptr()), out.ld, stream);
    }))
    return wrap(out.t);
}

PyObject* layer_norm_backward(PyObject* const* a) {  // dout, x, weight, eps, dx, workspace
    const Tensor& x = tensor(a[1], "x");
    const at::ScalarType type = x.scalar_type();
    const int64_t ldx = rows_of(x, "x", is_float(type), kFloats), rows = x.size(0);
    if (x.size(1) < 1) value_error("x must have at least one column");
    const int d = fits_int(x.size(1), "the number of columns");
    const Tensor& g = tensor(a[0], "dout");
    const int64_t ldg = rows_of(g, "dout", g.scalar_type() == type, at::toString(type));
    same_shape(g, "dout", x.sizes());
    same_device(g, "dout", x);
    const NormWeights n = norm_weights(a[2], nullptr, x);
    const float eps = number(a[3], "eps");
    const Out dx = output(a[4], "dx", {rows, d}, type, x);
    no_overlap(dx.t, "dx", g, "dout", true);
    no_overlap(dx.t, "dx", x, "x", false);
    apart(dx.t, "dx", THPVariable_Unpack(a[2]), "weight");
    const Tensor dw = at::empty({d}, x.options().dtype(at::kFloat)), db = at::empty_like(dw);
    const int64_t need = layer_norm_backward_workspace_bytes(rows, d);
    const Space ws = workspace(need, need, a[5], "layer_norm_backward", x);
    clear_of(ws, a[5], need, {{g, "dout"}, {x, "x"}, {THPVariable_Unpack(a[2]), "weight"}, {dx.t, "dx"}});
    KBIT_BY_TYPE(type, layer_norm_backward, run("layer_norm_backward", x, {&dx.t}, [&](void* stream) {
        return fn(static_cast<const T*>(g.data_ptr()), ldg, static_cast<const T*>(x.data_ptr()), ldx, rows, d, n.weight,
                  n.fp32, eps, static_cast<T*>(dx.t.data_ptr()), dx.ld, static_cast<float*>(dw.data_ptr()),
                  static_cast<float*>(db.data_ptr()), ws.p, ws.bytes, stream);
    }))
    return wrap({dx.t, dw, db});
}

}  // namespace

PyMethodDef mx_methods[] = {
    method<quantize, 3>("quantize_mxfp4"),
    method<dequantize, 5>("dequantize_mxfp4"),
    method<linear, 8>("linear_mxfp4"),
    method<linear_dynamic, 6>("linear_mxfp4_dynamic"),
    method<linear_backward, 9>("linear_mxfp4_backward"),
    method<layer_norm, 5>("layer_norm"),
    method<layer_norm_backward, 6>("layer_norm_backward"),
    {nullptr, nullptr, 0, nullptr},
};
