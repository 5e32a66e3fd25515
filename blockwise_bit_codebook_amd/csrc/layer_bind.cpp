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
#include <torch/csrc/Dtype.h>
#include <torch/csrc/autograd/python_variable.h>

#include <ATen/ATen.h>
#include <c10/core/GradMode.h>
#include <c10/hip/HIPFunctions.h>
#include <c10/hip/HIPStream.h>

#include <algorithm>
#include <initializer_list>
#include <sstream>
#include <string>
#include <utility>

#include "int8_choice.h"
#include "kbit.h"
#include "kbit_layer.h"

namespace {

using at::Tensor;

struct Raise {
    PyObject* type;
    std::string text;
};

[[noreturn]] void type_error(const std::string& text) { throw Raise{PyExc_TypeError, text}; }
[[noreturn]] void value_error(const std::string& text) { throw Raise{PyExc_ValueError, text}; }

template <class... A>
std::string cat(const A&... a) {
    std::ostringstream o;
    (void)std::initializer_list<int>{(o << a, 0)...};
    return o.str();
}

PyObject* kbit_error = nullptr;  // the package's exception, looked up once

[[noreturn]] void status_error(const char* name, int status) {
    if (kbit_error == nullptr) {
        PyObject* package = PyImport_ImportModule("blockwise_bit_codebook_amd");
        if (package != nullptr) {
            kbit_error = PyObject_GetAttrString(package, "KbitError");
            Py_DECREF(package);
        }
    }
    if (kbit_error != nullptr) {
        PyObject* e = PyObject_CallFunction(kbit_error, "sis", name, status, kbit_strerror(status));
        if (e != nullptr) {
            PyErr_SetObject(kbit_error, e);
            Py_DECREF(e);
        }
    }
    throw Raise{nullptr, ""};  // the Python error is set
}

// ---------------------------------------------------------------------------
// checks
// ---------------------------------------------------------------------------
const Tensor& tensor(PyObject* o, const char* what) {
    if (!THPVariable_Check(o)) type_error(cat(what, ": expected a tensor, got ", Py_TYPE(o)->tp_name));
    return THPVariable_Unpack(o);
}

bool is_float(at::ScalarType t) { return t == at::kFloat || t == at::kHalf || t == at::kBFloat16; }

void on_gpu(const Tensor& t, const char* what) {
    if (!t.is_cuda()) value_error(cat(what, " must live on the GPU"));
}

void same_device(const Tensor& t, const char* what, const Tensor& ref) {
    if (t.device() != ref.device()) value_error(cat(what, " is on ", t.device(), ", the input on ", ref.device()));
}

void same_shape(const Tensor& t, const char* what, at::IntArrayRef want) {
    if (t.sizes() != want) value_error(cat(what, ": shape ", t.sizes(), ", expected ", want));
}

// A 2-D tensor of contiguous rows that do not overlap: its row stride.
int64_t rows_of(const Tensor& t, const char* what, bool type_ok, const char* types) {
    if (!type_ok || t.dim() != 2)
        type_error(cat(what, " must be a 2-D tensor of ", types, ", got ", t.dim(), "-D ", t.scalar_type()));
    on_gpu(t, what);
    const int64_t n = t.size(0), d = t.size(1);
    if (d > 1 && t.stride(1) != 1) value_error(cat(what, ": the rows must be contiguous"));
    if (n <= 1) return d > 1 ? d : 1;  // a single row may carry any stride
    if (t.stride(0) < d) value_error(cat(what, ": the rows overlap"));
    return t.stride(0);
}

constexpr const char* kFloats = "float32, float16 or bfloat16";

// A contiguous tensor of at least count elements of a type.
void* vector(PyObject* o, const char* what, at::ScalarType type, int64_t count, const Tensor& ref) {
    const Tensor& t = tensor(o, what);
    if (t.scalar_type() != type) type_error(cat(what, ": element type ", t.scalar_type(), ", expected ", type));
    if (t.numel() < count) value_error(cat(what, ": ", t.numel(), " elements, at least ", count, " needed"));
    if (!t.is_contiguous()) value_error(cat(what, ": tensor must be contiguous"));
    same_device(t, what, ref);
    return t.data_ptr();
}

// One value for each of the channels, no more: a longer vector belongs to
// another layer.
void* channel_vector(PyObject* o, const char* what, at::ScalarType type, int64_t channels, const Tensor& ref) {
    void* p = vector(o, what, type, channels, ref);
    const int64_t n = THPVariable_Unpack(o).numel();
    if (n != channels) value_error(cat(what, ": ", n, " elements for ", channels, " channels"));
    return p;
}

int fits_int(int64_t n, const char* what) {
    if (n < 0 || n > INT32_MAX) value_error(cat(what, " is out of range"));
    return static_cast<int>(n);
}

// ---------------------------------------------------------------------------
// outputs that overlap
// ---------------------------------------------------------------------------
// Rows of `length` neighbouring elements, counted by up to three axes (strides
// are not negative).
struct Rows {
    int64_t size[3], stride[3], length, last;  // last: the last row's first element
};

Rows rows_in(const Tensor& t) {
    Rows r{{1, 1, 1}, {0, 0, 0}, t.size(-1), 0};
    for (int64_t i = 0; i + 1 < t.dim(); ++i) {
        r.size[i] = t.size(i);
        r.stride[i] = t.size(i) > 1 ? t.stride(i) : 0;
        r.last += (r.size[i] - 1) * r.stride[i];
    }
    return r;
}

// Steps lo .. hi of one stride; `reach`: how far the axes after it go down and up.
struct Axis {
    int64_t stride, lo, hi, down, up;
};

// Whether steps along the axes (largest stride first) take v to a value in
// (low, high).  `moved`: some step was not zero, which is asked for.  Each axis
// leaves one or two candidates where the strides are nested, as those of views
// are; `budget` ends the search in any other layout, which then counts as apart.
bool reaches(int64_t v, const Axis* a, int n, int64_t low, int64_t high, bool moved, int& budget) {
    if (n == 0) return moved && v > low && v < high;
    if (--budget < 0) return false;
    const int64_t from = low - a->up - v, to = high - a->down - v;  // of stride * step, both ends open
    int64_t lo = a->lo, hi = a->hi;
    if (a->stride == 0) {
        if (from >= 0 || to <= 0) return false;
    } else {
        const auto below = [](int64_t x, int64_t s) { return x >= 0 ? x / s : -((-x + s - 1) / s); };  // floor(x / s)
        lo = std::max(lo, below(from, a->stride) + 1);
        hi = std::min(hi, -below(-to, a->stride) - 1);
    }
    for (int64_t d = lo; d <= hi && budget >= 0; ++d)
        if (reaches(v + d * a->stride, a + 1, n - 1, low, high, moved || d != 0, budget)) return true;
    return false;
}

// Whether a row of x and a row of y, whose first elements are `apart` elements
// apart, have an element in common; with `self` two different rows of x.
bool rows_meet(const Rows& x, const Rows& y, int64_t apart, bool self) {
    if (apart + y.last + y.length <= 0 || apart >= x.last + x.length) return false;
    Axis axes[6];
    int n = 0;
    for (int i = 0; i < 3; ++i) {
        const int64_t sx = x.size[i] > 1 ? x.stride[i] : y.stride[i], sy = y.size[i] > 1 ? y.stride[i] : sx;
        if (sx == sy) {
            if (x.size[i] > 1 || y.size[i] > 1) axes[n++] = Axis{sx, 1 - x.size[i], y.size[i] - 1, 0, 0};
        } else {
            axes[n++] = Axis{sx, 1 - x.size[i], 0, 0, 0};
            axes[n++] = Axis{sy, 0, y.size[i] - 1, 0, 0};
        }
    }
    std::sort(axes, axes + n, [](const Axis& a, const Axis& b) { return a.stride > b.stride; });
    for (int i = n - 1; i > 0; --i) {
        axes[i - 1].down = axes[i].down + axes[i].lo * axes[i].stride;
        axes[i - 1].up = axes[i].up + axes[i].hi * axes[i].stride;
    }
    int budget = 4096;
    return reaches(apart, axes, n, -y.length, x.length, !self, budget);
}

// Refuses an output two rows of which share elements.
void no_overlap(const Tensor& out, const char* what) {
    if (out.numel() == 0 || out.is_non_overlapping_and_dense()) return;
    const Rows r = rows_in(out);
    if (rows_meet(r, r, 0, true)) value_error(cat(what, ": elements overlap"));
}

// Refuses an output that shares elements with another tensor of its type, but
// for `same`: the very same view, each row of which is read before it is written.
void no_overlap(const Tensor& out, const char* what, const Tensor& other, const char* name, bool same) {
    if (!out.is_alias_of(other) || out.numel() == 0 || other.numel() == 0) return;
    const int64_t bytes = static_cast<char*>(other.data_ptr()) - static_cast<char*>(out.data_ptr());
    if (same && bytes == 0 && out.sizes() == other.sizes() && out.strides() == other.strides()) return;
    const int64_t size = static_cast<int64_t>(out.element_size());
    if (bytes % size != 0 || rows_meet(rows_in(out), rows_in(other), bytes / size, false))
        value_error(cat(what, " overlaps ", name));
}

// ---------------------------------------------------------------------------
// calls
// ---------------------------------------------------------------------------
// The device's current stream, with the device made current for the call.
struct On {
    int before = -1;
    void* stream;
    explicit On(const Tensor& ref) {
        const auto index = ref.device().index();
        const int now = c10::hip::current_device();
        if (now != index) {
            c10::hip::set_device(index);
            before = now;
        }
        stream = c10::hip::getCurrentHIPStream(index).stream();
    }
    ~On() {
        if (before >= 0) (void)c10::hip::SetDevice(static_cast<c10::DeviceIndex>(before));
    }
};

// A tensor that a call wrote through its address: autograd then refuses a
// backward pass that saved the old values, as for any in-place operation.
// (Inference tensors have no version.)
void written(const Tensor& t) {
    if (!t.is_inference()) t.unsafeGetTensorImpl()->bump_version();
}

// f(stream) without the interpreter's lock; `outputs` are what it writes.
template <class F>
void run(const char* name, const Tensor& ref, std::initializer_list<const Tensor*> outputs, F f) {
    int status;
    {
        On on(ref);
        PyThreadState* save = PyEval_SaveThread();
        status = f(on.stream);
        PyEval_RestoreThread(save);
    }
    if (status != 0) status_error(name, status);
    for (const Tensor* t : outputs) written(*t);
}

// The entry point of a type (data arguments are passed as that type).
#define KBIT_BY_TYPE(TYPE, NAME, F)                                                            \
    switch (TYPE) {                                                                            \
        case at::kFloat: {                                                                     \
            using T [[maybe_unused]] = float;                                                  \
            constexpr auto fn = NAME##_fp32;                                                   \
            F;                                                                                 \
            break;                                                                             \
        }                                                                                      \
        case at::kHalf: {                                                                      \
            using T [[maybe_unused]] = uint16_t;                                               \
            constexpr auto fn = NAME##_fp16;                                                   \
            F;                                                                                 \
            break;                                                                             \
        }                                                                                      \
        default: {                                                                             \
            using T [[maybe_unused]] = uint16_t;                                               \
            constexpr auto fn = NAME##_bf16;                                                   \
            F;                                                                                 \
            break;                                                                             \
        }                                                                                      \
    }

struct Space {
    Tensor keep;  // lives until the call is enqueued; the allocator orders reuse by stream
    void* p = nullptr;
    int64_t bytes = 0;
};

// `need`: what a given workspace has to hold; `take`: what is allocated else,
// which may be less (this call's own need).
Space workspace(int64_t need, int64_t take, PyObject* given, const char* name, const Tensor& ref) {
    if (need < 0) status_error(name, KBIT_EINVAL);
    Space s;
    if (given != Py_None) {
        s.p = vector(given, "workspace", at::kByte, need, ref);
        s.bytes = THPVariable_Unpack(given).numel();
    } else if (take > 0) {
        s.keep = at::empty({take}, ref.options().dtype(at::kByte));
        s.p = s.keep.data_ptr();
        s.bytes = take;
    }
    return s;
}

PyObject* wrap(const Tensor& t) { return THPVariable_Wrap(t); }

PyObject* wrap(std::initializer_list<Tensor> ts) {
    PyObject* tuple = PyTuple_New(static_cast<Py_ssize_t>(ts.size()));
    if (tuple == nullptr) throw Raise{nullptr, ""};
    Py_ssize_t i = 0;
    for (const Tensor& t : ts) {
        PyObject* o = wrap(t);
        if (o == nullptr) {
            Py_DECREF(tuple);
            throw Raise{nullptr, ""};
        }
        PyTuple_SET_ITEM(tuple, i++, o);
    }
    return tuple;
}

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

float number(PyObject* o, const char* what) {
    const double v = PyFloat_AsDouble(o);
    if (v == -1.0 && PyErr_Occurred()) {
        PyErr_Clear();
        type_error(cat(what, " must be a number"));
    }
    return static_cast<float>(v);
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
// Whether autograd expects a gradient through one of the arguments.
bool gradient_wanted(PyObject* const* args, int n) {
    if (!c10::GradMode::is_enabled()) return false;
    auto* tensors = reinterpret_cast<PyTypeObject*>(THPVariableClass);
    for (int i = 0; i < n; ++i)
        if (PyType_IsSubtype(Py_TYPE(args[i]), tensors) && THPVariable_Unpack(args[i]).requires_grad()) return true;
    return false;
}

template <PyObject* (*F)(PyObject* const*), int kArgs>
PyObject* entry(PyObject*, PyObject* const* args, Py_ssize_t n) {
    if (n != kArgs) {
        PyErr_Format(PyExc_TypeError, "expected %d arguments, got %zd", kArgs, n);
        return nullptr;
    }
    try {
        // 2: the line that called the function of layer.py
        if (gradient_wanted(args, kArgs) &&
            PyErr_WarnEx(PyExc_UserWarning,
                         "an argument requires a gradient, but nothing is recorded for autograd: the outputs are cut off "
                         "from it (call this under torch.no_grad(), or in a torch.autograd.Function with the gradient's "
                         "own call)",
                         2) != 0)
            return nullptr;
        return F(args);
    } catch (const Raise& r) {
        if (r.type != nullptr) PyErr_SetString(r.type, r.text.c_str());
        else if (!PyErr_Occurred()) PyErr_SetString(PyExc_RuntimeError, "call failed");
    } catch (const std::exception& e) {
        if (!PyErr_Occurred()) PyErr_SetString(PyExc_RuntimeError, e.what());
    } catch (...) {
        if (!PyErr_Occurred()) PyErr_SetString(PyExc_RuntimeError, "call failed");
    }
    return nullptr;
}

template <PyObject* (*F)(PyObject* const*), int kArgs>
PyMethodDef method(const char* name) {
    return {name, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(&entry<F, kArgs>)), METH_FASTCALL, nullptr};
}

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

PyModuleDef module = {PyModuleDef_HEAD_INIT, "_layer", "Binding of include/kbit_layer.h for torch tensors.", -1, methods};

}  // namespace

PyMODINIT_FUNC PyInit__layer() { return PyModule_Create(&module); }
