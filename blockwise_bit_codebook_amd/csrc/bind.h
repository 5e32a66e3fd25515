// What the Python bindings of the operators on torch tensors share: checks,
// overlaps, workspaces, the call on torch's current stream of the inputs'
// device, and the entry that turns errors into Python's.
#pragma once

#include <torch/csrc/Dtype.h>
#include <torch/csrc/autograd/python_variable.h>

#include <ATen/ATen.h>
#include <c10/core/GradMode.h>
#include <c10/hip/HIPFunctions.h>
#include <c10/hip/HIPStream.h>

#include <algorithm>
#include <initializer_list>
#include <numeric>
#include <sstream>
#include <string>
#include <utility>

#include "kbit.h"

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
// apart, have an element in common; with `self` two different rows of x.  `unsure`:
// what a layout gives that the search does not get through.
bool rows_meet(const Rows& x, const Rows& y, int64_t apart, bool self, bool unsure = false) {
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
    // every step moves by a multiple of what the strides share
    int64_t g = 0;
    for (int i = 0; i < n; ++i) g = std::gcd(g, axes[i].stride);
    if (g > 0) {
        const int64_t first = ((apart + y.length - 1) % g + g) % g;  // how far the least such distance is above -y.length + 1
        if (first >= x.length + y.length - 1) return false;
    }
    std::sort(axes, axes + n, [](const Axis& a, const Axis& b) { return a.stride > b.stride; });
    for (int i = n - 1; i > 0; --i) {
        axes[i - 1].down = axes[i].down + axes[i].lo * axes[i].stride;
        axes[i - 1].up = axes[i].up + axes[i].hi * axes[i].stride;
    }
    int budget = 4096;
    return reaches(apart, axes, n, -y.length, x.length, !self, budget) || (unsure && budget < 0);
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

float number(PyObject* o, const char* what) {
    const double v = PyFloat_AsDouble(o);
    if (v == -1.0 && PyErr_Occurred()) {
        PyErr_Clear();
        type_error(cat(what, " must be a number"));
    }
    return static_cast<float>(v);
}

// ---------------------------------------------------------------------------
// entry
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

}  // namespace
