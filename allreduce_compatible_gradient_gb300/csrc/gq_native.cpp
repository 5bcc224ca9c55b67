// gq_native.cpp -- Python entry points of the activation operators (include/gq.h) on torch tensors.
//
// Argument checks, allocation of outputs and the call of libgq.so, in C++: a call on a small matrix
// takes 3 to 5 us on the GPU, and the same marshalling in Python took 11 to 22 us on the host.  The
// functions of libgq.so come in by address (bind), so that the extension works with whichever build
// of the library the package has loaded.  Nothing here touches data.
#include <Python.h>

#include <ATen/ATen.h>
#include <ATen/cuda/EmptyTensor.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include <cstdint>
#include <memory>

#include "gq.h"

namespace {

// The library's functions, in the order of kNames.
struct Api {
    decltype(&gq_act_quantize) act_quantize;
    decltype(&gq_act_dequantize) act_dequantize;
    decltype(&gq_layernorm_forward) layernorm_forward;
    decltype(&gq_layernorm_workspace_bytes) layernorm_workspace_bytes;
    decltype(&gq_layernorm_backward) layernorm_backward;
    decltype(&gq_gelu_forward) gelu_forward;
    decltype(&gq_gelu_backward) gelu_backward;
    decltype(&gq_linear_wgrad_workspace_bytes) linear_wgrad_workspace_bytes;
    decltype(&gq_linear_wgrad_plan) linear_wgrad_plan;
    decltype(&gq_linear_wgrad) linear_wgrad;
};
constexpr int kFunctions = sizeof(Api) / sizeof(void*);
Api api;
PyObject* gq_error = nullptr;  // the package's GQError

struct Refused {};  // a Python error is set

template <typename... A> [[noreturn]] void refuse(PyObject* type, const char* format, A... a) {
    PyErr_Format(type, format, a...);
    throw Refused{};
}

void check(int status, const char* where) {
    if (status == GQ_OK) return;
    PyObject* e = PyObject_CallFunction(gq_error, "is", status, where);
    if (e) {
        PyErr_SetObject(gq_error, e);
        Py_DECREF(e);
    }
    throw Refused{};
}

int type_code(at::ScalarType t) {
    return t == at::kFloat ? GQ_F32 : t == at::kBFloat16 ? GQ_BF16 : t == at::kHalf ? GQ_F16 : -1;
}

const at::Tensor& tensor(PyObject* o, const char* what) {
    if (!THPVariable_Check(o)) refuse(PyExc_TypeError, "%s must be a tensor", what);
    return THPVariable_Unpack(o);
}

// A tensor as a matrix: its leading dimensions seen as one, rows ld elements apart.
struct Matrix {
    int code, index;
    int64_t rows, cols, ld;
    void* p;
};

Matrix matrix(const at::Tensor& t, const char* what, bool half = false) {
    Matrix m;
    m.code = type_code(t.scalar_type());
    if (m.code < 0 || (m.code == GQ_F16 && !half))
        refuse(PyExc_TypeError, "%s must be float32 or bfloat16%s", what, half ? " or float16" : "");
    if (!t.is_cuda()) refuse(PyExc_ValueError, "%s must be a CUDA tensor", what);
    const int64_t dims = t.dim();
    if (dims < 2) refuse(PyExc_ValueError, "%s must have at least two dimensions", what);
    const auto size = t.sizes(), stride = t.strides();
    m.index = t.get_device();
    m.cols = size[dims - 1];
    if (m.cols < 1 || (stride[dims - 1] != 1 && m.cols > 1))
        refuse(PyExc_ValueError, "%s: the last dimension must be contiguous and not empty", what);
    m.rows = 1;
    m.ld = m.cols;  // a single row has no next one
    for (int64_t d = dims - 2; d >= 0; --d) {
        if (size[d] != 1 && m.rows == 1) {
            m.ld = stride[d];
        } else if (size[d] != 1 && m.rows > 0 && stride[d] != m.ld * m.rows) {
            refuse(PyExc_ValueError, "%s: the leading dimensions cannot be viewed as one", what);
        }
        m.rows *= size[d];
    }
    if (m.rows <= 1) m.ld = m.cols;
    if (m.rows > 1 && m.ld < m.cols) refuse(PyExc_ValueError, "%s: rows overlap", what);
    m.p = t.data_ptr();
    return m;
}

// The device of the call's tensors, made current, and its current stream.
struct Place {
    c10::cuda::OptionalCUDAGuard guard;
    void* stream;
    explicit Place(int index) {
        if (c10::cuda::current_device() != index) guard.set_index(static_cast<c10::DeviceIndex>(index));
        stream = c10::cuda::getCurrentCUDAStream(static_cast<c10::DeviceIndex>(index)).stream();
    }
};

at::Tensor empty(at::IntArrayRef size, at::ScalarType type, int index) {
    return at::detail::empty_cuda(size, type,
                                  c10::Device(c10::kCUDA, static_cast<c10::DeviceIndex>(index)),
                                  std::nullopt);
}

// An optional per-column vector: its address, and its type in *code.
const void* vector(PyObject* o, int64_t n, int index, int* code, const char* what) {
    if (o == Py_None) return nullptr;
    const at::Tensor& t = tensor(o, what);
    const int c = type_code(t.scalar_type());
    if (c < 0 || c == GQ_F16) refuse(PyExc_TypeError, "%s must be float32 or bfloat16", what);
    if (!t.is_cuda() || t.get_device() != index || t.dim() != 1 || t.size(0) != n || !t.is_contiguous())
        refuse(PyExc_ValueError, "%s must be contiguous, %lld elements, on cuda:%d", what,
               static_cast<long long>(n), index);
    if (*code >= 0 && *code != c) refuse(PyExc_TypeError, "%s must be of the other vector's type", what);
    *code = c;
    return t.data_ptr();
}
const float* floats(PyObject* o, int64_t n, int index, const char* what) {
    int code = GQ_F32;
    if (o == Py_None) refuse(PyExc_ValueError, "%s is missing", what);
    return static_cast<const float*>(vector(o, n, index, &code, what));
}

uint64_t unsigned64(PyObject* o, const char* what) {
    PyObject* n = PyNumber_Index(o);
    if (!n) throw Refused{};
    const unsigned long long v = PyLong_AsUnsignedLongLong(n);
    Py_DECREF(n);
    if (v == static_cast<unsigned long long>(-1) && PyErr_Occurred()) {
        PyErr_Clear();
        refuse(PyExc_ValueError, "%s must be an unsigned 64-bit number", what);
    }
    return v;
}
int64_t signed64(PyObject* o) {
    const long long v = PyLong_AsLongLong(o);
    if (v == -1 && PyErr_Occurred()) throw Refused{};
    return v;
}
bool truth(PyObject* o) {
    const int v = PyObject_IsTrue(o);
    if (v < 0) throw Refused{};
    return v != 0;
}

struct Rounding {
    int mode = GQ_ACT_NEAREST;
    uint64_t seed = 0, step = 0;
    Rounding(PyObject* s, PyObject* t) {
        step = unsigned64(t, "step");
        if (s == Py_None) return;
        mode = GQ_ACT_RANDOM;
        seed = unsigned64(s, "seed");
    }
};

int output_code(PyObject* o, const char* what) {  // GQ_F32 or GQ_BF16, as the package maps the types
    const int64_t c = signed64(o);
    if (c != GQ_F32 && c != GQ_BF16) refuse(PyExc_TypeError, "%s must be float32 or bfloat16", what);
    return static_cast<int>(c);
}
at::ScalarType scalar_of(int code) {
    return code == GQ_F32 ? at::kFloat : code == GQ_BF16 ? at::kBFloat16 : at::kHalf;
}

// A checkpoint as the package passes it: (codes, exponents, columns), or (bytes, None, columns) with the
// codes and behind them the exponents of all rows in one tensor.  Addresses are taken from the tensors at
// every call, and what the tensors hold is checked against the size: their storage may have been replaced.
struct Saved {
    const int8_t* codes = nullptr;
    const uint8_t* exps = nullptr;
    int64_t rows = 0, cols = 0;
    int index = 0;
    explicit Saved(PyObject* const* a) : cols(signed64(a[2])) {
        const at::Tensor& c = tensor(a[0], "the checkpoint");
        if (cols < 1 || cols >= int64_t(1) << 31) refuse(PyExc_ValueError, "the checkpoint has no columns");
        const int64_t pitch = (cols + 31) / 32 * 32, epitch = (pitch / 32 + 15) / 16 * 16;
        const bool apart = a[1] != Py_None;
        holds(c, apart ? pitch : pitch + epitch);
        index = c.get_device();
        rows = c.size(0);
        codes = static_cast<const int8_t*>(c.data_ptr());
        exps = reinterpret_cast<const uint8_t*>(codes) + rows * pitch;
        if (apart) {
            const at::Tensor& e = tensor(a[1], "the checkpoint's exponents");
            holds(e, epitch);
            if (e.get_device() != index || e.size(0) != rows)
                refuse(PyExc_ValueError, "the checkpoint's exponents are not those of its codes");
            exps = static_cast<const uint8_t*>(e.data_ptr());
        }
    }
    static void holds(const at::Tensor& t, int64_t pitch) {
        if (!t.is_cuda() || t.dim() != 2 || t.size(1) != pitch || t.element_size() != 1 || !t.is_contiguous())
            refuse(PyExc_ValueError, "the checkpoint must be contiguous rows of %lld bytes on a CUDA device",
                   static_cast<long long>(pitch));
    }
    void covers(int64_t r, int64_t c, int i) const {
        if (rows != r || (c >= 0 && cols != c) || index != i)
            refuse(PyExc_ValueError, "the checkpoint holds %lld x %lld on cuda:%d",
                   static_cast<long long>(rows), static_cast<long long>(cols), index);
    }
};
// A new one.
struct NewSaved {
    at::Tensor data;
    int8_t* codes = nullptr;
    uint8_t* exps = nullptr;
    void make(int64_t rows, int64_t cols, int index) {
        const int64_t pitch = (cols + 31) / 32 * 32, epitch = (pitch / 32 + 15) / 16 * 16;
        data = empty({rows, pitch + epitch}, at::kByte, index);
        codes = static_cast<int8_t*>(data.data_ptr());
        exps = reinterpret_cast<uint8_t*>(codes) + rows * pitch;
    }
};

PyObject* wrap(const at::Tensor& t) { return t.defined() ? THPVariable_Wrap(t) : Py_NewRef(Py_None); }

struct Workspace {
    at::Tensor own;
    void* p;
    size_t bytes;
    Workspace(PyObject* o, size_t need, int index) {
        if (o == Py_None) {
            own = empty({static_cast<int64_t>(need)}, at::kByte, index);
            p = own.data_ptr();
            bytes = need;
        } else {
            const at::Tensor& t = tensor(o, "the workspace");
            if (!t.is_cuda() || t.get_device() != index || !t.is_contiguous())
                refuse(PyExc_ValueError, "the workspace must be a contiguous tensor on cuda:%d", index);
            p = t.data_ptr();
            bytes = t.nbytes();
        }
    }
};

// ---- the entry points: positional arguments, all of them given ---------------------------------

void count(Py_ssize_t have, Py_ssize_t want) {
    if (have != want) refuse(PyExc_TypeError, "%zd arguments, %zd expected", have, want);
}

// (x, seed, step) -> data
PyObject* act_quantize(PyObject* const* a, Py_ssize_t n) {
    count(n, 3);
    const at::Tensor& x = tensor(a[0], "x");
    const Matrix m = matrix(x, "x");
    const Rounding r(a[1], a[2]);
    const Place at(m.index);
    NewSaved s;
    s.make(m.rows, m.cols, m.index);
    check(api.act_quantize(m.p, m.code, m.rows, m.cols, m.ld, r.mode, r.seed, r.step, s.codes, s.exps,
                           at.stream),
          "gq_act_quantize");
    return wrap(s.data);
}

// (checkpoint x 3, shape, out or None, type code) -> out
PyObject* act_dequantize(PyObject* const* a, Py_ssize_t n) {
    count(n, 6);
    const Saved s(a);
    const Place at(s.index);
    at::Tensor out;
    if (a[4] == Py_None) {
        const int64_t c = signed64(a[5]);
        if (c != GQ_F32 && c != GQ_BF16 && c != GQ_F16)
            refuse(PyExc_TypeError, "values are float32, bfloat16 or float16");
        const std::unique_ptr<PyObject, void (*)(PyObject*)> sizes(PySequence_Tuple(a[3]), Py_DecRef);
        if (!sizes) throw Refused{};
        c10::SmallVector<int64_t, 8> shape;
        for (Py_ssize_t i = 0; i < PyTuple_GET_SIZE(sizes.get()); ++i)
            shape.push_back(signed64(PyTuple_GET_ITEM(sizes.get(), i)));
        out = empty(shape, scalar_of(static_cast<int>(c)), s.index);
    } else {
        out = tensor(a[4], "out");
    }
    const Matrix m = matrix(out, "out", true);
    if (m.rows != s.rows || m.cols != s.cols || m.index != s.index)
        refuse(PyExc_ValueError, "out must hold %lld x %lld on cuda:%d", static_cast<long long>(s.rows),
               static_cast<long long>(s.cols), s.index);
    check(api.act_dequantize(s.codes, s.exps, s.rows, s.cols, m.p, m.code, m.ld, at.stream),
          "gq_act_dequantize");
    return wrap(out);
}

// (x, weight, bias, eps, checkpoint, seed, step)
//   -> (y, mean, rstd, data or None)
PyObject* layernorm_forward(PyObject* const* a, Py_ssize_t n) {
    count(n, 7);
    const at::Tensor& x = tensor(a[0], "x");
    const Matrix m = matrix(x, "x");
    int wcode = -1;
    const void* w = vector(a[1], m.cols, m.index, &wcode, "weight");
    const void* b = vector(a[2], m.cols, m.index, &wcode, "bias");
    const double eps = PyFloat_AsDouble(a[3]);
    if (eps == -1.0 && PyErr_Occurred()) throw Refused{};
    if (!(eps >= 0.0)) refuse(PyExc_ValueError, "eps must not be negative");
    const Rounding r(a[5], a[6]);
    const Place at(m.index);
    const at::Tensor y = empty(x.sizes(), x.scalar_type(), m.index);
    const at::Tensor mean = empty({m.rows}, at::kFloat, m.index), rstd = empty({m.rows}, at::kFloat, m.index);
    NewSaved s;
    if (truth(a[4])) s.make(m.rows, m.cols, m.index);
    check(api.layernorm_forward(m.p, m.code, m.rows, m.cols, m.ld, w, b, wcode < 0 ? GQ_F32 : wcode,
                                static_cast<float>(eps), y.data_ptr(), m.cols,
                                static_cast<float*>(mean.data_ptr()), static_cast<float*>(rstd.data_ptr()),
                                r.mode, r.seed, r.step, s.codes, s.exps, at.stream),
          "gq_layernorm_forward");
    return Py_BuildValue("NNNN", wrap(y), wrap(mean), wrap(rstd), wrap(s.data));
}

// (dy, weight, rstd, checkpoint x 3 or None x 3, x or None, mean or None, type code, ws or None)
//   -> (dx, dweight, dbias)
PyObject* layernorm_backward(PyObject* const* a, Py_ssize_t n) {
    count(n, 10);
    const at::Tensor& dy = tensor(a[0], "dy");
    const Matrix m = matrix(dy, "dy");
    int wcode = -1;
    const void* w = vector(a[1], m.cols, m.index, &wcode, "weight");
    const float* rstd = floats(a[2], m.rows, m.index, "rstd");
    const bool saved = a[3] != Py_None;
    if (saved == (a[6] != Py_None) || (a[6] == Py_None) != (a[7] == Py_None))
        refuse(PyExc_ValueError, "give either act, or x and mean");
    const int gcode = output_code(a[8], "grad_dtype");
    const int8_t* codes = nullptr;
    const uint8_t* exps = nullptr;
    const void* xp = nullptr;
    int64_t ldx = 0;
    const float* mean = nullptr;
    if (saved) {
        const Saved s(a + 3);
        s.covers(m.rows, m.cols, m.index);
        codes = s.codes;
        exps = s.exps;
    } else {
        const Matrix x = matrix(tensor(a[6], "x"), "x");
        if (x.code != m.code || x.rows != m.rows || x.cols != m.cols || x.index != m.index)
            refuse(PyExc_ValueError, "x must match dy in shape, type and device");
        xp = x.p;
        ldx = x.ld;
        mean = floats(a[7], m.rows, m.index, "mean");
    }
    const Place at(m.index);
    const Workspace ws(a[9], a[9] == Py_None ? api.layernorm_workspace_bytes(m.rows, m.cols) : 0, m.index);
    const at::Tensor dx = empty(dy.sizes(), dy.scalar_type(), m.index);
    const at::Tensor dw = empty({m.cols}, scalar_of(gcode), m.index);
    const at::Tensor db = empty({m.cols}, scalar_of(gcode), m.index);
    check(api.layernorm_backward(m.p, m.code, m.rows, m.cols, m.ld, w, wcode < 0 ? GQ_F32 : wcode, rstd,
                                 codes, exps, xp, ldx, mean, dx.data_ptr(), m.cols, dw.data_ptr(),
                                 db.data_ptr(), gcode, ws.p, ws.bytes, at.stream),
          "gq_layernorm_backward");
    return Py_BuildValue("NNN", wrap(dx), wrap(dw), wrap(db));
}

// (u, form, checkpoint, seed, step) -> (h, data or None)
PyObject* gelu_forward(PyObject* const* a, Py_ssize_t n) {
    count(n, 5);
    const at::Tensor& u = tensor(a[0], "u");
    const Matrix m = matrix(u, "u");
    const Rounding r(a[3], a[4]);
    const Place at(m.index);
    const at::Tensor h = empty(u.sizes(), u.scalar_type(), m.index);
    NewSaved s;
    if (truth(a[2])) s.make(m.rows, m.cols, m.index);
    check(api.gelu_forward(m.p, m.code, m.rows, m.cols, m.ld, static_cast<int>(signed64(a[1])), h.data_ptr(),
                           m.cols, r.mode, r.seed, r.step, s.codes, s.exps, at.stream),
          "gq_gelu_forward");
    return Py_BuildValue("NN", wrap(h), wrap(s.data));
}

// (dh, checkpoint x 3, form, output) -> du, or (du, h)
PyObject* gelu_backward(PyObject* const* a, Py_ssize_t n) {
    count(n, 6);
    const at::Tensor& dh = tensor(a[0], "dh");
    const Matrix m = matrix(dh, "dh");
    const Saved s(a + 1);
    s.covers(m.rows, m.cols, m.index);
    const Place at(m.index);
    const at::Tensor du = empty(dh.sizes(), dh.scalar_type(), m.index);
    at::Tensor h;
    if (truth(a[5])) h = empty(dh.sizes(), dh.scalar_type(), m.index);
    check(api.gelu_backward(m.p, m.code, m.rows, m.cols, m.ld, s.codes, s.exps,
                            static_cast<int>(signed64(a[4])), du.data_ptr(), m.cols,
                            h.defined() ? h.data_ptr() : nullptr, m.cols, at.stream),
          "gq_gelu_backward");
    if (!h.defined()) return wrap(du);
    return Py_BuildValue("NN", wrap(du), wrap(h));
}

// (dy, checkpoint x 3, scale, shift, type code, bias, ws or None) -> (dw, dbias or None)
PyObject* linear_wgrad(PyObject* const* a, Py_ssize_t n) {
    count(n, 9);
    const at::Tensor& dy = tensor(a[0], "dy");
    const Matrix m = matrix(dy, "dy");
    const Saved s(a + 1);
    s.covers(m.rows, -1, m.index);
    int f32 = GQ_F32;
    const float* scale = static_cast<const float*>(vector(a[4], s.cols, m.index, &f32, "scale"));
    const float* shift = static_cast<const float*>(vector(a[5], s.cols, m.index, &f32, "shift"));
    const int code = output_code(a[6], "out_dtype");
    const Place at(m.index);
    const Workspace ws(a[8], a[8] == Py_None ? api.linear_wgrad_workspace_bytes(m.p, m.code, m.rows, m.cols,
                                                                                m.ld, s.cols)
                                             : 0,
                       m.index);
    const at::Tensor dw = empty({m.cols, s.cols}, scalar_of(code), m.index);
    at::Tensor db;
    if (truth(a[7])) db = empty({m.cols}, at::kFloat, m.index);
    check(api.linear_wgrad(m.p, m.code, m.rows, m.cols, m.ld, s.codes, s.exps, s.cols, scale, shift,
                           dw.data_ptr(), code, s.cols,
                           db.defined() ? static_cast<float*>(db.data_ptr()) : nullptr, ws.p, ws.bytes,
                           at.stream),
          "gq_linear_wgrad");
    return Py_BuildValue("NN", wrap(dw), wrap(db));
}

// (dy, cols) -> bytes
PyObject* linear_wgrad_workspace_bytes(PyObject* const* a, Py_ssize_t n) {
    count(n, 2);
    const Matrix m = matrix(tensor(a[0], "dy"), "dy");
    return PyLong_FromSize_t(
        api.linear_wgrad_workspace_bytes(m.p, m.code, m.rows, m.cols, m.ld, signed64(a[1])));
}

// (dy, cols) -> 8 numbers
PyObject* linear_wgrad_plan(PyObject* const* a, Py_ssize_t n) {
    count(n, 2);
    const Matrix m = matrix(tensor(a[0], "dy"), "dy");
    const Place at(m.index);
    int64_t p[8];
    check(api.linear_wgrad_plan(m.p, m.code, m.rows, m.cols, m.ld, signed64(a[1]), p), "gq_linear_wgrad_plan");
    PyObject* out = PyTuple_New(8);
    for (Py_ssize_t i = 0; out && i < 8; ++i) {
        PyObject* v = PyLong_FromLongLong(p[i]);
        if (!v) {
            Py_DECREF(out);
            return nullptr;
        }
        PyTuple_SET_ITEM(out, i, v);
    }
    return out;
}

// (the package's GQError, the addresses of Api's functions)
PyObject* bind(PyObject* const* a, Py_ssize_t n) {
    count(n, 1 + kFunctions);
    void* f[kFunctions];
    for (int i = 0; i < kFunctions; ++i) {
        f[i] = PyLong_AsVoidPtr(a[1 + i]);
        if (!f[i]) refuse(PyExc_ValueError, "function %d is missing", i);
    }
    memcpy(&api, f, sizeof api);
    Py_XSETREF(gq_error, Py_NewRef(a[0]));
    return Py_NewRef(Py_None);
}

// No C++ exception leaves an entry point: torch's become Python's, a refusal has set one already.
template <PyObject* (*F)(PyObject* const*, Py_ssize_t)>
PyObject* entry(PyObject*, PyObject* const* a, Py_ssize_t n) {
    HANDLE_TH_ERRORS
    try {
        return F(a, n);
    } catch (const Refused&) {
        return nullptr;
    }
    END_HANDLE_TH_ERRORS
}
#define GQ_ENTRY(NAME) \
    {#NAME, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(&entry<NAME>)), METH_FASTCALL, nullptr}
PyMethodDef methods[] = {GQ_ENTRY(bind),
                         GQ_ENTRY(act_quantize),
                         GQ_ENTRY(act_dequantize),
                         GQ_ENTRY(layernorm_forward),
                         GQ_ENTRY(layernorm_backward),
                         GQ_ENTRY(gelu_forward),
                         GQ_ENTRY(gelu_backward),
                         GQ_ENTRY(linear_wgrad),
                         GQ_ENTRY(linear_wgrad_workspace_bytes),
                         GQ_ENTRY(linear_wgrad_plan),
                         {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "gq_native", nullptr, -1, methods,
                      nullptr,               nullptr,     nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit_gq_native() { return PyModule_Create(&module); }
