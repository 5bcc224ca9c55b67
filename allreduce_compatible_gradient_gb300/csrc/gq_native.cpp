// gq_native.cpp -- Python entry points of the operators around the linear layers of a training step and of
// the optimizer's step (include/gq.h) on torch tensors.
//
// Argument checks, allocation of outputs and the call of libgq.so, in C++: a call on a small matrix
// takes 3 to 5 us on the GPU, and the same marshalling in Python took 11 to 22 us on the host.  The
// functions of libgq.so come in by address (bind), so that the extension works with whichever build
// of the library the package has loaded.  Nothing here touches data.
#include <Python.h>

#include <ATen/ATen.h>
#include <ATen/cuda/EmptyTensor.h>
#include <c10/cuda/CUDACachingAllocator.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include <algorithm>
#include <cstdint>
#include <memory>
#include <utility>
#include <vector>

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
    decltype(&gq_fp8_quantize) fp8_quantize;
    decltype(&gq_fp8_dequantize) fp8_dequantize;
    decltype(&gq_fp8_linear_workspace_bytes) fp8_linear_workspace_bytes;
    decltype(&gq_fp8_linear) fp8_linear;
    decltype(&gq_fp8_linear_dgrad) fp8_linear_dgrad;
    decltype(&gq_tensors_norm_workspace_bytes) tensors_norm_workspace_bytes;
    decltype(&gq_tensors_norm) tensors_norm;
    decltype(&gq_adamw_step_places) adamw_step_places;
    decltype(&gq_adamw_values) adamw_values;
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

// Autograd's count of in-place changes: a backward pass that saved the old values refuses the new ones.
void changed(const at::Tensor& t) {
    if (!t.is_inference()) t.unsafeGetTensorImpl()->bump_version();
}

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
    if (a[4] != Py_None) changed(out);
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

// ---- 8-bit floating point ------------------------------------------------------------------

int64_t fp8_exp_bytes(int64_t rows, int64_t cols) { return (rows + 127) / 128 * ((cols + 511) / 512) * 512; }

// A matrix in 8-bit floating point as the package passes it: (codes, exps, exps_t or None, rows, columns,
// tiles), or (bytes, None, None, ...) with the codes, the exponents and (tiles) those of the transposed matrix
// one after the other.  Checked against the size at every call, like Saved.
struct Fp8 {
    uint8_t *codes = nullptr, *exps = nullptr, *exps_t = nullptr;
    int64_t rows = 0, cols = 0;
    bool tiles = false;
    int index = 0;
    explicit Fp8(PyObject* const* a) : rows(signed64(a[3])), cols(signed64(a[4])), tiles(truth(a[5])) {
        const at::Tensor& c = tensor(a[0], "the matrix's codes");
        if (rows < 0 || cols < 1 || rows >= int64_t(1) << 31 || cols >= int64_t(1) << 31)
            refuse(PyExc_ValueError, "the matrix has no such size");
        const int64_t pitch = (cols + 15) / 16 * 16, e = fp8_exp_bytes(rows, cols), et = fp8_exp_bytes(cols, rows);
        if (a[1] == Py_None) {
            codes = bytes(c, rows * pitch + e + (tiles ? et : 0), c);
            exps = codes + rows * pitch;
            if (tiles) exps_t = exps + e;
        } else {
            codes = bytes(c, rows * pitch, c);
            exps = bytes(tensor(a[1], "the matrix's exponents"), e, c);
            if (a[2] != Py_None) exps_t = bytes(tensor(a[2], "the transposed matrix's exponents"), et, c);
        }
        index = c.get_device();
    }
    static uint8_t* bytes(const at::Tensor& t, int64_t n, const at::Tensor& beside) {
        if (!t.is_cuda() || t.get_device() != beside.get_device() || t.element_size() != 1 || t.numel() != n ||
            !t.is_contiguous())
            refuse(PyExc_ValueError, "the matrix must be contiguous bytes on one CUDA device, %lld in one of its parts",
                   static_cast<long long>(n));
        return static_cast<uint8_t*>(t.data_ptr());
    }
};

// (x, tiles) -> data
PyObject* fp8_quantize(PyObject* const* a, Py_ssize_t n) {
    count(n, 2);
    const Matrix m = matrix(tensor(a[0], "x"), "x");
    const bool tiles = truth(a[1]);
    const Place at(m.index);
    const int64_t codes = m.rows * ((m.cols + 15) / 16 * 16), e = fp8_exp_bytes(m.rows, m.cols);
    const at::Tensor data =
        empty({codes + e + (tiles ? fp8_exp_bytes(m.cols, m.rows) : 0)}, at::kByte, m.index);
    uint8_t* p = static_cast<uint8_t*>(data.data_ptr());
    check(api.fp8_quantize(m.p, m.code, m.rows, m.cols, m.ld, tiles ? 128 : 1, p, p + codes,
                           tiles ? p + codes + e : nullptr, at.stream),
          "gq_fp8_quantize");
    return wrap(data);
}

c10::SmallVector<int64_t, 8> sizes_of(PyObject* o) {
    const std::unique_ptr<PyObject, void (*)(PyObject*)> sizes(PySequence_Tuple(o), Py_DecRef);
    if (!sizes) throw Refused{};
    c10::SmallVector<int64_t, 8> shape;
    for (Py_ssize_t i = 0; i < PyTuple_GET_SIZE(sizes.get()); ++i)
        shape.push_back(signed64(PyTuple_GET_ITEM(sizes.get(), i)));
    return shape;
}

// (matrix x 6, shape, out or None, type code) -> out
PyObject* fp8_dequantize(PyObject* const* a, Py_ssize_t n) {
    count(n, 9);
    const Fp8 s(a);
    const Place at(s.index);
    at::Tensor out;
    if (a[7] == Py_None) {
        const int64_t c = signed64(a[8]);
        if (c != GQ_F32 && c != GQ_BF16 && c != GQ_F16)
            refuse(PyExc_TypeError, "values are float32, bfloat16 or float16");
        out = empty(sizes_of(a[6]), scalar_of(static_cast<int>(c)), s.index);
    } else {
        out = tensor(a[7], "out");
    }
    const Matrix m = matrix(out, "out", true);
    if (m.rows != s.rows || m.cols != s.cols || m.index != s.index)
        refuse(PyExc_ValueError, "out must hold %lld x %lld on cuda:%d", static_cast<long long>(s.rows),
               static_cast<long long>(s.cols), s.index);
    check(api.fp8_dequantize(s.codes, s.exps, s.rows, s.cols, m.p, m.code, m.ld, at.stream), "gq_fp8_dequantize");
    if (a[7] != Py_None) changed(out);
    return wrap(out);
}

// The tokens' operand of a product: a tensor, whose codes then live in `own` for the call, or a matrix in
// 8-bit floating point.
struct Tokens {
    const void* p = nullptr;
    int code = GQ_BF16, index = 0;
    int64_t ld = 0, rows = 0, cols = 0;
    uint8_t *codes = nullptr, *exps = nullptr;
    c10::SmallVector<int64_t, 8> shape;  // of the tensor it was made from
    at::Tensor own;
    Tokens(PyObject* const* a, const char* what) {  // tensor or None, matrix x 6 or None x 6, shape or None
        if (a[0] != Py_None) {
            const at::Tensor& x = tensor(a[0], what);
            const Matrix m = matrix(x, what);
            p = m.p; code = m.code; index = m.index; ld = m.ld; rows = m.rows; cols = m.cols;
            shape.append(x.sizes().begin(), x.sizes().end());
        } else {
            const Fp8 s(a + 1);
            if (s.tiles)
                refuse(PyExc_ValueError, "%s must have an exponent for each of its rows' blocks (tiles=False)", what);
            index = s.index; rows = s.rows; cols = s.cols; codes = s.codes; exps = s.exps;
            shape = sizes_of(a[7]);
        }
    }
    void make(int64_t outs) {
        const size_t need = codes || !p ? 0 : api.fp8_linear_workspace_bytes(rows, cols, outs);
        if (need == 0) return;
        own = empty({static_cast<int64_t>(need)}, at::kByte, index);
        codes = static_cast<uint8_t*>(own.data_ptr());
        exps = codes + rows * ((cols + 15) / 16 * 16);
    }
    at::Tensor result(int64_t width, PyObject* type) {
        c10::SmallVector<int64_t, 8> size(shape);
        int64_t n = size.empty() ? -1 : 1;
        for (size_t i = 0; i + 1 < size.size(); ++i) n *= size[i];
        if (n != rows) refuse(PyExc_ValueError, "the matrix's shape is not that of its %lld rows", static_cast<long long>(rows));
        size.back() = width;
        return empty(size, scalar_of(output_code(type, "out_dtype")), index);
    }
};

// (x or None, matrix x 6 or None x 6, shape or None, weight x 6, bias or None, type code) -> y
PyObject* fp8_linear(PyObject* const* a, Py_ssize_t n) {
    count(n, 16);
    Tokens x(a, "x");
    const Fp8 w(a + 8);
    if (w.cols != x.cols || w.index != x.index)
        refuse(PyExc_ValueError, "the weight holds %lld x %lld on cuda:%d", static_cast<long long>(w.rows),
               static_cast<long long>(w.cols), w.index);
    if (w.rows < 1) refuse(PyExc_ValueError, "the weight has no rows");
    int f32 = GQ_F32;
    const float* bias = static_cast<const float*>(vector(a[14], w.rows, x.index, &f32, "bias"));
    const Place at(x.index);
    x.make(w.rows);
    const at::Tensor y = x.result(w.rows, a[15]);
    check(api.fp8_linear(x.p, x.code, x.ld, x.codes, x.exps, x.rows, x.cols, w.codes, w.exps, w.rows, bias,
                         y.data_ptr(), type_code(y.scalar_type()), w.rows, at.stream),
          "gq_fp8_linear");
    return wrap(y);
}

// (dy or None, matrix x 6 or None x 6, shape or None, weight x 6, type code) -> dx
PyObject* fp8_linear_dgrad(PyObject* const* a, Py_ssize_t n) {
    count(n, 15);
    Tokens dy(a, "dy");
    const Fp8 w(a + 8);
    if (w.rows != dy.cols || w.index != dy.index)
        refuse(PyExc_ValueError, "the weight holds %lld x %lld on cuda:%d", static_cast<long long>(w.rows),
               static_cast<long long>(w.cols), w.index);
    if (!w.exps_t) refuse(PyExc_ValueError, "the weight has no exponents of its transposed matrix (tiles=True)");
    const Place at(dy.index);
    dy.make(w.cols);
    const at::Tensor dx = dy.result(w.cols, a[14]);
    check(api.fp8_linear_dgrad(dy.p, dy.code, dy.ld, dy.codes, dy.exps, dy.rows, dy.cols, w.codes, w.exps_t,
                               w.cols, dx.data_ptr(), type_code(dx.scalar_type()), w.cols, at.stream),
          "gq_fp8_linear_dgrad");
    return wrap(dx);
}

// ---- the optimizer's step ------------------------------------------------------------------

// A list or tuple, borrowed for the call.
struct Items {
    PyObject* seq;
    Py_ssize_t n;
    Items(PyObject* o, const char* what) {
        if (!PyList_Check(o) && !PyTuple_Check(o)) refuse(PyExc_TypeError, "%s must be a list or a tuple", what);
        seq = PySequence_Fast(o, what);
        if (!seq) throw Refused{};
        n = PySequence_Fast_GET_SIZE(seq);
    }
    ~Items() { Py_DECREF(seq); }
    Items(const Items&) = delete;
    PyObject* operator[](Py_ssize_t i) const { return PySequence_Fast_GET_ITEM(seq, i); }
};

// A contiguous tensor of a list, on the list's device; index < 0 before the first.
const at::Tensor& part(PyObject* o, int* index, const char* what) {
    const at::Tensor& t = tensor(o, what);
    if (!t.is_cuda() || !t.is_contiguous()) refuse(PyExc_ValueError, "%s must be contiguous CUDA tensors", what);
    if (*index < 0) *index = t.get_device();
    if (t.get_device() != *index) refuse(PyExc_ValueError, "%s must be on cuda:%d like the others", what, *index);
    return t;
}
void same_type(int* code, const at::Tensor& t, const char* what) {
    const int c = type_code(t.scalar_type());
    if (c != GQ_F32 && c != GQ_BF16) refuse(PyExc_TypeError, "%s must be float32 or bfloat16", what);
    if (*code >= 0 && *code != c) refuse(PyExc_TypeError, "%s must be of one type", what);
    *code = c;
}

// Ranges of memory that a call writes, each element by a thread of its own: none twice.
struct Apart {
    std::vector<std::pair<uintptr_t, int64_t>> ranges;
    explicit Apart(Py_ssize_t n) { ranges.reserve(n); }
    void add(const void* p, int64_t bytes) {
        if (bytes > 0) ranges.emplace_back(reinterpret_cast<uintptr_t>(p), bytes);
    }
    void check(const char* what) {
        std::sort(ranges.begin(), ranges.end());
        for (size_t i = 1; i < ranges.size(); ++i)
            if (ranges[i].first - ranges[i - 1].first < static_cast<uintptr_t>(ranges[i - 1].second))
                refuse(PyExc_ValueError, "%s is there twice, or a part of it", what);
    }
};

struct State {
    void *m, *v;
    uint8_t* e = nullptr;
};
// (m, v) fp32, or (m, v, exps) bytes of a tensor of n elements.
State state(PyObject* o, int64_t n, int* index, bool eight) {
    if (!PyTuple_Check(o) || PyTuple_GET_SIZE(o) != (eight ? 3 : 2))
        refuse(PyExc_TypeError, "states must be Adam8, or pairs of float32 tensors, all of one kind");
    const at::Tensor &m = part(PyTuple_GET_ITEM(o, 0), index, "states"),
                     &v = part(PyTuple_GET_ITEM(o, 1), index, "states");
    State s;
    if (eight) {
        const at::Tensor& e = part(PyTuple_GET_ITEM(o, 2), index, "states");
        const int64_t room = (n + 31) / 32 * 32;
        if (m.scalar_type() != at::kByte || v.scalar_type() != at::kByte || e.scalar_type() != at::kByte)
            refuse(PyExc_TypeError, "8-bit states must be uint8 tensors");
        if (m.numel() != room || v.numel() != room || e.numel() != room / 16)
            refuse(PyExc_ValueError, "an 8-bit state of %lld elements has %lld, %lld and %lld bytes",
                   static_cast<long long>(n), static_cast<long long>(room), static_cast<long long>(room),
                   static_cast<long long>(room / 16));
        s.e = static_cast<uint8_t*>(e.data_ptr());
    } else {
        if (m.scalar_type() != at::kFloat || v.scalar_type() != at::kFloat)
            refuse(PyExc_TypeError, "states must be Adam8, or pairs of float32 tensors, all of one kind");
        if (m.numel() != n || v.numel() != n)
            refuse(PyExc_ValueError, "a state must have its parameter's %lld elements", static_cast<long long>(n));
    }
    s.m = m.data_ptr();
    s.v = v.data_ptr();
    return s;
}
bool in_8_bits(const Items& states) {
    return states.n > 0 && PyTuple_Check(states[0]) && PyTuple_GET_SIZE(states[0]) == 3;
}
double number(PyObject* o, const char* what) {
    const double v = PyFloat_AsDouble(o);
    if (v == -1.0 && PyErr_Occurred()) {
        PyErr_Clear();
        refuse(PyExc_TypeError, "%s must be a number", what);
    }
    return v;
}
const float* scalar(PyObject* o, int index, const char* what) {
    if (o == Py_None) return nullptr;
    const at::Tensor& t = tensor(o, what);
    if (!t.is_cuda() || t.get_device() != index || t.scalar_type() != at::kFloat || t.numel() != 1)
        refuse(PyExc_ValueError, "%s must be one float32 number on cuda:%d", what, index);
    return static_cast<const float*>(t.data_ptr());
}

// (tensors, ws or None) -> norm
PyObject* tensors_norm(PyObject* const* a, Py_ssize_t n) {
    count(n, 2);
    const Items list(a[0], "tensors");
    if (list.n == 0) refuse(PyExc_ValueError, "there are no tensors");
    std::vector<const void*> p(list.n);
    std::vector<int64_t> numel(list.n);
    int index = -1, code = -1;
    for (Py_ssize_t i = 0; i < list.n; ++i) {
        const at::Tensor& t = part(list[i], &index, "tensors");
        same_type(&code, t, "tensors");
        p[i] = t.data_ptr();
        numel[i] = t.numel();
    }
    const Place at(index);
    // (a norm that is kept holds no more than its four bytes; the workspace goes back to the allocator, in the
    // stream's order, without having been a tensor)
    const at::Tensor norm = empty({1}, at::kFloat, index);
    float* const out = static_cast<float*>(norm.data_ptr());
    if (a[1] == Py_None) {
        const size_t need = api.tensors_norm_workspace_bytes(list.n);
        const c10::DataPtr own = c10::cuda::CUDACachingAllocator::get()->allocate(need);
        check(api.tensors_norm(list.n, p.data(), numel.data(), code, out, own.get(), need, at.stream),
              "gq_tensors_norm");
    } else {
        const Workspace ws(a[1], 0, index);
        check(api.tensors_norm(list.n, p.data(), numel.data(), code, out, ws.p, ws.bytes, at.stream),
              "gq_tensors_norm");
    }
    return wrap(norm);
}

// (params, grads, states, step, lr, beta1, beta2, eps, weight_decay, norm or None, max_norm or None, seed or
// None, first, places or None, step's places or None) -> None
PyObject* adamw_step(PyObject* const* a, Py_ssize_t n) {
    count(n, 15);
    const Items params(a[0], "params"), grads(a[1], "grads"), states(a[2], "states");
    if (grads.n != params.n || states.n != params.n)
        refuse(PyExc_ValueError, "%zd parameters, %zd gradients and %zd states", params.n, grads.n, states.n);
    if (params.n == 0) return Py_NewRef(Py_None);
    const bool eight = in_8_bits(states);
    std::vector<void*> p(params.n), m(params.n), v(params.n);
    std::vector<const void*> g(params.n);
    std::vector<uint8_t*> e(eight ? params.n : 0);
    std::vector<int64_t> numel(params.n);
    int index = -1, pcode = -1, gcode = -1;
    for (Py_ssize_t i = 0; i < params.n; ++i) {
        const at::Tensor &t = part(params[i], &index, "params"), &d = part(grads[i], &index, "grads");
        same_type(&pcode, t, "params");
        same_type(&gcode, d, "grads");
        numel[i] = t.numel();
        if (d.numel() != numel[i])
            refuse(PyExc_ValueError, "gradient %zd has %lld elements, its parameter %lld", i,
                   static_cast<long long>(d.numel()), static_cast<long long>(numel[i]));
        p[i] = t.data_ptr();
        g[i] = d.data_ptr();
        const State s = state(states[i], numel[i], &index, eight);
        m[i] = s.m;
        v[i] = s.v;
        if (eight) e[i] = s.e;
    }
    Apart written(4 * params.n);
    for (Py_ssize_t i = 0; i < params.n; ++i) {
        const int64_t room = eight ? (numel[i] + 31) / 32 * 32 : 4 * numel[i];
        written.add(p[i], (pcode == GQ_F32 ? 4 : 2) * numel[i]);
        written.add(m[i], room);
        written.add(v[i], room);
        if (eight) written.add(e[i], room / 16);
    }
    written.check("a parameter or a state");
    const int64_t* counter = nullptr;
    int64_t step = 1, counters = 0;
    if (THPVariable_Check(a[3])) {
        const at::Tensor& t = THPVariable_Unpack(a[3]);
        if (!t.is_cuda() || t.get_device() != index || t.scalar_type() != at::kLong || !t.is_contiguous() ||
            (t.numel() != 1 && a[14] == Py_None))
            refuse(PyExc_ValueError, "step must be a number, or one int64 number on cuda:%d", index);
        counter = static_cast<const int64_t*>(t.data_ptr());
        counters = t.numel();
    } else {
        step = signed64(a[3]);
        if (step < 1) refuse(PyExc_ValueError, "step must be at least 1");
    }
    const double lr = number(a[4], "lr"), beta1 = number(a[5], "betas"), beta2 = number(a[6], "betas"),
                 eps = number(a[7], "eps"), decay = number(a[8], "weight_decay");
    if (!(beta1 >= 0.0 && beta1 < 1.0 && beta2 >= 0.0 && beta2 < 1.0))
        refuse(PyExc_ValueError, "betas must be at least 0 and below 1");
    if (!(eps >= 0.0)) refuse(PyExc_ValueError, "eps must not be negative");
    const float* norm = scalar(a[9], index, "norm");
    double most = -1.0;
    if (a[10] != Py_None) {
        most = number(a[10], "max_norm");
        if (!(most >= 0.0)) refuse(PyExc_ValueError, "max_norm must not be negative");
        if (!norm) refuse(PyExc_ValueError, "max_norm needs the norm");
    }
    const uint64_t seed = a[11] == Py_None ? 0 : unsigned64(a[11], "seed");
    const int64_t first = signed64(a[12]);
    if (first < 0 || first > (int64_t(1) << 30) - params.n) refuse(PyExc_ValueError, "first is out of range");
    std::vector<int64_t> places;
    if (a[13] != Py_None) {
        const Items list(a[13], "places");
        if (list.n != params.n) refuse(PyExc_ValueError, "%zd parameters and %zd places", params.n, list.n);
        places.reserve(list.n);
        for (Py_ssize_t i = 0; i < list.n; ++i) {
            const int64_t k = signed64(list[i]);
            if (k < (i > 0 ? places.back() + 1 : 0) || k >= (int64_t(1) << 30) - first)
                refuse(PyExc_ValueError, "places must ascend from 0, and stay below 2^30 with first");
            places.push_back(k);
        }
    }
    std::vector<int64_t> step_places;
    if (a[14] != Py_None) {
        const Items list(a[14], "step_places");
        if (list.n != params.n) refuse(PyExc_ValueError, "%zd parameters and %zd places of steps", params.n, list.n);
        step_places.reserve(list.n);
        for (Py_ssize_t i = 0; i < list.n; ++i) {
            const int64_t k = signed64(list[i]);
            if (k < 0 || k >= counters) refuse(PyExc_ValueError, "step_places must be places in a tensor of steps");
            step_places.push_back(k);
        }
    }
    const Place at(index);
    check(api.adamw_step_places(params.n, p.data(), pcode, g.data(), gcode, m.data(), v.data(),
                         eight ? e.data() : nullptr, numel.data(), step, counter, lr, beta1, beta2, eps, decay, norm,
                         most, a[11] == Py_None ? GQ_ACT_NEAREST : GQ_ACT_RANDOM, seed, first,
                         places.empty() ? nullptr : places.data(),
                         step_places.empty() ? nullptr : step_places.data(), at.stream),
          "gq_adamw_step");
    for (Py_ssize_t i = 0; i < params.n; ++i) {
        changed(THPVariable_Unpack(params[i]));
        for (Py_ssize_t k = 0; k < (eight ? 3 : 2); ++k) changed(THPVariable_Unpack(PyTuple_GET_ITEM(states[i], k)));
    }
    return Py_NewRef(Py_None);
}

// (states, moments, roots: lists of tensors, of which the first give the elements) -> None
PyObject* adamw_values(PyObject* const* a, Py_ssize_t n) {
    count(n, 3);
    const Items states(a[0], "states"), moments(a[1], "out"), roots(a[2], "out");
    if (moments.n != states.n || roots.n != states.n)
        refuse(PyExc_ValueError, "%zd states, %zd and %zd outputs", states.n, moments.n, roots.n);
    if (states.n == 0) return Py_NewRef(Py_None);
    std::vector<const uint8_t*> m(states.n), v(states.n), e(states.n);
    std::vector<void*> x(states.n), r(states.n);
    std::vector<int64_t> numel(states.n);
    int index = -1, code = -1;
    for (Py_ssize_t i = 0; i < states.n; ++i) {
        const at::Tensor &t = part(moments[i], &index, "out"), &u = part(roots[i], &index, "out");
        same_type(&code, t, "out");
        same_type(&code, u, "out");
        numel[i] = t.numel();
        if (u.numel() != numel[i]) refuse(PyExc_ValueError, "the outputs of state %zd differ in size", i);
        const State s = state(states[i], numel[i], &index, true);
        m[i] = static_cast<const uint8_t*>(s.m);
        v[i] = static_cast<const uint8_t*>(s.v);
        e[i] = s.e;
        x[i] = t.data_ptr();
        r[i] = u.data_ptr();
    }
    Apart written(2 * states.n);
    for (Py_ssize_t i = 0; i < states.n; ++i)
        for (void* q : {x[i], r[i]}) written.add(q, (code == GQ_F32 ? 4 : 2) * numel[i]);
    written.check("an output");
    const Place at(index);
    check(api.adamw_values(states.n, m.data(), v.data(), e.data(), numel.data(), x.data(), r.data(), code, at.stream),
          "gq_adamw_values");
    for (Py_ssize_t i = 0; i < states.n; ++i) {
        changed(THPVariable_Unpack(moments[i]));
        changed(THPVariable_Unpack(roots[i]));
    }
    return Py_NewRef(Py_None);
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
                         GQ_ENTRY(fp8_quantize),
                         GQ_ENTRY(fp8_dequantize),
                         GQ_ENTRY(fp8_linear),
                         GQ_ENTRY(fp8_linear_dgrad),
                         GQ_ENTRY(tensors_norm),
                         GQ_ENTRY(adamw_step),
                         GQ_ENTRY(adamw_values),
                         {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "gq_native", nullptr, -1, methods,
                      nullptr,               nullptr,     nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit_gq_native() { return PyModule_Create(&module); }
