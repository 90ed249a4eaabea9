// Python entry points of the training-step operators: tensors checked and
// turned into the C ABI's pointers and sizes.
//
// The smallest calls (one layer's step, the rows of one token) run about 3 us
// on the GPU and take about as long to launch, so the binding may not cost
// more than that: the same checks through ctypes and Python attribute reads
// took 3.3 to 4.5 us a call, in which the GPU ran dry.
//
// Every function returns the C ABI's status (0 is success); wrong types and
// layouts raise TypeError, wrong sizes ValueError.
#define PY_SSIZE_T_CLEAN
#include <Python.h>
#include <torch/csrc/autograd/python_variable.h>

#include <algorithm>
#include <cstdint>
#include <stdexcept>
#include <string>

#include "../../include/adacomp.h"

namespace {

struct WrongType : std::runtime_error {
    using std::runtime_error::runtime_error;
};
struct WrongValue : std::runtime_error {
    using std::runtime_error::runtime_error;
};
struct PythonError {};   // already set

PyObject* current_device = nullptr;   // torch._C functions
PyObject* current_stream = nullptr;

const at::Tensor& tensor(PyObject* o, const char* name) {
    if (!THPVariable_Check(o)) throw WrongType(std::string(name) + " must be a tensor");
    return THPVariable_Unpack(o);
}

// The current device, asked once a call: the C ABI launches there, on its stream, so every tensor has to
// be there.
thread_local int device = -1;
int here() {
    if (device >= 0) return device;
    PyObject* o = PyObject_CallNoArgs(current_device);
    if (o == nullptr) throw PythonError();
    device = int(PyLong_AsLong(o));
    Py_DECREF(o);
    if (device < 0) throw PythonError();
    return device;
}
// Of a CUDA tensor.
void check_device(const at::Tensor& t, const char* name) {
    if (t.device().index() != here()) throw WrongValue(std::string(name) + " must be on the current device");
}

int type_of(const at::Tensor& t, const char* name) {
    if (t.is_cuda()) check_device(t, name);
    if (t.is_cuda()) switch (t.scalar_type()) {
        case at::kFloat: return ADACOMP_FLOAT;
        case at::kBFloat16: return ADACOMP_BFLOAT;
        case at::kHalf: return ADACOMP_HALF;
        default: break;
    }
    throw WrongType(std::string(name) + " must be a float32, bfloat16 or float16 CUDA tensor");
}

template <typename T = void>
T* address(const at::Tensor& t) {
    return static_cast<T*>(t.data_ptr());
}

// A contiguous tensor of one type.
void check(const at::Tensor& t, at::ScalarType type, const char* name) {
    if (t.scalar_type() != type || !t.is_cuda() || !t.is_contiguous())
        throw WrongType(std::string(name) + " must be a contiguous CUDA tensor of " + at::toString(type));
    check_device(t, name);
}

// Address of a nullable contiguous tensor of n elements.
template <typename T = float>
T* optional(PyObject* o, int64_t n, const char* name, at::ScalarType type = at::kFloat) {
    if (o == Py_None) return nullptr;
    const at::Tensor& t = tensor(o, name);
    if (t.numel() != n) throw WrongValue(std::string(name) + " must have " + std::to_string(n) + " elements");
    check(t, type, name);
    return address<T>(t);
}

struct Workspace {
    void* p = nullptr;
    uint64_t bytes = 0;
    explicit Workspace(PyObject* o) {
        if (o == Py_None) return;
        const at::Tensor& t = tensor(o, "ws");
        check(t, at::kByte, "ws");
        p = address(t);
        bytes = uint64_t(t.numel());
    }
};

float real(PyObject* o) {
    const double x = PyFloat_AsDouble(o);
    if (x == -1.0 && PyErr_Occurred()) throw PythonError();
    return float(x);
}
uint64_t whole(PyObject* o) {
    const unsigned long long x = PyLong_AsUnsignedLongLong(o);
    if (x == ~0ull && PyErr_Occurred()) throw PythonError();
    return x;
}
uint32_t whole32(PyObject* o, const char* name) {
    const uint64_t x = whole(o);
    if (x > 0xFFFFFFFFull) throw WrongValue(std::string(name) + " must fit in 32 bits");
    return uint32_t(x);
}
bool truth(PyObject* o) {
    const int x = PyObject_IsTrue(o);
    if (x < 0) throw PythonError();
    return x != 0;
}

// A stream's handle, or the current device's current stream for None.
void* stream_of(PyObject* o) {
    PyObject* handle = nullptr;
    if (o == Py_None) {
        PyObject* index = PyLong_FromLong(here());
        if (index != nullptr) {
            handle = PyObject_CallOneArg(current_stream, index);
            Py_DECREF(index);
        }
    } else {
        handle = PyObject_GetAttrString(o, "cuda_stream");
    }
    if (handle == nullptr) throw PythonError();
    void* p = PyLong_AsVoidPtr(handle);
    Py_DECREF(handle);
    if (p == nullptr && PyErr_Occurred()) throw PythonError();
    return p;
}

// A C call without the interpreter's lock: other threads go on while a launch waits for room in a queue,
// also a host function in that queue that needs the lock.
template <typename F>
int unlocked(F f) {
    PyThreadState* state = PyEval_SaveThread();
    const int status = f();   // the C ABI throws nothing
    PyEval_RestoreThread(state);
    return status;
}

// The gradient of an optimizer call.
struct Gradient {
    int type;
    void* p;
    int64_t n;
    explicit Gradient(PyObject* o) {
        const at::Tensor& t = tensor(o, "grad");
        type = type_of(t, "grad");
        if (!t.is_contiguous()) throw WrongType("grad must be contiguous");
        p = address(t);
        n = t.numel();
    }
};

PyObject* gradient(PyObject* const* a) {
    const Gradient g(a[0]);
    return Py_BuildValue("(iK)", g.type, static_cast<unsigned long long>(reinterpret_cast<uintptr_t>(g.p)));
}

// optimizer, grad, clip, ws, max_norm, scale, stream
int grad_norm(PyObject* const* a) {
    const auto* opt = reinterpret_cast<const adacomp_optimizer*>(whole(a[0]));
    const Gradient g(a[1]);
    float* clip = optional(a[2], 2, "clip");
    const Workspace ws(a[3]);
    const float max_norm = real(a[4]), scale = real(a[5]);
    void* stream = stream_of(a[6]);
    return unlocked([&] {
        return adacomp_grad_norm(opt, g.p, g.type, uint64_t(g.n), max_norm, scale, clip, ws.p, ws.bytes, stream);
    });
}

// optimizer, span, nblocks, weights, grad, m, v, scales (None: float32 moments), lr, beta1, beta2, eps, step, scale,
// seed, clip, weights_bf16, stream
int adamw(PyObject* const* a) {
    const auto* opt = reinterpret_cast<const adacomp_optimizer*>(whole(a[0]));
    const int64_t span = int64_t(whole(a[1])), nblocks = int64_t(whole(a[2]));
    const bool packed = a[7] != Py_None;
    const Gradient g(a[4]);
    const at::Tensor &w = tensor(a[3], "weights"), &m = tensor(a[5], "m"), &v = tensor(a[6], "v");
    check(w, at::kFloat, "weights");
    void* scales = nullptr;
    if (packed) {
        const at::Tensor& s = tensor(a[7], "scales");
        if (s.numel() < 2 * nblocks) throw WrongValue("scales shorter than the optimizer's blocks");
        check(s, at::kByte, "scales");
        scales = address(s);
        for (const at::Tensor* t : {&m, &v}) {
            if ((t->scalar_type() != at::kByte && t->scalar_type() != at::kFloat8_e4m3fn) || !t->is_cuda() ||
                !t->is_contiguous())
                throw WrongType("m and v must be contiguous float8_e4m3fn or uint8 CUDA tensors");
            check_device(*t, "m and v");
        }
    } else {
        check(m, at::kFloat, "m");
        check(v, at::kFloat, "v");
    }
    const uint64_t n = uint64_t(std::min({w.numel(), g.n, m.numel(), v.numel()}));
    void* copy = nullptr;
    if (a[16] != Py_None) {
        const at::Tensor& t = tensor(a[16], "weights_bf16");
        if (t.numel() < span) throw WrongValue("weights_bf16 shorter than the other buffers");
        check(t, at::kBFloat16, "weights_bf16");
        copy = address(t);
    }
    const adacomp_adamw p = {real(a[8]), real(a[9]), real(a[10]), real(a[11]), real(a[13]), whole32(a[12], "step")};
    const float* clip = optional(a[15], 2, "clip");
    const uint32_t seed = whole32(a[14], "seed");
    void* stream = stream_of(a[17]);
    float *wp = address<float>(w), *mp = address<float>(m), *vp = address<float>(v);
    return unlocked([&] {
        return packed ? adacomp_adamw_packed_step(opt, wp, g.p, g.type, mp, vp, scales, copy, n, &p, seed, clip, stream)
                      : adacomp_adamw_step(opt, wp, g.p, g.type, mp, vp, copy, n, &p, clip, stream);
    });
}

// A tensor whose columns are adjacent and whose rows, over all leading axes, lie at one distance.
struct Rows {
    void* p;
    uint64_t stride, rows;
    uint32_t cols;
    int type;
    Rows(const at::Tensor& t, const char* name) {
        type = type_of(t, name);
        if (t.dim() == 0) throw WrongValue(std::string(name) + " must have at least one axis");
        const int64_t n = t.size(-1);
        // more columns than 32 bits hold are more than the C ABI takes, in any number
        cols = uint32_t(std::min<int64_t>(n, 0xFFFFFFFF));
        rows = n ? uint64_t(t.numel() / n) : 0;
        if (t.is_contiguous()) {
            stride = uint64_t(n);
        } else {
            // the leading axes of more than one place, innermost first: each has to go on where the one
            // inside it ends
            bool one = n == 1 || t.stride(-1) == 1;
            int64_t step = -1, next = 0;
            for (int64_t i = t.dim() - 2; i >= 0 && one; --i) {
                if (t.size(i) == 1) continue;
                if (step < 0) step = t.stride(i);
                else one = t.stride(i) == next;
                next = t.stride(i) * t.size(i);
            }
            if (!one) throw WrongType(std::string(name) + " must have adjacent columns and one distance between its rows");
            stride = uint64_t(rows > 1 ? step : n);
        }
        p = address(t);
    }
    Rows(const at::Tensor& t, const char* name, const at::Tensor& like) : Rows(t, name) {
        if (t.sizes() != like.sizes() || t.scalar_type() != like.scalar_type())
            throw WrongValue(std::string(name) + " must have the shape and type of the input");
    }
};

// x, weight, bias, out, mean, rstd, eps, stream
int layer_norm(PyObject* const* a) {
    const at::Tensor& tx = tensor(a[0], "x");
    const Rows x(tx, "x"), y(tensor(a[3], "out"), "out", tx);
    const int64_t rows = int64_t(x.rows);
    const float *weight = optional(a[1], x.cols, "weight"), *bias = optional(a[2], x.cols, "bias");
    float *mean = optional(a[4], rows, "mean"), *rstd = optional(a[5], rows, "rstd");
    const float eps = real(a[6]);
    void* stream = stream_of(a[7]);
    return unlocked([&] {
        return adacomp_layer_norm(x.p, x.stride, weight, bias, y.p, y.stride, mean, rstd, x.rows, x.cols, x.type, eps,
                                  stream);
    });
}

// dy, x, weight, mean, rstd, dx, dweight, dbias, ws, stream
int layer_norm_backward(PyObject* const* a) {
    const at::Tensor& td = tensor(a[0], "dy");
    const Rows dy(td, "dy"), x(tensor(a[1], "x"), "x", td), dx(tensor(a[5], "dx"), "dx", td);
    const int64_t rows = int64_t(dy.rows), cols = dy.cols;
    const Workspace ws(a[8]);
    const float *weight = optional(a[2], cols, "weight"), *mean = optional(a[3], rows, "mean"),
                *rstd = optional(a[4], rows, "rstd");
    float *dweight = optional(a[6], cols, "dweight"), *dbias = optional(a[7], cols, "dbias");
    void* stream = stream_of(a[9]);
    return unlocked([&] {
        return adacomp_layer_norm_backward(dy.p, dy.stride, x.p, x.stride, weight, mean, rstd, dx.p, dx.stride, dweight,
                                           dbias, dy.rows, dy.cols, dy.type, ws.p, ws.bytes, stream);
    });
}

// The gate, whose shape and type the other tensors of a scan have.
struct Gate {
    const at::Tensor& t;
    adacomp_scan_shape shape;
    int64_t states;
    Gate(PyObject* o, bool sigmoid) : t(tensor(o, "gate")) {
        const int type = type_of(t, "gate");
        if (t.dim() != 3) throw WrongValue("gate must be [batch, length, channels]");
        // sizes past 32 bits are past the C ABI's limits, in any number
        auto narrow = [](int64_t n) { return uint32_t(std::min<int64_t>(n, 0xFFFFFFFF)); };
        shape = {uint64_t(t.size(1)), narrow(t.size(0)), narrow(t.size(2)), type, sigmoid ? 1 : 0};
        states = t.size(0) * t.size(2);
    }
};

struct View : adacomp_view {
    View(PyObject* o, const Gate& gate, const char* name) {
        const at::Tensor& t = tensor(o, name);
        if (!t.is_cuda() || t.scalar_type() != gate.t.scalar_type() || t.sizes() != gate.t.sizes())
            throw WrongValue(std::string(name) + " must be a CUDA tensor of the gate's shape and type");
        check_device(t, name);
        const int64_t B = t.size(0), T = t.size(1), D = t.size(2);
        data = address(t);
        if (t.is_contiguous()) {
            batch_stride = uint64_t(T * D);
            time_stride = uint64_t(D);
            return;
        }
        if (D > 1 && t.stride(2) != 1) throw WrongType(std::string(name) + " must have adjacent channels");
        batch_stride = uint64_t(B > 1 ? t.stride(0) : 0);
        time_stride = uint64_t(T > 1 ? t.stride(1) : D);
    }
};

const int32_t* lengths_of(PyObject* o, const Gate& gate) {
    return optional<int32_t>(o, gate.t.size(0), "lengths", at::kInt);
}

// gate, x, h, h0, h_last, lengths, sigmoid, ws, stream
int gated_scan(PyObject* const* a) {
    const Gate gate(a[0], truth(a[6]));
    const View z(a[0], gate, "gate"), x(a[1], gate, "x"), h(a[2], gate, "h");
    const Workspace ws(a[7]);
    const float* h0 = optional(a[3], gate.states, "h0");
    float* last = optional(a[4], gate.states, "h_last");
    const int32_t* lengths = lengths_of(a[5], gate);
    void* stream = stream_of(a[8]);
    return unlocked([&] {
        return adacomp_gated_scan(&gate.shape, &z, &x, &h, h0, last, lengths, ws.p, ws.bytes, stream);
    });
}

// gate, x (or None), h, dh, dgate, dx, h0, dh_last, dh0, lengths, sigmoid, ws, stream
int gated_scan_backward(PyObject* const* a) {
    const Gate gate(a[0], truth(a[10]));
    const View z(a[0], gate, "gate"), x(a[1] == Py_None ? a[0] : a[1], gate, "x"), h(a[2], gate, "h"),
        dh(a[3], gate, "dh"), dz(a[4], gate, "dgate"), dx(a[5], gate, "dx");
    const Workspace ws(a[11]);
    const bool with_x = a[1] != Py_None;
    const float *h0 = optional(a[6], gate.states, "h0"), *dh_last = optional(a[7], gate.states, "dh_last");
    float* dh0 = optional(a[8], gate.states, "dh0");
    const int32_t* lengths = lengths_of(a[9], gate);
    void* stream = stream_of(a[12]);
    return unlocked([&] {
        return adacomp_gated_scan_backward(&gate.shape, &z, with_x ? &x : nullptr, &h, &dh, &dz, &dx, h0, dh_last, dh0,
                                           lengths, ws.p, ws.bytes, stream);
    });
}

// No C++ exception leaves an entry point.
template <typename F>
PyObject* guarded(Py_ssize_t n, Py_ssize_t want, F f) {
    device = -1;
    try {
        if (n != want) throw WrongType("wrong number of arguments");
        return f();
    } catch (const WrongType& e) {
        PyErr_SetString(PyExc_TypeError, e.what());
    } catch (const WrongValue& e) {
        PyErr_SetString(PyExc_ValueError, e.what());
    } catch (const PythonError&) {
    } catch (const std::exception& e) {
        PyErr_SetString(PyExc_RuntimeError, e.what());
    } catch (...) {
        PyErr_SetString(PyExc_RuntimeError, "unknown C++ exception");
    }
    return nullptr;
}

template <int (*F)(PyObject* const*), int N>
PyObject* entry(PyObject*, PyObject* const* a, Py_ssize_t n) {
    return guarded(n, N, [&] { return PyLong_FromLong(F(a)); });
}
PyObject* gradient_entry(PyObject*, PyObject* const* a, Py_ssize_t n) {
    return guarded(n, 1, [&] { return gradient(a); });
}

#define ENTRY(name, f) {name, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(f)), METH_FASTCALL, nullptr}
PyMethodDef methods[] = {
    ENTRY("gradient", gradient_entry),
    ENTRY("grad_norm", (entry<grad_norm, 7>)),
    ENTRY("adamw", (entry<adamw, 18>)),
    ENTRY("layer_norm", (entry<layer_norm, 8>)),
    ENTRY("layer_norm_backward", (entry<layer_norm_backward, 10>)),
    ENTRY("gated_scan", (entry<gated_scan, 9>)),
    ENTRY("gated_scan_backward", (entry<gated_scan_backward, 13>)),
    {nullptr, nullptr, 0, nullptr}};

PyModuleDef module = {PyModuleDef_HEAD_INIT, "_binding", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__binding() {
    PyObject* c = PyImport_ImportModule("torch._C");
    if (c == nullptr) return nullptr;
    current_device = PyObject_GetAttrString(c, "_cuda_getDevice");
    if (current_device != nullptr) current_stream = PyObject_GetAttrString(c, "_cuda_getCurrentRawStream");
    Py_DECREF(c);
    return current_stream == nullptr ? nullptr : PyModule_Create(&module);
}
