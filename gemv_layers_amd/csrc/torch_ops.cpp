// PyTorch marshalling of the 8-bit and training calls, as a CPython module (_torch_ops): checks the
// tensors, makes the outputs, and calls the C ABI on their addresses and the device's current stream.
// No arithmetic, and no tensor is kept. It is C++ because a small product takes the GPU 5 us: the
// same steps in Python take the host 5 us on top of the launch, these 1.5.
//
// The C ABI's functions come in by address (bind), so that this module links to PyTorch alone. A call
// runs with its tensors' device as the current one, as the library asks.

#include <Python.h>

#include <ATen/ops/empty.h>
#include <c10/core/DeviceGuard.h>
#include <c10/core/GradMode.h>
#include <c10/hip/HIPStream.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include <exception>

#include "gemm_bf16.h"

namespace {

struct Abi {
    decltype(&gemm_i8_quantize) quantize;
    decltype(&gemm_i8) i8, i8_swiglu;
    decltype(&gemm_i8_bf16) i8_bf16, i8_swiglu_bf16;
    decltype(&gemm_bf16_bwd) bwd;
    decltype(&gemm_bf16_swiglu_train) train;
    decltype(&gemm_bf16_swiglu_bwd) swiglu_bwd;
} abi;
PyObject* on_error = nullptr;  // called with (function, status); raises

// thrown with a Python error set
struct Failed {};

[[noreturn]] void fail(PyObject* type, const char* format, ...) {
    va_list args;
    va_start(args, format);
    PyErr_FormatV(type, format, args);
    va_end(args);
    throw Failed();
}

const at::Tensor& tensor(PyObject* o, const char* name) {
    if (!THPVariable_Check(o)) fail(PyExc_TypeError, "%s must be a tensor", name);
    return THPVariable_Unpack(o);
}

const char* type_name(at::ScalarType t) {
    switch (t) {
        case at::kBFloat16: return "torch.bfloat16";
        case at::kChar: return "torch.int8";
        case at::kFloat: return "torch.float32";
        default: return "torch.uint8";
    }
}

// The calls record no graph. Their results' gradients would be lost without a word where autograd is to
// follow them: refused, as PyTorch refuses out=.
void no_graph(const at::Tensor& t, const char* name) {
    if (c10::GradMode::is_enabled() && t.requires_grad())
        fail(PyExc_RuntimeError,
             "%s requires grad, and this call records no graph: use it in a torch.autograd.Function or under "
             "torch.no_grad(), or detach %s",
             name, name);
}

struct Rows {
    int64_t rows, cols, ld;
    void* p;
};

// a 2-D device tensor with unit column stride and rows that do not overlap; -1: any size. `codes_only`:
// the call's results are codes and their scales, which have no gradient.
Rows rows_of(const at::Tensor& t, const char* name, at::ScalarType type, int64_t rows = -1, int64_t cols = -1,
             int device = -1, bool codes_only = false) {
    if (t.scalar_type() != type) fail(PyExc_TypeError, "%s must be %s", name, type_name(type));
    if (t.dim() != 2) fail(PyExc_ValueError, "%s must have two dimensions, not %lld", name, (long long)t.dim());
    Rows r{t.size(0), t.size(1), t.stride(0), nullptr};
    if ((rows >= 0 && r.rows != rows) || (cols >= 0 && r.cols != cols))
        fail(PyExc_ValueError, "%s must be %lld x %lld (-1: any), not %lld x %lld", name, (long long)rows,
             (long long)cols, (long long)r.rows, (long long)r.cols);
    if (!codes_only) no_graph(t, name);
    if (!t.is_cuda()) fail(PyExc_ValueError, "%s must be a device tensor", name);
    if (device >= 0 && t.get_device() != device) fail(PyExc_ValueError, "all tensors must be on one device");
    if (t.stride(1) != 1 && r.cols > 1 && r.rows > 0) fail(PyExc_ValueError, "%s needs unit column stride", name);
    if (r.ld < r.cols) {
        if (r.rows > 1) fail(PyExc_ValueError, "%s has overlapping rows", name);
        r.ld = r.cols;
    }
    r.p = t.data_ptr();
    return r;
}

const float* scales_of(const at::Tensor& t, const char* name, int64_t n, int device) {
    if (t.scalar_type() != at::kFloat || t.dim() != 1 || t.size(0) != n || !t.is_cuda())
        fail(PyExc_ValueError, "%s must be a device vector of %lld float32 values", name, (long long)n);
    no_graph(t, name);
    if (t.get_device() != device) fail(PyExc_ValueError, "all tensors must be on one device");
    if (n > 1 && t.stride(0) != 1) fail(PyExc_ValueError, "%s needs unit stride", name);
    return static_cast<const float*>(t.data_ptr());
}

at::Tensor make(const at::Tensor& like, at::ScalarType type, int64_t rows, int64_t cols) {
    return at::empty({rows, cols}, like.options().dtype(type).requires_grad(false).memory_format(std::nullopt));
}

// a handle as an integer or a ctypes pointer
gemm_stream_t handle_of(PyObject* o) {
    if (PyLong_Check(o)) {
        void* p = PyLong_AsVoidPtr(o);
        if (PyErr_Occurred()) throw Failed();
        return static_cast<gemm_stream_t>(p);
    }
    PyObject* v = PyObject_GetAttrString(o, "value");
    if (!v) throw Failed();
    void* p = v == Py_None ? nullptr : PyLong_AsVoidPtr(v);
    Py_DECREF(v);
    if (PyErr_Occurred()) throw Failed();
    return static_cast<gemm_stream_t>(p);
}

// Where a call runs: on the tensors' device and, None, its current stream, else the given one, which is
// the current one meanwhile. So outputs and work buffers come from the memory of the stream that uses
// them: memory of another stream could still be in use there, and be given out again when a work buffer
// is dropped at the end of the call.
class Place {
    const c10::DeviceGuard guard;
    const c10::hip::HIPStream before;
    bool moved = false;

public:
    gemm_stream_t stream;
    Place(PyObject* o, const at::Tensor& t)
        : guard(t.device()), before(c10::hip::getCurrentHIPStream(t.get_device())), stream(before.stream()) {
        if (o == Py_None) return;
        const gemm_stream_t s = handle_of(o);
        if (s == stream) return;
        c10::hip::setCurrentHIPStream(c10::hip::getStreamFromExternal(static_cast<hipStream_t>(s), t.get_device()));
        stream = s;
        moved = true;
    }
    ~Place() {
        if (moved) c10::hip::setCurrentHIPStream(before);
    }
    Place(const Place&) = delete;
    Place& operator=(const Place&) = delete;
};

void check(const char* name, int status) {
    if (status == GEMM_OK) return;
    PyObject* r = PyObject_CallFunction(on_error, "si", name, status);
    Py_XDECREF(r);
    if (!PyErr_Occurred()) PyErr_SetString(PyExc_RuntimeError, name);
    throw Failed();
}

// calls the library without the interpreter's lock (a launch may wait for room in the queue)
template <class F>
int unlocked(F f) {
    PyThreadState* s = PyEval_SaveThread();
    const int status = f();
    PyEval_RestoreThread(s);
    return status;
}

PyObject* wrap(at::Tensor t) {
    PyObject* o = THPVariable_Wrap(std::move(t));
    if (!o) throw Failed();
    return o;
}

PyObject* pack(std::initializer_list<PyObject*> items) {  // takes the references
    PyObject* t = PyTuple_New((Py_ssize_t)items.size());
    Py_ssize_t i = 0;
    for (PyObject* o : items) PyTuple_SET_ITEM(t, i++, o);
    return t;
}
PyObject* none() { return Py_NewRef(Py_None); }

bool truth(PyObject* o) {
    const int v = PyObject_IsTrue(o);
    if (v < 0) throw Failed();
    return v != 0;
}

// a call's Python face: `want` positional arguments, C++ exceptions turned into the Python ones that
// PyTorch's own functions raise for them (torch.OutOfMemoryError among them)
template <PyObject* (*F)(PyObject* const*), Py_ssize_t want>
PyObject* entry(PyObject*, PyObject* const* a, Py_ssize_t n) {
    try {
        if (n != want) fail(PyExc_TypeError, "%zd arguments wanted", want);
        return F(a);
    } catch (const Failed&) {
        return nullptr;
    } catch (...) {
        torch::translate_exception_to_python(std::current_exception());
        return nullptr;
    }
}

// the M x N output: the one given, or a new one
at::Tensor output(PyObject* out, const at::Tensor& like, int64_t M, int64_t N, int device, Rows* r) {
    at::Tensor t = out == Py_None ? make(like, at::kBFloat16, M, N) : tensor(out, "out");
    *r = rows_of(t, "out", at::kBFloat16, M, N, device);
    return t;
}

// (X, stream) -> (Q, S)
PyObject* quantize(PyObject* const* a) {
    const at::Tensor& X = tensor(a[0], "X");
    const Rows x = rows_of(X, "X", at::kBFloat16, -1, -1, -1, true);
    const Place at(a[1], X);
    const int64_t ldq = (x.cols + 15) / 16 * 16;
    at::Tensor Q = make(X, at::kChar, x.rows, ldq);
    at::Tensor S = at::empty({x.rows}, X.options().dtype(at::kFloat).requires_grad(false).memory_format(std::nullopt));
    check("gemm_i8_quantize", unlocked([&] {
              return abi.quantize(x.rows, x.cols, x.p, x.ld, Q.data_ptr(), ldq, static_cast<float*>(S.data_ptr()),
                                  at.stream);
          }));
    if (ldq != x.cols) Q = Q.narrow(1, 0, x.cols);
    PyObject* q = wrap(std::move(Q));
    return pack({q, wrap(std::move(S))});
}

// an 8-bit weight: N outputs (2N rows when gated), codes and scales
struct Weight {
    int64_t N;
    Rows w;
    const float* scales;
};
Weight weight_of(PyObject* wq, PyObject* sw, int64_t K, bool glu, int device) {
    Weight r;
    r.w = rows_of(tensor(wq, "Wq"), "Wq", at::kChar, -1, K, device);
    if (glu && r.w.rows % 2) fail(PyExc_ValueError, "Wq must have 2N rows, gate then up");
    r.N = glu ? r.w.rows / 2 : r.w.rows;
    r.scales = scales_of(tensor(sw, "Sw"), "Sw", r.w.rows, device);
    return r;
}

// (Aq, Sa, Wq, Sw, out, stream, glu) -> C
PyObject* i8(PyObject* const* a) {
    const bool glu = truth(a[6]);
    const at::Tensor& A = tensor(a[0], "Aq");
    const Rows q = rows_of(A, "Aq", at::kChar);
    const int device = A.get_device();
    const Weight w = weight_of(a[2], a[3], q.cols, glu, device);
    const float* sa = scales_of(tensor(a[1], "Sa"), "Sa", q.rows, device);
    const Place at(a[5], A);
    Rows c;
    at::Tensor C = output(a[4], A, q.rows, w.N, device, &c);
    check(glu ? "gemm_i8_swiglu" : "gemm_i8", unlocked([&] {
              return (glu ? abi.i8_swiglu : abi.i8)(q.rows, w.N, q.cols, q.p, q.ld, sa, w.w.p, w.w.ld, w.scales,
                                                c.p, c.ld, at.stream);
          }));
    return wrap(std::move(C));
}

// (A, Wq, Sw, out, work, stream, glu) -> C
PyObject* i8_dynamic(PyObject* const* a) {
    const bool glu = truth(a[6]);
    const at::Tensor& A = tensor(a[0], "A");
    const Rows x = rows_of(A, "A", at::kBFloat16);
    const int device = A.get_device();
    const Weight w = weight_of(a[1], a[2], x.cols, glu, device);
    const Place at(a[5], A);
    Rows c;
    at::Tensor C = output(a[3], A, x.rows, w.N, device, &c);
    at::Tensor work;
    if (a[4] == Py_None) {  // gemm_i8_work_bytes
        work = at::empty({x.rows * ((x.cols + 15) / 16 * 16 + 4)},
                         A.options().dtype(at::kByte).requires_grad(false).memory_format(std::nullopt));
    } else {
        work = tensor(a[4], "work");
        if (work.scalar_type() != at::kByte || !work.is_contiguous() || !work.is_cuda() || work.get_device() != device)
            fail(PyExc_ValueError, "work must be a contiguous uint8 tensor on the same device");
    }
    check(glu ? "gemm_i8_swiglu_bf16" : "gemm_i8_bf16", unlocked([&] {
              return (glu ? abi.i8_swiglu_bf16 : abi.i8_bf16)(x.rows, w.N, x.cols, x.p, x.ld, w.w.p, w.w.ld, w.scales,
                                                              c.p, c.ld, work.data_ptr(), work.numel(), at.stream);
          }));
    return wrap(std::move(C));
}

// the operands that both backward passes share: A (M x K), B (K x W), dC
struct Operands {
    Rows a, b;
    int device;
    at::Tensor dA, dB;
    void *da = nullptr, *db = nullptr;
    Operands(const at::Tensor& A, const at::Tensor& B) : a(rows_of(A, "A", at::kBFloat16)), device(A.get_device()) {
        b = rows_of(B, "B", at::kBFloat16, a.cols, -1, device);
    }
    void gradients(const at::Tensor& A, bool need_a, bool need_b) {
        if (need_a) da = (dA = make(A, at::kBFloat16, a.rows, a.cols)).data_ptr();
        if (need_b) db = (dB = make(A, at::kBFloat16, b.rows, b.cols)).data_ptr();
    }
    PyObject* grad_a() { return dA.defined() ? wrap(std::move(dA)) : none(); }
    PyObject* grad_b() { return dB.defined() ? wrap(std::move(dB)) : none(); }
};

// (dC, A, B, need_dA, need_dB, stream) -> (dA, dB)
PyObject* bwd(PyObject* const* a) {
    const at::Tensor& A = tensor(a[1], "A");
    Operands o(A, tensor(a[2], "B"));
    const Rows d = rows_of(tensor(a[0], "dC"), "dC", at::kBFloat16, o.a.rows, o.b.cols, o.device);
    const Place at(a[5], A);
    o.gradients(A, truth(a[3]), truth(a[4]));
    check("gemm_bf16_bwd", unlocked([&] {
              return abi.bwd(o.a.rows, o.b.cols, o.a.cols, d.p, d.ld, o.a.p, o.a.ld, o.b.p, o.b.ld, o.da, o.a.cols, o.db,
                             o.b.cols, at.stream);
          }));
    PyObject* ga = o.grad_a();
    return pack({ga, o.grad_b()});
}

// (A, B, stream) -> (C, GU)
PyObject* train(PyObject* const* a) {
    const at::Tensor& A = tensor(a[0], "A");
    const Operands o(A, tensor(a[1], "B"));
    if (o.b.cols % 2) fail(PyExc_ValueError, "B must be K x 2N, gate then up");
    const int64_t N = o.b.cols / 2;
    const Place at(a[2], A);
    at::Tensor C = make(A, at::kBFloat16, o.a.rows, N), GU = make(A, at::kBFloat16, o.a.rows, 2 * N);
    check("gemm_bf16_swiglu_train", unlocked([&] {
              return abi.train(o.a.rows, N, o.a.cols, o.a.p, o.a.ld, o.b.p, o.b.ld, GU.data_ptr(), 2 * N,
                               C.data_ptr(), N, at.stream);
          }));
    PyObject* c = wrap(std::move(C));
    return pack({c, wrap(std::move(GU))});
}

// (dC, GU, A, B, need_dA, need_dB, inplace, stream) -> (dA, dB, dGU)
PyObject* swiglu_bwd(PyObject* const* a) {
    const at::Tensor &GU = tensor(a[1], "GU"), &A = tensor(a[2], "A");
    Operands o(A, tensor(a[3], "B"));
    if (o.b.cols % 2) fail(PyExc_ValueError, "B must be K x 2N, gate then up");
    const int64_t N = o.b.cols / 2;
    const Rows d = rows_of(tensor(a[0], "dC"), "dC", at::kBFloat16, o.a.rows, N, o.device);
    const Rows gu = rows_of(GU, "GU", at::kBFloat16, o.a.rows, 2 * N, o.device);
    const Place at(a[7], A);
    o.gradients(A, truth(a[4]), truth(a[5]));
    const bool inplace = truth(a[6]);
    at::Tensor dGU = inplace ? GU : make(A, at::kBFloat16, o.a.rows, 2 * N);
    check("gemm_bf16_swiglu_bwd", unlocked([&] {
              return abi.swiglu_bwd(o.a.rows, N, o.a.cols, d.p, d.ld, gu.p, gu.ld, o.a.p, o.a.ld, o.b.p, o.b.ld,
                                    dGU.data_ptr(), inplace ? gu.ld : 2 * N, o.da, o.a.cols, o.db, o.b.cols, at.stream);
          }));
    PyObject* ga = o.grad_a();
    PyObject* gb = o.grad_b();
    return pack({ga, gb, wrap(std::move(dGU))});
}

// (on_error, address of each function of Abi in its order)
PyObject* bind(PyObject* const* a) {
    void* at[8];
    for (int i = 0; i < 8; ++i) {
        at[i] = PyLong_AsVoidPtr(a[1 + i]);
        if (PyErr_Occurred()) throw Failed();
    }
    static_assert(sizeof(Abi) == sizeof(at), "one address each");
    memcpy(&abi, at, sizeof at);
    Py_XSETREF(on_error, Py_NewRef(a[0]));
    return none();
}

#define CALL(name, want) {#name, reinterpret_cast<PyCFunction>(reinterpret_cast<void*>(entry<name, want>)), METH_FASTCALL, nullptr}
PyMethodDef methods[] = {CALL(bind, 9),  CALL(quantize, 2), CALL(i8, 7),         CALL(i8_dynamic, 7),
                         CALL(bwd, 6),   CALL(train, 3),    CALL(swiglu_bwd, 8), {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_torch_ops", "Tensor marshalling of the 8-bit and training calls.", -1,
                      methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__torch_ops() { return PyModule_Create(&module); }
