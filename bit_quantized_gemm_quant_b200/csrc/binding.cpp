// binding.cpp -- CPython marshalling of the products with an epilogue and their
// gradients: argument checks, outputs and workspace from PyTorch's allocator, one call of
// the C ABI on the current stream.
//
// A decode call runs 4 to 10 microseconds on the GPU; marshalled through ctypes it took 13
// on the host (a gradient 25), most of it in Python attribute reads, argument conversion
// and tensor creation.  Errors are those of the Python layer: TypeError, ValueError,
// BqError with the library's status, and PyTorch's own (OutOfMemoryError) as PyTorch raises them.
#define PY_SSIZE_T_CLEAN
#include <Python.h>

#include <ATen/core/Tensor.h>
#include <ATen/ops/empty.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include <exception>
#include <initializer_list>

#include "bqgemm.h"

namespace {

PyObject* g_error = nullptr;            // BqError

struct Raised {};                       // a Python exception is set

using Types = std::initializer_list<at::ScalarType>;
const Types kBf16Bits = {at::kBFloat16, at::kShort, at::kUInt16};
const Types kBits16 = {at::kBFloat16, at::kHalf, at::kShort, at::kUInt16};
const Types kBytes = {at::kByte, at::kChar};
const Types kWords = {at::kInt, at::kUInt32};

constexpr uintptr_t kEmptyTag = 16;     // non-NULL, aligned, never dereferenced (empty tensor)

[[noreturn]] void raise(PyObject* type, const char* fmt, const char* a, const char* b = "")
{
    PyErr_Format(type, fmt, a, b);
    throw Raised{};
}

// The tensor of an argument, NULL for None.
const at::Tensor* tensor(PyObject* o, const char* name)
{
    if (o == Py_None) return nullptr;
    if (!THPVariable_Check(o)) raise(PyExc_TypeError, "%s: expected a tensor, got %s", name, Py_TYPE(o)->tp_name);
    return &THPVariable_Unpack(o);
}

const at::Tensor& needed(PyObject* o, const char* name)
{
    const at::Tensor* t = tensor(o, name);
    if (!t) raise(PyExc_TypeError, "%s: expected a tensor, got None%s", name);
    return *t;
}

template <typename T = void>
T* address(const at::Tensor& t)
{
    void* p = t.data_ptr();
    return reinterpret_cast<T*>(p ? p : reinterpret_cast<void*>(kEmptyTag));
}

// One call's device and the check that every operand meets: type, exact shape, device,
// contiguous.
struct Call {
    c10::Device dev;

    template <typename T = uint16_t>
    T* operand(const at::Tensor* t, Types types, at::IntArrayRef shape, const char* name) const
    {
        if (!t) return nullptr;
        bool type_ok = false;
        for (at::ScalarType s : types) type_ok = type_ok || t->scalar_type() == s;
        if (!type_ok) {
            std::string want;
            for (at::ScalarType s : types) want += std::string(want.empty() ? "" : " or ") + c10::toString(s);
            PyErr_Format(PyExc_TypeError, "%s: expected %s, got %s", name, want.c_str(), c10::toString(t->scalar_type()));
            throw Raised{};
        }
        if (t->sizes() != shape) {
            std::ostringstream m;
            m << name << ": shape " << t->sizes() << ", the call needs " << shape;
            PyErr_SetString(PyExc_ValueError, m.str().c_str());
            throw Raised{};
        }
        if (t->device() != dev)
            raise(PyExc_ValueError, "%s: on %s, not on the call's device", name, t->device().str().c_str());
        if (!t->is_contiguous()) raise(PyExc_ValueError, "%s: tensors must be contiguous%s", name);
        return address<T>(*t);
    }

    at::Tensor make(at::IntArrayRef shape, at::ScalarType type = at::kBFloat16) const
    {
        return at::empty(shape, at::TensorOptions().dtype(type).device(dev));
    }

    bq_stream_t stream() const { return c10::cuda::getCurrentCUDAStream(dev.index()).stream(); }
};

// `out` given by the caller and one of the call's inputs: shared memory would be written while
// other CTAs still read it.
void apart(const at::Tensor* out, const at::Tensor* in, const char* name)
{
    if (!out || !in || out->nbytes() == 0 || in->nbytes() == 0) return;
    const char *o = static_cast<const char*>(out->data_ptr()), *i = static_cast<const char*>(in->data_ptr());
    if (o < i + in->nbytes() && i < o + out->nbytes()) raise(PyExc_ValueError, "out: shares memory with %s%s", name);
}

Call on(const at::Tensor& t, const char* name)
{
    if (!t.is_cuda()) raise(PyExc_ValueError, "%s: tensors must live on a CUDA device%s", name);
    if (t.dim() != 2) raise(PyExc_ValueError, "%s: expected a matrix%s", name);
    return Call{t.device()};
}

struct Matrix {
    const void *wq, *scales, *biases;
};

// (wq, scales, biases | None) with W [N][K].
Matrix matrix(const Call& c, const at::Tensor& wq, const at::Tensor& scales, const at::Tensor* biases, int64_t N,
              int64_t K, int gs, int bits, const char* nq, const char* ns, const char* nb)
{
    if (!biases)
        return {c.operand<void>(&wq, kBytes, {N, K / 2}, nq), c.operand<void>(&scales, kBits16, {N, K / 32}, ns), nullptr};
    const int64_t groups = K / (gs > 0 ? gs : 1);
    return {c.operand<void>(&wq, kWords, {N, K * bits / 32}, nq), c.operand<void>(&scales, kBf16Bits, {N, groups}, ns),
            c.operand<void>(biases, kBf16Bits, {N, groups}, nb)};
}

// Columns of W from its codes.
int64_t columns(const at::Tensor& wq, const at::Tensor* biases, int bits, const char* name)
{
    if (wq.dim() != 2) raise(PyExc_ValueError, "%s: expected a matrix%s", name);
    return biases ? wq.size(1) * 32 / (bits > 0 ? bits : 1) : wq.size(1) * 2;
}

struct Scratch {
    at::Tensor keep;
    void* ptr = nullptr;
    size_t bytes = 0;
    Scratch(const Call& c, int op, int64_t M, int64_t N, int64_t K, int gs, int bits)
        : bytes(quant_matmul_epilogue_workspace_size(op, M, N, K, gs, bits))
    {
        if (bytes == 0) return;
        keep = c.make({(int64_t)bytes}, at::kByte);
        ptr = keep.data_ptr();
    }
};

void check(bq_status s, const char* where)
{
    if (s == BQ_OK) return;
    PyObject* e = PyObject_CallFunction(g_error, "is", (int)s, where);
    if (e) {
        PyErr_SetObject(g_error, e);
        Py_DECREF(e);
    }
    throw Raised{};
}

PyObject* wrap(std::initializer_list<const at::Tensor*> ts)
{
    PyObject* out = PyTuple_New((Py_ssize_t)ts.size());
    if (!out) throw Raised{};
    Py_ssize_t i = 0;
    for (const at::Tensor* t : ts) {
        PyObject* o = THPVariable_Wrap(*t);
        if (!o) {
            Py_DECREF(out);
            throw Raised{};
        }
        PyTuple_SET_ITEM(out, i++, o);
    }
    return out;
}

int integer(PyObject* o)
{
    const long v = PyLong_AsLong(o);
    if (v == -1 && PyErr_Occurred()) throw Raised{};
    if (v < INT32_MIN || v > INT32_MAX) raise(PyExc_ValueError, "an integer argument is out of range%s%s", "");
    return (int)v;
}

bool truth(PyObject* o)
{
    const int v = PyObject_IsTrue(o);
    if (v < 0) throw Raised{};
    return v != 0;
}

// No C++ exception leaves a call.
template <typename F>
PyObject* guarded(Py_ssize_t got, Py_ssize_t want, F&& f)
{
    if (got != want) {
        PyErr_Format(PyExc_TypeError, "expected %zd arguments, got %zd", want, got);
        return nullptr;
    }
    try {
        return f();
    } catch (const Raised&) {
        return nullptr;
    } catch (const std::exception&) {
        torch::translate_exception_to_python(std::current_exception());
    } catch (...) {
        PyErr_SetString(PyExc_RuntimeError, "unknown error");
    }
    return nullptr;
}

// act(x, wq, scales, biases, out_bias, act, residual, group_size, bits, save, out)
PyObject* py_act(PyObject*, PyObject* const* a, Py_ssize_t n)
{
    return guarded(n, 11, [&] {
        const at::Tensor &x = needed(a[0], "x"), &wq = needed(a[1], "w.wq"), &sc = needed(a[2], "w.scales");
        const at::Tensor *bi = tensor(a[3], "w.biases"), *ob = tensor(a[4], "out_bias"), *res = tensor(a[6], "residual"),
                         *given = tensor(a[10], "out");
        const int act = integer(a[5]), gs = integer(a[7]), bits = integer(a[8]);
        const bool save = truth(a[9]);
        const Call c = on(x, "x");
        const int64_t M = x.size(0), K = x.size(1), N = wq.dim() == 2 ? wq.size(0) : 0;
        const c10::cuda::CUDAGuard guard(c.dev);
        const Matrix w = matrix(c, wq, sc, bi, N, K, gs, bits, "w.wq", "w.scales", "w.biases");
        const uint16_t* xp = c.operand(&x, kBf16Bits, {M, K}, "x");
        const uint16_t* bp = c.operand(ob, kBf16Bits, {N}, "out_bias");
        const uint16_t* rp = c.operand(res, kBf16Bits, {M, N}, "residual");
        uint16_t* gp = c.operand(given, kBf16Bits, {M, N}, "out");
        apart(given, &x, "x");
        apart(given, &wq, "w.wq");
        apart(given, &sc, "w.scales");
        apart(given, bi, "w.biases");
        apart(given, ob, "out_bias");
        if (rp != gp) apart(given, res, "residual");          // the residual itself: each element is read, then written
        const at::Tensor y = given ? *given : c.make({M, N}), z = save ? c.make({M, N}) : at::Tensor();
        const Scratch s(c, BQ_OP_ACT, M, N, K, gs, bits);
        check(quant_matmul_act(xp, w.wq, w.scales, w.biases, bp, rp, act, given ? gp : address<uint16_t>(y),
                               save ? address<uint16_t>(z) : nullptr, M, N, K, gs, bits, s.ptr, s.bytes, c.stream()),
              "quant_matmul_act");
        if (save) return wrap({&y, &z});
        if (given) {
            Py_INCREF(a[10]);
            return a[10];
        }
        return THPVariable_Wrap(y);
    });
}

// act_backward(dy, wq, scales, biases, preact, act, group_size, bits, need_dbias)
PyObject* py_act_backward(PyObject*, PyObject* const* a, Py_ssize_t n)
{
    return guarded(n, 9, [&] {
        const at::Tensor &dy = needed(a[0], "dy"), &wq = needed(a[1], "w.wq"), &sc = needed(a[2], "w.scales");
        const at::Tensor *bi = tensor(a[3], "w.biases"), *pre = tensor(a[4], "preact");
        const int act = integer(a[5]), gs = integer(a[6]), bits = integer(a[7]);
        const bool need = truth(a[8]);
        const Call c = on(dy, "dy");
        const int64_t M = dy.size(0), N = dy.size(1), K = columns(wq, bi, bits, "w.wq");
        const c10::cuda::CUDAGuard guard(c.dev);
        const Matrix w = matrix(c, wq, sc, bi, N, K, gs, bits, "w.wq", "w.scales", "w.biases");
        const uint16_t* dyp = c.operand(&dy, kBf16Bits, {M, N}, "dy");
        const uint16_t* pp = c.operand(pre, kBf16Bits, {M, N}, "preact");
        const at::Tensor dx = c.make({M, K}), dz = act == BQ_ACT_NONE ? dy : c.make({M, N}),
                         db = need ? c.make({N}) : at::Tensor();
        const Scratch s(c, BQ_OP_ACT_BACKWARD, M, N, K, gs, bits);
        check(quant_matmul_act_backward(dyp, pp, w.wq, w.scales, w.biases, act, address<uint16_t>(dx),
                                        act == BQ_ACT_NONE ? nullptr : address<uint16_t>(dz),
                                        need ? address<uint16_t>(db) : nullptr, M, N, K, gs, bits, s.ptr, s.bytes,
                                        c.stream()),
              "quant_matmul_act_backward");
        return need ? wrap({&dx, &dz, &db}) : wrap({&dx, &dz});
    });
}

// Gate and up matrices of one format from (wq, scales, biases | None) sequences a[0], a[1].
struct Gated {
    const void *wq[2], *scales[2], *biases[2];
    bool affine;
};

struct Triple {
    PyObject* seq;
    explicit Triple(PyObject* o, const char* name) : seq(PySequence_Fast(o, "expected (wq, scales, biases | None)"))
    {
        if (!seq) throw Raised{};
        if (PySequence_Fast_GET_SIZE(seq) != 3) {
            Py_DECREF(seq);
            raise(PyExc_ValueError, "%s: expected (wq, scales, biases | None)%s", name);
        }
    }
    Triple(const Triple&) = delete;
    ~Triple() { Py_DECREF(seq); }
    PyObject* at(int i) const { return PySequence_Fast_GET_ITEM(seq, i); }
};

Gated gated(const Call& c, const Triple& g, const Triple& u, int64_t N, int64_t K, int gs, int bits)
{
    const at::Tensor *gb = tensor(g.at(2), "gate.biases"), *ub = tensor(u.at(2), "up.biases");
    if (!gb != !ub)
        raise(PyExc_ValueError, "gate and up must both be Q4_0 (biases None) or both be affine%s%s", "");
    const Matrix m0 = matrix(c, needed(g.at(0), "gate.wq"), needed(g.at(1), "gate.scales"), gb, N, K, gs, bits, "gate.wq",
                             "gate.scales", "gate.biases");
    const Matrix m1 = matrix(c, needed(u.at(0), "up.wq"), needed(u.at(1), "up.scales"), ub, N, K, gs, bits, "up.wq",
                             "up.scales", "up.biases");
    return {{m0.wq, m1.wq}, {m0.scales, m1.scales}, {m0.biases, m1.biases}, gb != nullptr};
}

// glu(x, gate, up, gate_bias, up_bias, act, group_size, bits, save, out)
PyObject* py_glu(PyObject*, PyObject* const* a, Py_ssize_t n)
{
    return guarded(n, 10, [&] {
        const at::Tensor& x = needed(a[0], "x");
        const Triple gt(a[1], "gate"), ut(a[2], "up");
        const at::Tensor *gb = tensor(a[3], "gate_bias"), *ub = tensor(a[4], "up_bias"), *given = tensor(a[9], "out");
        const int act = integer(a[5]), gs = integer(a[6]), bits = integer(a[7]);
        const bool save = truth(a[8]);
        const Call c = on(x, "x");
        const at::Tensor& gq = needed(gt.at(0), "gate.wq");
        const int64_t M = x.size(0), K = x.size(1), N = gq.dim() == 2 ? gq.size(0) : 0;
        const c10::cuda::CUDAGuard guard(c.dev);
        const Gated w = gated(c, gt, ut, N, K, gs, bits);
        const uint16_t* xp = c.operand(&x, kBf16Bits, {M, K}, "x");
        const uint16_t* gbp = c.operand(gb, kBf16Bits, {N}, "gate_bias");
        const uint16_t* ubp = c.operand(ub, kBf16Bits, {N}, "up_bias");
        uint16_t* op = c.operand(given, kBf16Bits, {M, N}, "out");
        apart(given, &x, "x");
        for (const Triple* t : {&gt, &ut})
            for (int i = 0; i < 3; ++i) apart(given, tensor(t->at(i), ""), t == &gt ? "gate" : "up");
        apart(given, gb, "gate_bias");
        apart(given, ub, "up_bias");
        const at::Tensor h = given ? *given : c.make({M, N}), g = save ? c.make({M, N}) : at::Tensor(),
                         u = save ? c.make({M, N}) : at::Tensor();
        const Scratch s(c, BQ_OP_GLU, M, N, K, gs, bits);
        check(quant_matmul_glu(xp, w.wq, w.scales, w.affine ? w.biases : nullptr, gbp, ubp, act,
                               given ? op : address<uint16_t>(h), save ? address<uint16_t>(g) : nullptr,
                               save ? address<uint16_t>(u) : nullptr, M, N, K, gs, bits, s.ptr, s.bytes, c.stream()),
              "quant_matmul_glu");
        if (save) return wrap({&h, &g, &u});
        if (given) {
            Py_INCREF(a[9]);
            return a[9];
        }
        return THPVariable_Wrap(h);
    });
}

// glu_backward(dh, g, u, gate, up, act, group_size, bits, need_dbias)
PyObject* py_glu_backward(PyObject*, PyObject* const* a, Py_ssize_t n)
{
    return guarded(n, 9, [&] {
        const at::Tensor &dh = needed(a[0], "dh"), &g = needed(a[1], "g"), &u = needed(a[2], "u");
        const Triple gt(a[3], "gate"), ut(a[4], "up");
        const int act = integer(a[5]), gs = integer(a[6]), bits = integer(a[7]);
        const bool need = truth(a[8]);
        const Call c = on(dh, "dh");
        const int64_t M = dh.size(0), N = dh.size(1);
        const int64_t K = columns(needed(gt.at(0), "gate.wq"), tensor(gt.at(2), "gate.biases"), bits, "gate.wq");
        const c10::cuda::CUDAGuard guard(c.dev);
        const Gated w = gated(c, gt, ut, N, K, gs, bits);
        const uint16_t* dhp = c.operand(&dh, kBf16Bits, {M, N}, "dh");
        const uint16_t* gp = c.operand(&g, kBf16Bits, {M, N}, "g");
        const uint16_t* up = c.operand(&u, kBf16Bits, {M, N}, "u");
        const at::Tensor dx = c.make({M, K}), dg = c.make({M, N}), du = c.make({M, N});
        const at::Tensor dgb = need ? c.make({N}) : at::Tensor(), dub = need ? c.make({N}) : at::Tensor();
        const Scratch s(c, BQ_OP_GLU_BACKWARD, M, N, K, gs, bits);
        check(quant_matmul_glu_backward(dhp, gp, up, w.wq, w.scales, w.affine ? w.biases : nullptr, act,
                                        address<uint16_t>(dx), address<uint16_t>(dg), address<uint16_t>(du),
                                        need ? address<uint16_t>(dgb) : nullptr, need ? address<uint16_t>(dub) : nullptr, M,
                                        N, K, gs, bits, s.ptr, s.bytes, c.stream()),
              "quant_matmul_glu_backward");
        return need ? wrap({&dx, &dg, &du, &dgb, &dub}) : wrap({&dx, &dg, &du});
    });
}

PyObject* py_set_error(PyObject*, PyObject* type)
{
    Py_INCREF(type);
    Py_XSETREF(g_error, type);
    Py_RETURN_NONE;
}

#define BQ_FAST(f) reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(f))
PyMethodDef kMethods[] = {
    {"act", BQ_FAST(py_act), METH_FASTCALL, nullptr},
    {"act_backward", BQ_FAST(py_act_backward), METH_FASTCALL, nullptr},
    {"glu", BQ_FAST(py_glu), METH_FASTCALL, nullptr},
    {"glu_backward", BQ_FAST(py_glu_backward), METH_FASTCALL, nullptr},
    {"set_error", py_set_error, METH_O, nullptr},
    {nullptr, nullptr, 0, nullptr},
};
PyModuleDef kModule = {PyModuleDef_HEAD_INIT, "_binding", nullptr, -1, kMethods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__binding() { return PyModule_Create(&kModule); }
