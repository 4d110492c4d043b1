// layers_bind.cpp -- the Python side of include/emu_layers.h: checks of shapes,
// types, strides and devices, the outputs, and the call on the current stream.
//
// A call for a few tokens takes the GPU 5 to 30 us.  A call's host time on a
// Grace core, against the same steps in Python (ctypes and the tensors'
// attributes, some fifty a call): norm and rotation 5.0 us (18.1 in Python),
// their backward pass 10.2 (26.7), the gated product 7.0 (17.2), the adapters
// 12.2 (23.0).  Three quarters of what is left are the launches.
#include <Python.h>

#include <ATen/ops/empty.h>
#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include <algorithm>
#include <string>

#include "emu_layers.h"

namespace {

// The library's entry points (their addresses come with bind()) and the Python
// function that raises for a status.
struct {
    decltype(&emu_gated_rows) gated_rows;
    decltype(&emu_gated_pack) gated_pack;
    decltype(&emu_gated) gated;
    decltype(&emu_gated_bwd) gated_bwd;
    decltype(&emu_lora) lora;
    decltype(&emu_qk_norm_rope) qk;
    decltype(&emu_qk_norm_rope_bwd) qk_bwd;
} api;
PyObject* check_status;

struct Refused {                     // an argument that is refused
    PyObject* type;
    std::string why;
};
[[noreturn]] void value_error(std::string why) { throw Refused{PyExc_ValueError, std::move(why)}; }
[[noreturn]] void type_error(std::string why) { throw Refused{PyExc_TypeError, std::move(why)}; }
struct Raised {};                    // a Python error that is set

std::string show(at::IntArrayRef s) {
    std::string r = "(";
    for (size_t i = 0; i < s.size(); ++i) r += (i ? ", " : "") + std::to_string(s[i]);
    return r + (s.size() == 1 ? ",)" : ")");
}
const char* show(at::ScalarType t) { return c10::toString(t); }

// Tensors are borrowed from the call's arguments; null: None.
using T = const at::Tensor*;

T maybe(PyObject* o, const char* name) {
    if (o == Py_None) return nullptr;
    if (!THPVariable_Check(o)) type_error(std::string(name) + " must be a tensor, got " + Py_TYPE(o)->tp_name);
    return &THPVariable_Unpack(o);
}
T tensor(PyObject* o, const char* name) {
    T t = maybe(o, name);
    if (!t) type_error(std::string(name) + " must be a tensor, got None");
    return t;
}
bool truth(PyObject* o) {
    const int b = PyObject_IsTrue(o);
    if (b < 0) throw Raised{};
    return b != 0;
}
int64_t integer(PyObject* o) {
    const long long v = PyLong_AsLongLong(o);
    if (v == -1 && PyErr_Occurred()) throw Raised{};
    return v;
}

// The current device, which holds every tensor of the call.
int device_of(std::initializer_list<T> tensors) {
    const int dev = c10::cuda::current_device();
    for (T t : tensors)
        if (t && !(t->is_cuda() && t->get_device() == dev))
            value_error("expected tensors on the current CUDA device (cuda:" + std::to_string(dev) + "), got " +
                        t->device().str());
    return dev;
}
emu_stream_t stream_of(int dev) {
    return reinterpret_cast<emu_stream_t>(c10::cuda::getCurrentCUDAStream((c10::DeviceIndex)dev).stream());
}

// Row stride of a 2-D float32 matrix with unit stride along its rows (-1: any size).
int64_t rows_of(const at::Tensor& X, const char* name, int64_t rows = -1, int64_t cols = -1) {
    if (X.scalar_type() != at::kFloat) type_error(std::string(name) + " must be float32, got " + show(X.scalar_type()));
    const auto s = X.sizes();
    if (s.size() != 2 || (rows >= 0 && s[0] != rows) || (cols >= 0 && s[1] != cols))
        value_error(std::string(name) + " must be " + (rows >= 0 ? std::to_string(rows) : "M") + " x " +
                    (cols >= 0 ? std::to_string(cols) : "K") + ", got " + show(s));
    const auto st = X.strides();
    if (st[1] != 1 && s[1] > 1) value_error(std::string(name) + " needs unit stride along its rows");
    if (s[0] <= 1) return std::max<int64_t>(s[1], 1);
    if (st[0] < s[1]) value_error(std::string(name) + "'s rows overlap");
    return std::max<int64_t>(st[0], 1);
}

const float* floats(T x, const char* name, int64_t n) {
    if (!x) return nullptr;
    if (x->scalar_type() != at::kFloat || x->dim() != 1 || x->size(0) != n || (n > 1 && x->stride(0) != 1))
        value_error(std::string(name) + " must be " + std::to_string(n) + " contiguous float32 values");
    return static_cast<const float*>(x->data_ptr());
}
const int32_t* indices(T x, const char* name, int64_t n) {
    if (!x || x->scalar_type() != at::kInt || x->dim() != 1 || x->size(0) != n || (n > 1 && x->stride(0) != 1))
        value_error(std::string(name) + " must be " + std::to_string(n) + " contiguous int32 values");
    return static_cast<const int32_t*>(x->data_ptr());
}
float* f32(const at::Tensor& t) { return static_cast<float*>(t.data_ptr()); }

at::Tensor empty(at::IntArrayRef size, at::ScalarType type, int dev) {
    return at::empty(size, at::TensorOptions().dtype(type).device(at::kCUDA, (c10::DeviceIndex)dev));
}

// The outputs and the call need no Python: without its lock, as other threads
// may hold the allocator's or the library's and wait for it.
struct NoGil {
    PyThreadState* state = PyEval_SaveThread();
    ~NoGil() { PyEval_RestoreThread(state); }
};

void check(emu_status_t st, const char* where) {
    if (st == EMU_OK) return;
    PyObject* r = PyObject_CallFunction(check_status, "is", (int)st, where);
    Py_XDECREF(r);
    if (!r) throw Raised{};
    throw Refused{PyExc_RuntimeError, where};
}

PyObject* wrap(at::Tensor t) {
    PyObject* o = THPVariable_Wrap(std::move(t));
    if (!o) throw Raised{};
    return o;
}
PyObject* none() { Py_RETURN_NONE; }
PyObject* wrap_or_none(at::Tensor t) { return t.defined() ? wrap(std::move(t)) : none(); }
// The tuple of the objects, which it takes over.
template <size_t N>
PyObject* tuple(PyObject* const (&items)[N]) {
    PyObject* r = PyTuple_New(N);
    if (!r) throw Raised{};
    for (size_t i = 0; i < N; ++i) PyTuple_SET_ITEM(r, i, items[i]);
    return r;
}

// The version that in-place changes of a tensor raise (-1: an inference tensor,
// which has none).
int64_t version_of(const at::Tensor& t) { return t.is_inference() ? -1 : (int64_t)t._version(); }

// A function of exactly N positional arguments.
template <PyObject* (*F)(PyObject* const*), int N>
PyObject* entry(PyObject*, PyObject* const* a, Py_ssize_t n) {
    HANDLE_TH_ERRORS
    if (n != N) {
        PyErr_Format(PyExc_TypeError, "expected %d arguments, got %zd", N, n);
        return nullptr;
    }
    try {
        return F(a);
    } catch (const Refused& e) {
        PyErr_SetString(e.type, e.why.c_str());
        return nullptr;
    } catch (const Raised&) {
        return nullptr;
    }
    END_HANDLE_TH_ERRORS
}

// ------------------------------------------------- gated feed-forward --

// The tuple (Wg, Wu, pieces, version of Wg, version of Wu).
struct Gated {
    T Wg, Wu, pieces;
    int64_t F, K, ldg, ldu;
    explicit Gated(PyObject* o) {
        if (!PyTuple_Check(o) || PyTuple_GET_SIZE(o) != 5) type_error("w must come from emu_gated_pack");
        Wg = tensor(PyTuple_GET_ITEM(o, 0), "Wg");
        Wu = tensor(PyTuple_GET_ITEM(o, 1), "Wu");
        pieces = tensor(PyTuple_GET_ITEM(o, 2), "pieces");
        if (version_of(*Wg) != integer(PyTuple_GET_ITEM(o, 3)) || version_of(*Wu) != integer(PyTuple_GET_ITEM(o, 4)))
            value_error("a weight was changed in place since emu_gated_pack: pack again");
        ldg = rows_of(*Wg, "Wg");
        F = Wg->size(0);
        K = Wg->size(1);
        ldu = rows_of(*Wu, "Wu", F, K);
    }
};

PyObject* gated_pack(PyObject* const* a) {           // Wg, Wu
    T Wg = tensor(a[0], "Wg"), Wu = tensor(a[1], "Wu");
    const int64_t ldg = rows_of(*Wg, "Wg"), F = Wg->size(0), K = Wg->size(1);
    const int64_t ldu = rows_of(*Wu, "Wu", F, K);
    const int dev = device_of({Wg, Wu});
    at::Tensor P;
    emu_status_t st;
    {
        NoGil no;
        P = empty({3, 2 * api.gated_rows(F), std::max<int64_t>((K + 63) / 64 * 64, 64)}, at::kShort, dev);
        st = api.gated_pack(F, K, f32(*Wg), ldg, f32(*Wu), ldu, P.data_ptr(), P.size(2), stream_of(dev));
    }
    check(st, "emu_gated_pack");
    return wrap(P);
}

PyObject* gated(PyObject* const* a) {                // act, X, weights, save, out
    const int act = (int)integer(a[0]);
    T X = tensor(a[1], "X"), out = maybe(a[4], "out");
    const Gated w(a[2]);
    const bool save = truth(a[3]);
    const int64_t ldx = rows_of(*X, "X", -1, w.K), M = X->size(0), F = w.F;
    const int dev = device_of({X, w.Wg, w.Wu, out});
    const int64_t ldh = out ? rows_of(*out, "out", M, F) : std::max<int64_t>(F, 1);
    // G's and U's rows: whole 16-byte groups, so that they are stored and read as such
    const int64_t ldg = save ? std::max<int64_t>((F + 3) / 4 * 4, 4) : 0;
    at::Tensor H, G, U;
    emu_status_t st;
    {
        NoGil no;
        H = out ? *out : empty({M, F}, at::kFloat, dev);
        if (save) {
            G = empty({M, ldg}, at::kFloat, dev);
            U = empty({M, ldg}, at::kFloat, dev);
            if (ldg != F) {
                G = G.narrow(1, 0, F);
                U = U.narrow(1, 0, F);
            }
        }
        st = api.gated(act, M, F, w.K, f32(*X), ldx, f32(*w.Wg), w.ldg, f32(*w.Wu), w.ldu, w.pieces->data_ptr(),
                       w.pieces->size(2), f32(H), ldh, save ? f32(G) : nullptr, save ? f32(U) : nullptr, ldg,
                       stream_of(dev));
    }
    check(st, "emu_gated");
    return save ? tuple({wrap(H), wrap(G), wrap(U)}) : wrap(H);
}

PyObject* gated_bwd(PyObject* const* a) {            // act, dH, X, weights, G, U, need_dx, need_dw
    const int act = (int)integer(a[0]);
    T dH = tensor(a[1], "dH"), X = tensor(a[2], "X"), G = tensor(a[4], "G"), U = tensor(a[5], "U");
    const Gated w(a[3]);
    const bool need_dx = truth(a[6]), need_dw = truth(a[7]);
    const int64_t F = w.F, K = w.K, ldx = rows_of(*X, "X", -1, K), M = X->size(0);
    const int64_t lddh = rows_of(*dH, "dH", M, F), ldg = rows_of(*G, "G", M, F);
    if (rows_of(*U, "U", M, F) != ldg) value_error("G and U need the same row stride");
    const int dev = device_of({dH, X, G, U, w.Wg, w.Wu});
    const int64_t rows = w.pieces->size(1) / 2, ld = std::max<int64_t>(K, 1);
    at::Tensor dX, dWg, dWu;
    emu_status_t st;
    {
        NoGil no;
        at::Tensor dW;
        if (need_dx) dX = empty({M, K}, at::kFloat, dev);
        if (need_dw) {
            dW = empty({2 * rows, K}, at::kFloat, dev);
            dWg = dW.narrow(0, 0, F);
            dWu = dW.narrow(0, rows, F);
        }
        st = api.gated_bwd(act, M, F, K, f32(*dH), lddh, f32(*X), ldx, w.pieces->data_ptr(), w.pieces->size(2),
                           f32(*G), f32(*U), ldg, need_dx ? f32(dX) : nullptr, ld, need_dw ? f32(dW) : nullptr, ld,
                           stream_of(dev));
    }
    check(st, "emu_gated_bwd");
    return tuple({wrap_or_none(dX), wrap_or_none(dWg), wrap_or_none(dWu)});
}

// -------------------------------------------------- low-rank adapters --

PyObject* lora_weights(PyObject* const* a) {         // W, bias: checked only
    T W = tensor(a[0], "W"), bias = maybe(a[1], "bias");
    rows_of(*W, "W");
    floats(bias, "bias", W->size(0));
    device_of({W, bias});
    return none();
}

PyObject* lora(PyObject* const* a) {   // X, (W, bias, pieces, version of W), A, B, index, scale, out
    T X = tensor(a[0], "X"), A = tensor(a[2], "A"), B = tensor(a[3], "B");
    T index = maybe(a[4], "index"), scale = maybe(a[5], "scale"), out = maybe(a[6], "out");
    if (!PyTuple_Check(a[1]) || PyTuple_GET_SIZE(a[1]) != 4) type_error("w must come from emu_lora_pack");
    T W = tensor(PyTuple_GET_ITEM(a[1], 0), "W"), bias = maybe(PyTuple_GET_ITEM(a[1], 1), "bias");
    T pieces = tensor(PyTuple_GET_ITEM(a[1], 2), "pieces");
    if (version_of(*W) != integer(PyTuple_GET_ITEM(a[1], 3)))
        value_error("the weight was changed in place since emu_lora_pack: pack again");
    const int64_t ldw = rows_of(*W, "W"), N = W->size(0), K = W->size(1);
    const int64_t ldx = rows_of(*X, "X", -1, K), M = X->size(0);
    if (A->scalar_type() != at::kFloat || B->scalar_type() != at::kFloat) type_error("A and B must be float32");
    const auto sa = A->sizes(), sb = B->sizes();
    if (sa.size() != 3 || sb.size() != 3 || sa[2] != K || sb[0] != sa[0] || sb[1] != N || sb[2] != sa[1])
        value_error("A must be adapters x R x " + std::to_string(K) + " and B adapters x " + std::to_string(N) +
                    " x R, got " + show(sa) + " and " + show(sb));
    if (!A->is_contiguous() || !B->is_contiguous()) value_error("A and B must be contiguous");
    const int64_t n = sa[0], R = sa[1];
    const int32_t* ip = indices(index, "index", M);
    const float *sp = floats(scale, "scale", n), *bp = floats(bias, "bias", N);
    const int dev = device_of({X, W, bias, A, B, index, scale, out});
    const int64_t ldy = out ? rows_of(*out, "out", M, N) : std::max<int64_t>(N, 1);
    at::Tensor Y;
    emu_status_t st;
    {
        NoGil no;
        Y = out ? *out : empty({M, N}, at::kFloat, dev);
        st = api.lora(M, N, K, f32(*X), ldx, f32(*W), ldw, pieces->data_ptr(), pieces->size(2), bp, R, n, f32(*A),
                      f32(*B), sp, ip, f32(Y), ldy, stream_of(dev));
    }
    check(st, "emu_lora");
    return wrap(Y);
}

// ----------------------------- norm and rotation of queries and keys --

emu_heads_t heads_of(const at::Tensor& x, const char* name, at::IntArrayRef shape, at::ScalarType type) {
    if (x.scalar_type() != type)
        type_error(std::string("expected tensors of one type, got ") + show(type) + " and " + show(x.scalar_type()) +
                   " for " + name);
    if (x.sizes() != shape)
        value_error(std::string(name) + " must be tokens x heads x D = " + show(shape) + ", got " + show(x.sizes()));
    const auto st = x.strides();
    if (st[2] != 1 && shape[2] > 1) value_error(std::string(name) + " needs unit stride along the values of a head");
    return {x.data_ptr(), shape[1], st[0], st[1]};
}
// The same of an output: no two of its elements in one place.
emu_heads_t output_heads(const at::Tensor& x, const char* name, at::IntArrayRef shape, at::ScalarType type) {
    const emu_heads_t h = heads_of(x, name, shape, type);
    if ((h.token_stride == 0 && shape[0] > 1) || (h.head_stride == 0 && shape[1] > 1))
        if (x.numel() > 0) value_error(std::string(name) + "'s elements share memory");
    return h;
}
emu_heads_t dense_heads(const at::Tensor& x, int64_t heads, int64_t D) { return {x.data_ptr(), heads, heads * D, D}; }

// What both directions take: q, k, wq, wk, cos, sin, positions, eps, interleaved.
struct Qk {
    T q, k, wq, wk, cos, sin, positions;
    at::ScalarType type;
    int dtype, interleaved;
    float eps;
    int64_t tokens, D, rot = 0, table_rows = 0;
    emu_heads_t hq, hk;
    const float *pq, *pk, *pc = nullptr, *ps = nullptr;
    const int32_t* pp = nullptr;

    explicit Qk(PyObject* const* a)
        : q(tensor(a[0], "q")), k(tensor(a[1], "k")), wq(maybe(a[2], "wq")), wk(maybe(a[3], "wk")),
          cos(maybe(a[4], "cos")), sin(maybe(a[5], "sin")), positions(maybe(a[6], "positions")) {
        type = q->scalar_type();
        dtype = type == at::kFloat ? EMU_F32 : type == at::kBFloat16 ? EMU_BF16 : type == at::kHalf ? EMU_F16 : -1;
        if (dtype < 0) type_error(std::string("q and k must be float32, bfloat16 or float16, got ") + show(type));
        const auto qs = q->sizes(), ks = k->sizes();
        if (qs.size() != 3 || ks.size() != 3 || ks[0] != qs[0] || ks[2] != qs[2])
            value_error("q and k must be tokens x heads x D with the same tokens and D, got " + show(qs) + ", " +
                        show(ks));
        tokens = qs[0];
        D = qs[2];
        hq = heads_of(*q, "q", qs, type);
        hk = heads_of(*k, "k", ks, type);
        pq = floats(wq, "wq", D);
        pk = floats(wk, "wk", D);
        const double e = PyFloat_AsDouble(a[7]);
        if (e == -1.0 && PyErr_Occurred()) throw Raised{};
        eps = (float)e;
        interleaved = truth(a[8]);
        if (!cos != !sin) value_error("cos and sin go together");
        if (!cos) return;
        if (cos->scalar_type() != at::kFloat || sin->scalar_type() != at::kFloat)
            type_error("cos and sin must be float32");
        if (cos->dim() != 2 || sin->sizes() != cos->sizes() || !cos->is_contiguous() || !sin->is_contiguous())
            value_error("cos and sin must be contiguous matrices of one shape, positions x rot/2");
        rot = 2 * cos->size(1);
        table_rows = cos->size(0);
        pc = f32(*cos);
        ps = f32(*sin);
        pp = indices(positions, "positions", tokens);
    }
};

PyObject* qk(PyObject* const* a) {                   // what Qk takes, q', k' (both or neither None)
    const Qk x(a);
    T qo = maybe(a[9], "out[0]"), ko = maybe(a[10], "out[1]");
    if (!qo != !ko) type_error("out must be two tensors");
    emu_heads_t h[4] = {x.hq, x.hk, {}, {}};
    if (qo) {
        h[2] = output_heads(*qo, "out[0]", x.q->sizes(), x.type);
        h[3] = output_heads(*ko, "out[1]", x.k->sizes(), x.type);
    }
    const int dev = device_of({x.q, x.k, x.wq, x.wk, x.cos, x.sin, x.positions, qo, ko});
    at::Tensor q, k;
    emu_status_t st;
    {
        NoGil no;
        if (qo) {
            q = *qo;
            k = *ko;
        } else {
            q = empty(x.q->sizes(), x.type, dev);
            k = empty(x.k->sizes(), x.type, dev);
            h[2] = dense_heads(q, x.hq.heads, x.D);
            h[3] = dense_heads(k, x.hk.heads, x.D);
        }
        st = api.qk(x.dtype, x.tokens, x.D, x.rot, x.interleaved, x.eps, h, x.pq, x.pk, x.pc, x.ps, x.table_rows,
                    x.pp, stream_of(dev));
    }
    check(st, "emu_qk_norm_rope");
    return tuple({wrap(q), wrap(k)});
}

PyObject* qk_bwd(PyObject* const* a) {               // what Qk takes, dq', dk'
    const Qk x(a);
    T dqo = tensor(a[9], "dq_out"), dko = tensor(a[10], "dk_out");
    const int dev = device_of({x.q, x.k, x.wq, x.wk, x.cos, x.sin, x.positions, dqo, dko});
    emu_heads_t h[6] = {x.hq, x.hk, {}, {}, heads_of(*dqo, "dq_out", x.q->sizes(), x.type),
                        heads_of(*dko, "dk_out", x.k->sizes(), x.type)};
    at::Tensor dq, dk, dwq, dwk;
    emu_status_t st;
    {
        NoGil no;
        dq = empty(x.q->sizes(), x.type, dev);
        dk = empty(x.k->sizes(), x.type, dev);
        if (x.wq) dwq = empty({x.D}, at::kFloat, dev);
        if (x.wk) dwk = empty({x.D}, at::kFloat, dev);
        h[2] = dense_heads(dq, x.hq.heads, x.D);
        h[3] = dense_heads(dk, x.hk.heads, x.D);
        st = api.qk_bwd(x.dtype, x.tokens, x.D, x.rot, x.interleaved, x.eps, h, x.pq, x.pk, x.pc, x.ps, x.table_rows,
                        x.pp, x.wq ? f32(dwq) : nullptr, x.wk ? f32(dwk) : nullptr, stream_of(dev));
    }
    check(st, "emu_qk_norm_rope_bwd");
    return tuple({wrap(dq), wrap(dk), wrap_or_none(dwq), wrap_or_none(dwk)});
}

// (function that raises for a status, the entry points' addresses in api's order)
PyObject* bind(PyObject*, PyObject* args) {
    static_assert(sizeof(api) == 7 * sizeof(void*), "one pointer each");
    unsigned long long p[7];
    PyObject* f;
    if (!PyArg_ParseTuple(args, "OKKKKKKK", &f, &p[0], &p[1], &p[2], &p[3], &p[4], &p[5], &p[6])) return nullptr;
    auto set = [&](auto& to, int i) { to = reinterpret_cast<std::decay_t<decltype(to)>>((uintptr_t)p[i]); };
    set(api.gated_rows, 0);
    set(api.gated_pack, 1);
    set(api.gated, 2);
    set(api.gated_bwd, 3);
    set(api.lora, 4);
    set(api.qk, 5);
    set(api.qk_bwd, 6);
    Py_INCREF(f);
    Py_XDECREF(check_status);
    check_status = f;
    Py_RETURN_NONE;
}

template <PyObject* (*F)(PyObject* const*), int N>
PyCFunction fast() {
    return reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(&entry<F, N>));
}

PyMethodDef* methods() {
    static PyMethodDef m[] = {
        {"bind", bind, METH_VARARGS, nullptr},
        {"gated_pack", fast<gated_pack, 2>(), METH_FASTCALL, nullptr},
        {"gated", fast<gated, 5>(), METH_FASTCALL, nullptr},
        {"gated_bwd", fast<gated_bwd, 8>(), METH_FASTCALL, nullptr},
        {"lora_weights", fast<lora_weights, 2>(), METH_FASTCALL, nullptr},
        {"lora", fast<lora, 7>(), METH_FASTCALL, nullptr},
        {"qk_norm_rope", fast<qk, 11>(), METH_FASTCALL, nullptr},
        {"qk_norm_rope_bwd", fast<qk_bwd, 11>(), METH_FASTCALL, nullptr},
        {nullptr, nullptr, 0, nullptr}};
    return m;
}

}  // namespace

PyMODINIT_FUNC PyInit_emu_layers_bind() {
    static PyModuleDef def = {PyModuleDef_HEAD_INIT, "emu_layers_bind", nullptr, -1, methods(),
                              nullptr, nullptr, nullptr, nullptr};
    return PyModule_Create(&def);
}
