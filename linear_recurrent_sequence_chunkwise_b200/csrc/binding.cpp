// binding.cpp -- the common calls of the short operators without Python on the
// way: a decode step or the norm of a few tokens takes the GPU 4 to 6 us, and
// checks, outputs and pointers handled in Python cost 15 us around it.
//
// Each function takes the arguments of its Python namesake that are left when
// no output, workspace or stream is passed in, checks everything that the C ABI
// cannot see, makes the outputs and calls the C entry point.  It returns None
// for whatever it does not take (other layouts, devices or types, arguments
// that do not fit): the Python function then goes its general way, which also
// words the errors.  Once the entry point has been called nothing is done twice (a
// decode step updates its state): an error status comes back as an int, which the
// Python function raises.
#include <Python.h>

#include <ATen/cuda/EmptyTensor.h>
#include <ATen/core/Tensor.h>
#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/autograd/python_variable.h>

#include "retention.h"

namespace {

using at::Tensor;

// A plain tensor argument (no subclass: those have Python behaviour of their own).
const Tensor* tensor(PyObject* o) {
    if (!THPVariable_CheckExact(o) && !(THPVariable_Check(o) && Py_TYPE(o) == reinterpret_cast<PyTypeObject*>(ParameterClass)))
        return nullptr;
    return &THPVariable_Unpack(o);
}
bool plain(const Tensor& t, int dev) { return t.is_cuda() && t.get_device() == dev && t.is_contiguous(); }
bool is_float(const Tensor& t) { return t.scalar_type() == at::kFloat || t.scalar_type() == at::kBFloat16; }
ret_dtype code(const Tensor& t) { return t.scalar_type() == at::kFloat ? RET_F32 : RET_BF16; }
bool f32(const Tensor& t, int dev, at::IntArrayRef sizes) {
    return t.scalar_type() == at::kFloat && plain(t, dev) && t.sizes() == sizes;
}
Tensor make(at::IntArrayRef sizes, at::ScalarType type, int dev) {
    return at::detail::empty_cuda(sizes, type, c10::Device(c10::kCUDA, (c10::DeviceIndex)dev), std::nullopt);
}
cudaStream_t stream(int dev) { return c10::cuda::getCurrentCUDAStream((c10::DeviceIndex)dev).stream(); }
// The inputs' device, if it is the current one; -1 else.
int device_of(const Tensor& t) {
    if (!t.is_cuda()) return -1;
    const int dev = t.get_device();
    return dev == c10::cuda::current_device() ? dev : -1;
}

PyObject* pass() { Py_RETURN_NONE; }
PyObject* error(ret_status st) { return PyLong_FromLong(st); }
// A tuple of tensors, None for an undefined one.
PyObject* tuple(std::initializer_list<Tensor> ts) {
    PyObject* r = PyTuple_New((Py_ssize_t)ts.size());
    Py_ssize_t i = 0;
    for (const Tensor& t : ts) PyTuple_SET_ITEM(r, i++, t.defined() ? THPVariable_Wrap(t) : pass());
    return r;
}
const float* fptr(const Tensor* t) { return t ? t->data_ptr<float>() : nullptr; }

// q, k, v, g, beta, lengths, initial_state of a call over sequences.
struct Delta {
    const Tensor *q, *k, *v, *g, *beta, *lengths, *state;
    int dev, B, N, Hk, H, dk, dv;
    bool read(PyObject* const* a) {
        const Tensor** t[] = {&q, &k, &v, &g, &beta};
        for (int i = 0; i < 5; i++)
            if (!(*t[i] = tensor(a[i]))) return false;
        lengths = a[5] == Py_None ? nullptr : tensor(a[5]);
        state = a[6] == Py_None ? nullptr : tensor(a[6]);
        if ((a[5] != Py_None && !lengths) || (a[6] != Py_None && !state)) return false;
        dev = device_of(*q);
        if (dev < 0 || !is_float(*q) || q->dim() != 4 || v->dim() != 4 || k->sizes() != q->sizes() || v->size(0) != q->size(0) ||
            v->size(1) != q->size(1))
            return false;
        for (const Tensor* x : {q, k, v})
            if (!plain(*x, dev) || x->scalar_type() != q->scalar_type()) return false;
        for (int64_t x : {q->size(0), q->size(1), q->size(2), q->size(3), v->size(2), v->size(3)})
            if (x < 1 || x > INT32_MAX) return false;
        B = (int)q->size(0), N = (int)q->size(1), Hk = (int)q->size(2), dk = (int)q->size(3);
        H = (int)v->size(2), dv = (int)v->size(3);
        return f32(*g, dev, {B, N, H}) && f32(*beta, dev, {B, N, H}) && (!state || f32(*state, dev, {B, H, dk, dv})) &&
               (!lengths || (lengths->scalar_type() == at::kInt && plain(*lengths, dev) && lengths->sizes() == at::IntArrayRef({B})));
    }
    const int32_t* lens() const { return lengths ? lengths->data_ptr<int32_t>() : nullptr; }
};
// Runs f; a C++ exception (no memory for an output, say: before the entry point's
// call) becomes None, and the general way meets it again.
template <typename F>
PyObject* guarded(F f) {
    try {
        return f();
    } catch (...) {
        PyErr_Clear();
        return pass();
    }
}

// (x, gain, bias, eps, want_stats)
PyObject* layernorm_forward(PyObject*, PyObject* const* a, Py_ssize_t n) {
    return guarded([&]() -> PyObject* {
        if (n != 5) return pass();
        const Tensor* x = tensor(a[0]);
        const Tensor *gain = a[1] == Py_None ? nullptr : tensor(a[1]), *bias = a[2] == Py_None ? nullptr : tensor(a[2]);
        if (!x || (a[1] != Py_None && !gain) || (a[2] != Py_None && !bias) || !PyFloat_CheckExact(a[3])) return pass();
        const int dev = device_of(*x);
        if (dev < 0 || !is_float(*x) || !plain(*x, dev) || x->dim() < 1 || x->numel() == 0) return pass();
        const int64_t d = x->size(-1), rows = x->numel() / d;
        for (const Tensor* w : {gain, bias})
            if (w && (!is_float(*w) || !plain(*w, dev) || w->dim() != 1 || w->size(0) != d)) return pass();
        if ((gain && bias && gain->scalar_type() != bias->scalar_type()) || d > INT32_MAX) return pass();
        const bool stats = PyObject_IsTrue(a[4]) == 1;
        const at::IntArrayRef lead = x->sizes().slice(0, x->dim() - 1);
        Tensor y = make(x->sizes(), x->scalar_type(), dev), mean, rstd;
        if (stats) {
            mean = make(lead, at::kFloat, dev);
            rstd = make(lead, at::kFloat, dev);
        }
        const Tensor* w = gain ? gain : bias;
        const ret_status st =
            ret_layernorm_forward(x->data_ptr(), gain ? gain->data_ptr() : nullptr, bias ? bias->data_ptr() : nullptr,
                                  PyFloat_AS_DOUBLE(a[3]), rows, (int)d, y.data_ptr(),
                                  stats ? mean.data_ptr<float>() : nullptr, stats ? rstd.data_ptr<float>() : nullptr,
                                  code(*x), w ? code(*w) : RET_F32, stream(dev));
        if (st != RET_OK) return error(st);
        return stats ? tuple({y, mean, rstd}) : THPVariable_Wrap(y);
    });
}

// (dout, x, mean, rstd, gain): with the gradients of the weights
PyObject* layernorm_backward(PyObject*, PyObject* const* a, Py_ssize_t n) {
    return guarded([&]() -> PyObject* {
        if (n != 5) return pass();
        const Tensor *dy = tensor(a[0]), *x = tensor(a[1]), *mean = tensor(a[2]), *rstd = tensor(a[3]);
        const Tensor* gain = a[4] == Py_None ? nullptr : tensor(a[4]);
        if (!dy || !x || !mean || !rstd || (a[4] != Py_None && !gain)) return pass();
        const int dev = device_of(*x);
        if (dev < 0 || !is_float(*x) || !plain(*x, dev) || x->dim() < 1 || x->numel() == 0) return pass();
        const int64_t d = x->size(-1), rows = x->numel() / d;
        const at::IntArrayRef lead = x->sizes().slice(0, x->dim() - 1);
        if (!plain(*dy, dev) || dy->scalar_type() != x->scalar_type() || dy->sizes() != x->sizes() || !f32(*mean, dev, lead) ||
            !f32(*rstd, dev, lead) || d > INT32_MAX ||
            (gain && (!is_float(*gain) || !plain(*gain, dev) || gain->dim() != 1 || gain->size(0) != d)))
            return pass();
        const size_t need = ret_layernorm_backward_workspace_bytes(rows, (int)d);
        Tensor dx = make(x->sizes(), x->scalar_type(), dev), dgain = make({d}, at::kFloat, dev), dbias = make({d}, at::kFloat, dev);
        Tensor ws = make({(int64_t)need}, at::kByte, dev);
        const ret_status st =
            ret_layernorm_backward(dy->data_ptr(), x->data_ptr(), mean->data_ptr<float>(), rstd->data_ptr<float>(),
                                   gain ? gain->data_ptr() : nullptr, rows, (int)d, dx.data_ptr(), dgain.data_ptr<float>(),
                                   dbias.data_ptr<float>(), code(*x), gain ? code(*gain) : RET_F32, ws.data_ptr(), need,
                                   stream(dev));
        if (st != RET_OK) return error(st);
        return tuple({dx, dgain, dbias});
    });
}

// (q, k, v, g, beta, state, out in bf16)
PyObject* delta_decode_step(PyObject*, PyObject* const* a, Py_ssize_t n) {
    return guarded([&]() -> PyObject* {
        if (n != 7) return pass();
        const Tensor* t[6];
        for (int i = 0; i < 6; i++)
            if (!(t[i] = tensor(a[i]))) return pass();
        const Tensor &q = *t[0], &k = *t[1], &v = *t[2], &state = *t[5];
        const int dev = device_of(q);
        if (dev < 0 || !is_float(q) || q.dim() != 3 || v.dim() != 3 || k.sizes() != q.sizes() || v.size(0) != q.size(0)) return pass();
        for (const Tensor* x : {&q, &k, &v})
            if (!plain(*x, dev) || x->scalar_type() != q.scalar_type()) return pass();
        const int64_t B = q.size(0), Hk = q.size(1), dk = q.size(2), H = v.size(1), dv = v.size(2);
        if (!f32(*t[3], dev, {B, H}) || !f32(*t[4], dev, {B, H}) || !f32(state, dev, {B, H, dk, dv}) ||
            std::max(std::max(B, H), std::max(Hk, std::max(dk, dv))) > INT32_MAX)
            return pass();
        const bool bf16 = PyObject_IsTrue(a[6]) == 1;
        Tensor out = make({B, H, dv}, bf16 ? at::kBFloat16 : at::kFloat, dev);
        const ret_status st =
            ret_delta_decode_step(q.data_ptr(), k.data_ptr(), v.data_ptr(), t[3]->data_ptr<float>(), t[4]->data_ptr<float>(),
                                  state.data_ptr<float>(), out.data_ptr(), stream(dev), (int)B, (int)Hk, (int)H, (int)dk,
                                  (int)dv, code(q), bf16 ? RET_BF16 : RET_F32);
        if (st != RET_OK) return error(st);
        return THPVariable_Wrap(out);
    });
}

// (q, k, v, g, beta, lengths, initial_state, out, out in bf16, want_final_state)
PyObject* delta_forward(PyObject*, PyObject* const* a, Py_ssize_t n) {
    return guarded([&]() -> PyObject* {
        Delta d;
        if (n != 10 || !d.read(a)) return pass();
        Tensor out, final_state, ws;
        if (a[7] == Py_None) {
            out = make({d.B, d.N, d.H, d.dv}, PyObject_IsTrue(a[8]) == 1 ? at::kBFloat16 : at::kFloat, d.dev);
        } else {
            const Tensor* o = tensor(a[7]);
            if (!o || !is_float(*o) || !plain(*o, d.dev) || o->sizes() != d.v->sizes()) return pass();
            out = *o;
        }
        if (PyObject_IsTrue(a[9]) == 1) final_state = make({d.B, d.H, d.dk, d.dv}, at::kFloat, d.dev);
        const size_t need = ret_delta_workspace_bytes(d.B, d.N, d.Hk, d.H, d.dk, d.dv, code(*d.q));
        if (need) ws = make({(int64_t)need}, at::kByte, d.dev);
        const ret_status st =
            ret_delta_forward_chunkwise(d.q->data_ptr(), d.k->data_ptr(), d.v->data_ptr(), fptr(d.g), fptr(d.beta), d.lens(),
                                        fptr(d.state), d.B, d.N, d.Hk, d.H, d.dk, d.dv, out.data_ptr(),
                                        final_state.defined() ? final_state.data_ptr<float>() : nullptr, stream(d.dev),
                                        code(*d.q), code(out), need ? ws.data_ptr() : nullptr, need);
        if (st != RET_OK) return error(st);
        return final_state.defined() ? tuple({out, final_state}) : THPVariable_Wrap(out);
    });
}

// (q, k, v, g, beta, lengths, initial_state, dout, dfinal_state, gradients in bf16, want_dinitial_state)
PyObject* delta_backward(PyObject*, PyObject* const* a, Py_ssize_t n) {
    return guarded([&]() -> PyObject* {
        Delta d;
        if (n != 11 || !d.read(a)) return pass();
        const Tensor *dout = tensor(a[7]), *dfinal = a[8] == Py_None ? nullptr : tensor(a[8]);
        if (!dout || dout->scalar_type() != d.q->scalar_type() || !plain(*dout, d.dev) || dout->sizes() != d.v->sizes() ||
            (a[8] != Py_None && (!dfinal || !f32(*dfinal, d.dev, {d.B, d.H, d.dk, d.dv}))))
            return pass();
        const size_t need = ret_delta_backward_workspace_bytes(d.B, d.N, d.Hk, d.H, d.dk, d.dv, code(*d.q));
        if (!need) return pass();
        const at::ScalarType type = PyObject_IsTrue(a[9]) == 1 ? at::kBFloat16 : at::kFloat;
        Tensor dq = make(d.q->sizes(), type, d.dev), dk = make(d.k->sizes(), type, d.dev), dv = make(d.v->sizes(), type, d.dev);
        Tensor dg = make(d.g->sizes(), at::kFloat, d.dev), dbeta = make(d.g->sizes(), at::kFloat, d.dev), ds0;
        if (PyObject_IsTrue(a[10]) == 1) ds0 = make({d.B, d.H, d.dk, d.dv}, at::kFloat, d.dev);
        Tensor ws = make({(int64_t)need}, at::kByte, d.dev);
        const ret_status st =
            ret_delta_backward_chunkwise(d.q->data_ptr(), d.k->data_ptr(), d.v->data_ptr(), fptr(d.g), fptr(d.beta),
                                         dout->data_ptr(), d.lens(), fptr(d.state), fptr(dfinal), d.B, d.N, d.Hk, d.H, d.dk, d.dv,
                                         dq.data_ptr(), dk.data_ptr(), dv.data_ptr(), dg.data_ptr<float>(),
                                         dbeta.data_ptr<float>(), ds0.defined() ? ds0.data_ptr<float>() : nullptr, stream(d.dev),
                                         code(*d.q), code(dq), ws.data_ptr(), need);
        if (st != RET_OK) return error(st);
        return tuple({dq, dk, dv, dg, dbeta, ds0});
    });
}

// (q, k, freqs, positions, pos_offset, half, scale, inverse)
PyObject* rotary(PyObject*, PyObject* const* a, Py_ssize_t n) {
    return guarded([&]() -> PyObject* {
        if (n != 8) return pass();
        const Tensor *q = tensor(a[0]), *k = a[1] == Py_None ? nullptr : tensor(a[1]), *freqs = tensor(a[2]);
        const Tensor* pos = a[3] == Py_None ? nullptr : tensor(a[3]);
        if (!q || !freqs || (a[1] != Py_None && !k) || (a[3] != Py_None && !pos) || !PyLong_CheckExact(a[4]) ||
            !PyFloat_CheckExact(a[6]))
            return pass();
        const int dev = device_of(*q);
        if (dev < 0 || !is_float(*q) || q->dim() != 4 || !plain(*q, dev)) return pass();
        const int64_t B = q->size(0), N = q->size(1), H = q->size(2), d = q->size(3), Hk = k ? k->dim() == 4 ? k->size(2) : 0 : 0;
        if (k && (!plain(*k, dev) || k->scalar_type() != q->scalar_type() || k->sizes() != at::IntArrayRef({B, N, Hk, d}))) return pass();
        if (freqs->is_cuda() || freqs->scalar_type() != at::kDouble || freqs->dim() != 1 || !freqs->is_contiguous()) return pass();
        if (pos && (!plain(*pos, dev) || pos->scalar_type() != at::kLong || pos->sizes() != at::IntArrayRef({B, N}))) return pass();
        int over = 0;
        const long long offset = PyLong_AsLongLongAndOverflow(a[4], &over);
        if (over || std::max(std::max(B, N), std::max(std::max(H, Hk), std::max(d, 2 * freqs->numel()))) > INT32_MAX) return pass();
        Tensor qo = make(q->sizes(), q->scalar_type(), dev), ko;
        if (k) ko = make(k->sizes(), q->scalar_type(), dev);
        const ret_status st =
            ret_rotary(q->data_ptr(), k ? k->data_ptr() : nullptr, qo.data_ptr(), k ? ko.data_ptr() : nullptr, nullptr, nullptr,
                       nullptr, nullptr, freqs->data_ptr<double>(), PyFloat_AS_DOUBLE(a[6]),
                       pos ? pos->data_ptr<int64_t>() : nullptr, offset, PyObject_IsTrue(a[7]) == 1,
                       PyObject_IsTrue(a[5]) == 1 ? RET_ROTARY_HALF : RET_ROTARY_INTERLEAVED, (int)B, (int)N, (int)H, (int)Hk,
                       (int)d, (int)(2 * freqs->numel()), code(*q), stream(dev));
        if (st != RET_OK) return error(st);
        return k ? tuple({qo, ko}) : THPVariable_Wrap(qo);
    });
}

PyMethodDef methods[] = {
    {"layernorm_forward", (PyCFunction)(void*)layernorm_forward, METH_FASTCALL, nullptr},
    {"layernorm_backward", (PyCFunction)(void*)layernorm_backward, METH_FASTCALL, nullptr},
    {"delta_decode_step", (PyCFunction)(void*)delta_decode_step, METH_FASTCALL, nullptr},
    {"delta_forward", (PyCFunction)(void*)delta_forward, METH_FASTCALL, nullptr},
    {"delta_backward", (PyCFunction)(void*)delta_backward, METH_FASTCALL, nullptr},
    {"rotary", (PyCFunction)(void*)rotary, METH_FASTCALL, nullptr},
    {nullptr, nullptr, 0, nullptr},
};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_binding", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__binding() { return PyModule_Create(&module); }
