// The binding's common case for calls of a few microseconds: contiguous
// tensors of the expected types on the current device.  Every function checks,
// allocates its results, takes torch's current stream and calls the C ABI; for
// anything else, and for any status but IQ_OK, it returns None and the binding
// in Python goes through its own checks, which say what is wrong.
#include <Python.h>

#include <ATen/core/Tensor.h>
#include <ATen/ops/empty.h>
#include <c10/core/GradMode.h>
#include <c10/hip/HIPFunctions.h>
#include <c10/hip/HIPStream.h>
#include <torch/csrc/autograd/python_variable.h>

#include <algorithm>
#include <initializer_list>

#include "../../include/iq.h"

namespace {

decltype(&iq_layer_norm) f_layer_norm;
decltype(&iq_layer_norm_backward) f_layer_norm_backward;
decltype(&iq_layer_norm_workspace_bytes) f_layer_norm_workspace_bytes;
decltype(&iq_gated_forward) f_gated_forward;
decltype(&iq_gated_backward) f_gated_backward;
decltype(&iq_gated_workspace_bytes) f_gated_workspace_bytes;
decltype(&iq_packed_gemv) f_packed_gemv;
decltype(&iq_packed_gated) f_packed_gated;

// bind(address, ...): the entry points in the order above.
PyObject* bind(PyObject*, PyObject* const* args, Py_ssize_t n) {
    void** to[] = {(void**)&f_layer_norm, (void**)&f_layer_norm_backward, (void**)&f_layer_norm_workspace_bytes,
                   (void**)&f_gated_forward, (void**)&f_gated_backward, (void**)&f_gated_workspace_bytes,
                   (void**)&f_packed_gemv, (void**)&f_packed_gated};
    if (n != 8) return PyErr_Format(PyExc_TypeError, "eight addresses");
    for (int i = 0; i < 8; ++i) {
        *to[i] = PyLong_AsVoidPtr(args[i]);
        if (PyErr_Occurred()) return nullptr;
    }
    Py_RETURN_NONE;
}

struct Other {};          // not the common case

// A tensor that no graph follows; of others the binding in Python says that their gradients would be lost.
const at::Tensor& tensor(PyObject* o) {
    if (!THPVariable_CheckExact(o)) throw Other();
    const at::Tensor& t = THPVariable_Unpack(o);
    if (t.requires_grad() && c10::GradMode::is_enabled()) throw Other();
    return t;
}
int64_t whole(PyObject* o) {
    const long long v = PyLong_AsLongLong(o);
    if (v == -1 && PyErr_Occurred()) { PyErr_Clear(); throw Other(); }
    return v;
}
void need(bool yes) {
    if (!yes) throw Other();
}

int32_t dtype(const at::Tensor& t) {
    if (t.scalar_type() == at::kBFloat16) return IQ_BF16;
    need(t.scalar_type() == at::kFloat);
    return IQ_F32;
}

// x of a call: two dimensions, dense, on the current device.
void check_x(const at::Tensor& x) { need(x.is_cuda() && x.dim() == 2 && x.is_contiguous() && x.get_device() == c10::hip::current_device()); }
void check(const at::Tensor& t, const at::Tensor& x, at::ScalarType type, std::initializer_list<int64_t> shape) {
    need(t.scalar_type() == type && t.sizes() == at::IntArrayRef(shape) && t.is_cuda() && t.get_device() == x.get_device() && t.is_contiguous());
}
void* at_least(const at::Tensor& t, const at::Tensor& x, int64_t bytes) {
    need(t.is_cuda() && t.get_device() == x.get_device() && t.is_contiguous() && (int64_t)t.nbytes() >= bytes);
    return t.data_ptr();
}
at::Tensor make(const at::Tensor& x, std::initializer_list<int64_t> shape, at::ScalarType type) {
    return at::empty(at::IntArrayRef(shape), x.options().dtype(type).requires_grad(false));
}
hipStream_t stream(const at::Tensor& x) { return c10::hip::getCurrentHIPStream(x.get_device()).stream(); }

PyObject* wrap(std::initializer_list<at::Tensor> results) {
    PyObject* t = PyTuple_New((Py_ssize_t)results.size());
    Py_ssize_t i = 0;
    for (const at::Tensor& r : results) PyTuple_SET_ITEM(t, i++, THPVariable_Wrap(r));
    return t;
}

template <PyObject* (*F)(PyObject* const*)> PyObject* guarded(PyObject*, PyObject* const* args, Py_ssize_t) {
    try {
        return F(args);
    } catch (...) {          // out of memory among them: the call in Python meets it too and reports it
        PyErr_Clear();
        Py_RETURN_NONE;
    }
}

// layer_norm(x, weight, bias, eps)
PyObject* layer_norm(PyObject* const* a) {
    const at::Tensor& x = tensor(a[0]);
    check_x(x);
    const int64_t rows = x.size(0), cols = x.size(1);
    const double eps = PyFloat_Check(a[3]) ? PyFloat_AS_DOUBLE(a[3]) : throw Other();
    const void* param[2] = {nullptr, nullptr};
    int32_t pt = IQ_F32;
    at::ScalarType type = at::kFloat;
    for (int i = 1; i >= 0; --i)
        if (a[1 + i] != Py_None) {
            const at::Tensor& p = tensor(a[1 + i]);
            if (param[1]) need(p.scalar_type() == type);
            type = p.scalar_type();
            pt = dtype(p);
            check(p, x, type, {cols});
            param[i] = p.data_ptr();
        }
    const iq_desc d = {0, 0, dtype(x), 0, rows, cols, cols, 0, 0};
    at::Tensor y = make(x, {rows, cols}, x.scalar_type()), mean = make(x, {rows}, at::kFloat), rstd = make(x, {rows}, at::kFloat);
    need(f_layer_norm(&d, x.data_ptr(), param[0], param[1], pt, (float)eps, y.data_ptr(), mean.data_ptr<float>(),
                      rstd.data_ptr<float>(), stream(x)) == IQ_OK);
    return wrap({y, mean, rstd});
}

// layer_norm_backward(dy, x, weight, mean, rstd)
PyObject* layer_norm_backward(PyObject* const* a) {
    const at::Tensor &dy = tensor(a[0]), &x = tensor(a[1]), &mean = tensor(a[3]), &rstd = tensor(a[4]);
    check_x(x);
    const int64_t rows = x.size(0), cols = x.size(1);
    check(dy, x, x.scalar_type(), {rows, cols});
    check(mean, x, at::kFloat, {rows});
    check(rstd, x, at::kFloat, {rows});
    const void* weight = nullptr;
    at::ScalarType type = at::kFloat;
    int32_t pt = IQ_F32;
    if (a[2] != Py_None) {
        const at::Tensor& w = tensor(a[2]);
        type = w.scalar_type();
        pt = dtype(w);
        check(w, x, type, {cols});
        weight = w.data_ptr();
    }
    const iq_desc d = {0, 0, dtype(x), 0, rows, cols, cols, 0, 0};
    at::Tensor dx = make(x, {rows, cols}, x.scalar_type()), dw = make(x, {cols}, type), db = make(x, {cols}, type);
    at::Tensor ws = make(x, {std::max<int64_t>(256, (int64_t)f_layer_norm_workspace_bytes(&d))}, at::kByte);
    need(f_layer_norm_backward(&d, x.data_ptr(), dy.data_ptr(), weight, pt, mean.data_ptr<float>(), rstd.data_ptr<float>(),
                               dx.data_ptr(), dw.data_ptr(), db.data_ptr(), ws.data_ptr(), stream(x)) == IQ_OK);
    return wrap({dx, dw, db});
}

iq_gated_desc gated_desc(const at::Tensor& x, const at::Tensor& wg, const at::Tensor& wu, int64_t act) {
    check_x(x);
    need(wg.dim() == 2);
    const int64_t cols = x.size(1), features = wg.size(0);
    need(x.scalar_type() == at::kBFloat16);
    check(wg, x, at::kBFloat16, {features, cols});
    check(wu, x, at::kBFloat16, {features, cols});
    return {(int32_t)act, IQ_BF16, x.size(0), cols, features, cols, 0, 0};
}

// gated(x, w_gate, w_up, act, save)
PyObject* gated(PyObject* const* a) {
    const at::Tensor &x = tensor(a[0]), &wg = tensor(a[1]), &wu = tensor(a[2]);
    const iq_gated_desc d = gated_desc(x, wg, wu, whole(a[3]));
    const bool save = a[4] == Py_True;
    at::Tensor h = make(x, {d.tokens, d.features}, at::kBFloat16), saved;
    if (save) saved = make(x, {2, d.tokens, d.features}, at::kFloat);
    need(f_gated_forward(&d, x.data_ptr(), wg.data_ptr(), wu.data_ptr(), h.data_ptr(), save ? saved.data_ptr() : nullptr, stream(x)) == IQ_OK);
    return save ? wrap({h, saved}) : THPVariable_Wrap(h);
}

// gated_backward(dh, x, w_gate, w_up, saved, act)
PyObject* gated_backward(PyObject* const* a) {
    const at::Tensor &dh = tensor(a[0]), &x = tensor(a[1]), &wg = tensor(a[2]), &wu = tensor(a[3]), &saved = tensor(a[4]);
    const iq_gated_desc d = gated_desc(x, wg, wu, whole(a[5]));
    check(dh, x, at::kBFloat16, {d.tokens, d.features});
    check(saved, x, at::kFloat, {2, d.tokens, d.features});
    at::Tensor dx = make(x, {d.tokens, d.cols}, at::kBFloat16);
    at::Tensor dwg = make(x, {d.features, d.cols}, at::kBFloat16), dwu = make(x, {d.features, d.cols}, at::kBFloat16);
    at::Tensor ws = make(x, {std::max<int64_t>(256, (int64_t)f_gated_workspace_bytes(&d))}, at::kByte);
    need(f_gated_backward(&d, dh.data_ptr(), x.data_ptr(), wg.data_ptr(), wu.data_ptr(), saved.data_ptr(), dx.data_ptr(), dwg.data_ptr(),
                          dwu.data_ptr(), ws.data_ptr(), stream(x)) == IQ_OK);
    return wrap({dx, dwg, dwu});
}

// Packed weights at a[0 .. 2]: codes, scales and global scale (or None).
struct Packed {
    const void *codes, *scales;
    const float* global;
};
Packed packed(PyObject* const* a, const at::Tensor& x, const iq_desc& d) {
    const int64_t group = d.fmt == IQ_INT4 ? 128 : d.fmt == IQ_NVFP4 ? 16 : 32, size = d.fmt == IQ_INT4 ? 2 : 1;
    const at::Tensor& codes = tensor(a[0]);
    need(codes.scalar_type() == at::kByte);
    Packed p = {at_least(codes, x, d.rows * (d.cols / 2)), at_least(tensor(a[1]), x, d.rows * (d.cols / group) * size), nullptr};
    if (d.fmt == IQ_NVFP4) {
        const at::Tensor& g = tensor(a[2]);
        need(g.scalar_type() == at::kFloat);
        p.global = (const float*)at_least(g, x, 4);
    }
    return p;
}
// x, format, rows and cols at a[0 .. 3]
iq_desc packed_desc(PyObject* const* a) {
    const at::Tensor& x = tensor(a[0]);
    check_x(x);
    const iq_desc d = {(int32_t)whole(a[1]), IQ_PER_BLOCK, IQ_BF16, 0, whole(a[2]), whole(a[3]), whole(a[3]), 0, 0};
    need((d.fmt == IQ_INT4 || d.fmt == IQ_NVFP4 || d.fmt == IQ_MXFP4) && d.rows >= 0 && d.rows < (1 << 30) && d.cols >= 0 && d.cols < (1 << 30));
    need(x.scalar_type() == at::kBFloat16 && x.size(1) == d.cols);
    return d;
}

// packed_gemv(x, format, rows, cols, out_f32, codes, scales, global_scale)
PyObject* packed_gemv(PyObject* const* a) {
    const at::Tensor& x = tensor(a[0]);
    const iq_desc d = packed_desc(a);
    const bool f32 = a[4] == Py_True;
    const Packed w = packed(a + 5, x, d);
    at::Tensor z = make(x, {x.size(0), d.rows}, f32 ? at::kFloat : at::kBFloat16);
    need(f_packed_gemv(&d, w.codes, w.scales, w.global, x.data_ptr(), IQ_BF16, x.size(0), z.data_ptr(), f32 ? IQ_F32 : IQ_BF16, stream(x)) == IQ_OK);
    return THPVariable_Wrap(z);
}

// packed_gated(x, format, rows, cols, out_f32, act, codes, scales, global_scale of the gate, ... of up)
PyObject* packed_gated(PyObject* const* a) {
    const at::Tensor& x = tensor(a[0]);
    const iq_desc d = packed_desc(a);
    const bool f32 = a[4] == Py_True;
    const Packed g = packed(a + 6, x, d), u = packed(a + 9, x, d);
    at::Tensor h = make(x, {x.size(0), d.rows}, f32 ? at::kFloat : at::kBFloat16);
    need(f_packed_gated(&d, (int32_t)whole(a[5]), g.codes, g.scales, g.global, u.codes, u.scales, u.global, x.data_ptr(), IQ_BF16, x.size(0),
                        h.data_ptr(), f32 ? IQ_F32 : IQ_BF16, stream(x)) == IQ_OK);
    return THPVariable_Wrap(h);
}

#define IQ_METHOD(name) {#name, (PyCFunction)(void (*)())guarded<name>, METH_FASTCALL, nullptr}
PyMethodDef methods[] = {{"bind", (PyCFunction)(void (*)())bind, METH_FASTCALL, nullptr},
                         IQ_METHOD(layer_norm), IQ_METHOD(layer_norm_backward), IQ_METHOD(gated), IQ_METHOD(gated_backward),
                         IQ_METHOD(packed_gemv), IQ_METHOD(packed_gated), {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_fast", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__fast() { return PyModule_Create(&module); }
