// Short cut of the Python binding for the layer operators' usual calls (module _calls): plain contiguous tensors on the
// current device, on the current stream.  It checks that a call is one of those, allocates the outputs and calls the C
// ABI; anything else, every refusal among it, it leaves to the checked functions of binding.py by returning None.
// Those calls take a few microseconds on the device, and the same steps in Python some ten on the host
// (gla_step of one sequence and 8 heads: 17 us a call by ctypes, against 2.6 us of GPU time).
#include <Python.h>

#include <ATen/ops/empty.h>
#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/Dtype.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include "gla.h"

namespace {

constexpr int kDevices = 128;
constexpr size_t kStatusBytes = 256;

// The library's own status workspace on the current device, or nullptr.
void *status(int device)
{
    static void *known[kDevices] = {};   // the interpreter's lock is held
    if (!known[device])
        known[device] = gla_scan_shared_workspace();
    return known[device];
}

// One call's tensors: whether all of them are usual.
struct Call {
    bool ok = true;
    int device = -1;

    // A tensor argument (nullptr for None): plain, contiguous, on the first one's device.
    const at::Tensor *take(PyObject *o, bool optional = false)
    {
        if (o == Py_None && optional)
            return nullptr;
        if (!THPVariable_CheckExact(o)) {
            ok = false;
            return nullptr;
        }
        const at::Tensor &t = THPVariable_Unpack(o);
        if (t.layout() != at::kStrided || !t.is_cuda() || !t.is_contiguous() ||
            (device >= 0 && t.get_device() != device)) {
            ok = false;
            return nullptr;
        }
        if (device < 0) {
            device = t.get_device();
            if (device >= kDevices || c10::cuda::current_device() != device)
                ok = false;
        }
        return &t;
    }
    void need(bool that) { ok = ok && that; }
    void like(const at::Tensor *t, const at::Tensor &shape, at::ScalarType type)
    {
        if (t)
            need(t->scalar_type() == type && t->sizes() == shape.sizes());
    }
    void shaped(const at::Tensor *t, at::IntArrayRef sizes, at::ScalarType type)
    {
        if (t)
            need(t->scalar_type() == type && t->sizes() == sizes);
    }
    void *stream() const { return c10::cuda::getCurrentCUDAStream((c10::DeviceIndex)device).stream(); }
};

at::ScalarType dtype_or(PyObject *o, at::ScalarType otherwise, Call &c)
{
    if (o == Py_None)
        return otherwise;
    if (!THPDtype_Check(o)) {
        c.ok = false;
        return otherwise;
    }
    return reinterpret_cast<THPDtype *>(o)->scalar_type;
}

// The dtype code of (x, gate, output) types, or -1.
int scan_code(at::ScalarType x, at::ScalarType g, at::ScalarType o)
{
    const auto f = at::kFloat, b = at::kBFloat16, h = at::kHalf;
    if (x == f && g == f && o == f) return GLA_F32;
    if (x == b && g == b) return o == f ? GLA_BF16 : o == b ? GLA_BF16_OBF16 : -1;
    if (x == h && g == h) return o == f ? GLA_F16 : o == h ? GLA_F16_OF16 : -1;
    if (g == f && o == f) return x == b ? GLA_BF16_GF32 : x == h ? GLA_F16_GF32 : -1;
    return -1;
}

int norm_code(at::ScalarType x, at::ScalarType r)
{
    const int code = x == at::kFloat ? GLA_F32 : x == at::kBFloat16 ? GLA_BF16 : x == at::kHalf ? GLA_F16 : -1;
    return code < 0 || (r != x && r != at::kFloat) ? -1 : r == x ? code : code | GLA_RES_F32;
}

at::Tensor empty(at::IntArrayRef sizes, const at::Tensor &like, at::ScalarType type)
{
    return at::empty(sizes, at::TensorOptions().dtype(type).device(like.device()));
}

void *at_of(const at::Tensor *t) { return t ? t->data_ptr() : nullptr; }
float *floats(const at::Tensor *t) { return static_cast<float *>(at_of(t)); }
int32_t *ints(const at::Tensor *t) { return static_cast<int32_t *>(at_of(t)); }

PyObject *none() { Py_RETURN_NONE; }
PyObject *wrap(at::Tensor t) { return t.defined() ? THPVariable_Wrap(std::move(t)) : none(); }

// A tuple of outputs (undefined ones as None).
template <typename... T>
PyObject *tuple_of(T... t)
{
    PyObject *items[] = {wrap(std::move(t))...};
    PyObject *out = PyTuple_New(sizeof...(T));
    for (size_t i = 0; i < sizeof...(T); ++i) {
        if (!out || !items[i]) {
            for (size_t j = i; j < sizeof...(T); ++j)
                Py_XDECREF(items[j]);
            Py_XDECREF(out);
            return nullptr;
        }
        PyTuple_SET_ITEM(out, i, items[i]);
    }
    return out;
}

// Sequences of a recurrence over [B, T, D].
int sequences(Call &c, const at::Tensor &x, const at::Tensor *cu)
{
    c.need(x.dim() == 3 && x.size(0) <= INT32_MAX && x.size(1) <= INT32_MAX && x.size(2) <= INT32_MAX);
    if (!c.ok || !cu)
        return c.ok ? (int)x.size(0) : 0;
    c.need(cu->scalar_type() == at::kInt && cu->dim() == 1 && cu->numel() >= 1 && cu->numel() <= INT32_MAX);
    return c.ok ? (int)cu->numel() - 1 : 0;
}

// scan_fwd(x, g, initial_state, output_final_state, cu_seqlens, out_dtype)
PyObject *scan_fwd(PyObject *, PyObject *const *a, Py_ssize_t n)
{
    HANDLE_TH_ERRORS
    Call c;
    if (n != 6)
        return none();
    const at::Tensor *x = c.take(a[0]), *g = c.take(a[1]), *h0 = c.take(a[2], true), *cu = c.take(a[4], true);
    if (!c.ok)
        return none();
    const at::ScalarType type = dtype_or(a[5], g->scalar_type(), c);
    const int code = scan_code(x->scalar_type(), g->scalar_type(), type), N = sequences(c, *x, cu);
    c.need(code >= 0 && g->sizes() == x->sizes() && status(c.device));
    if (!c.ok)
        return none();
    const int64_t D = x->size(2);
    c.shaped(h0, {N, D}, at::kFloat);
    if (!c.ok)
        return none();
    at::Tensor h = empty(x->sizes(), *x, type), ht;
    if (PyObject_IsTrue(a[3]))
        ht = empty({N, D}, *x, at::kFloat);
    const int rc = gla_scan_fwd(x->data_ptr(), g->data_ptr(), h.data_ptr(), floats(h0), ht.defined() ? floats(&ht) : nullptr,
                                ints(cu), N, (int)x->size(0), (int)x->size(1), (int)D, D, D, code, status(c.device),
                                kStatusBytes, c.stream());
    return rc == GLA_OK ? tuple_of(std::move(h), std::move(ht)) : none();
    END_HANDLE_TH_ERRORS
}

// scan_bwd(g, h, dh, initial_state, dht, cu_seqlens, dx_dtype, want_dh0)
PyObject *scan_bwd(PyObject *, PyObject *const *a, Py_ssize_t n)
{
    HANDLE_TH_ERRORS
    Call c;
    if (n != 8)
        return none();
    const at::Tensor *g = c.take(a[0]), *h = c.take(a[1]), *dh = c.take(a[2]), *h0 = c.take(a[3], true),
                     *dht = c.take(a[4], true), *cu = c.take(a[5], true);
    if (!c.ok)
        return none();
    const at::ScalarType type = dtype_or(a[6], g->scalar_type(), c);
    const int code = scan_code(type, g->scalar_type(), h->scalar_type()), N = sequences(c, *g, cu);
    c.need(code >= 0 && h->sizes() == g->sizes() && status(c.device));
    c.like(dh, *g, h->scalar_type());
    if (!c.ok)
        return none();
    const int64_t D = g->size(2);
    c.shaped(h0, {N, D}, at::kFloat);
    c.shaped(dht, {N, D}, at::kFloat);
    if (!c.ok)
        return none();
    at::Tensor dx = empty(g->sizes(), *g, type), dg = empty(g->sizes(), *g, g->scalar_type()), dh0;
    if (PyObject_IsTrue(a[7]))
        dh0 = empty({N, D}, *g, at::kFloat);
    const int rc = gla_scan_bwd(g->data_ptr(), h->data_ptr(), dh->data_ptr(), floats(h0), floats(dht), dx.data_ptr(),
                                dg.data_ptr(), dh0.defined() ? floats(&dh0) : nullptr, ints(cu), N, (int)g->size(0),
                                (int)g->size(1), (int)D, D, D, D, code, status(c.device), kStatusBytes, c.stream());
    return rc == GLA_OK ? tuple_of(std::move(dx), std::move(dg), std::move(dh0)) : none();
    END_HANDLE_TH_ERRORS
}

// The state pools of a one-token update; the rows of one, or -1.
int64_t pool(Call &c, const at::Tensor *state, const at::Tensor *out, const at::Tensor *slots, int64_t B,
             at::IntArrayRef tail)
{
    c.need(state->scalar_type() == at::kFloat && state->dim() == (int64_t)tail.size() + 1 &&
           state->sizes().slice(1) == tail && state->size(0) <= INT32_MAX && B <= INT32_MAX);
    if (!c.ok)
        return -1;
    c.like(out, *state, at::kFloat);
    if (slots)
        c.shaped(slots, {B}, at::kInt);
    else
        c.need(state->size(0) == B);
    c.need(status(c.device));
    return state->size(0);
}

// scan_step(x, g, state, slots, state_out, out_dtype)
PyObject *scan_step(PyObject *, PyObject *const *a, Py_ssize_t n)
{
    HANDLE_TH_ERRORS
    Call c;
    if (n != 6)
        return none();
    const at::Tensor *x = c.take(a[0]), *g = c.take(a[1]), *state = c.take(a[2]), *slots = c.take(a[3], true),
                     *out = c.take(a[4], true);
    if (!c.ok)
        return none();
    const at::ScalarType type = dtype_or(a[5], g->scalar_type(), c);
    const int code = scan_code(x->scalar_type(), g->scalar_type(), type);
    c.need(code >= 0 && x->dim() == 2 && g->sizes() == x->sizes() && x->size(1) <= INT32_MAX);
    if (!c.ok)
        return none();
    const int64_t B = x->size(0), D = x->size(1), S = pool(c, state, out, slots, B, {D});
    if (!c.ok)
        return none();
    at::Tensor h = empty(x->sizes(), *x, type);
    const int rc = gla_scan_step(x->data_ptr(), g->data_ptr(), h.data_ptr(), floats(state), floats(out ? out : state),
                                 ints(slots), (int)B, (int)S, (int)D, D, D, code, status(c.device), kStatusBytes,
                                 c.stream());
    return rc == GLA_OK ? wrap(std::move(h)) : none();
    END_HANDLE_TH_ERRORS
}

// gla_step(q, k, v, g, state, scale, slots, state_out, out_dtype)
PyObject *step(PyObject *, PyObject *const *a, Py_ssize_t n)
{
    HANDLE_TH_ERRORS
    Call c;
    if (n != 9)
        return none();
    const at::Tensor *q = c.take(a[0]), *k = c.take(a[1]), *v = c.take(a[2]), *g = c.take(a[3]), *state = c.take(a[4]),
                     *slots = c.take(a[6], true), *out = c.take(a[7], true);
    if (!c.ok)
        return none();
    const at::ScalarType type = dtype_or(a[8], at::kFloat, c);
    const int code = scan_code(q->scalar_type(), g->scalar_type(), type);
    c.need(code >= 0 && q->dim() == 3 && v->dim() == 3 && g->sizes() == q->sizes() && v->size(0) == q->size(0) &&
           v->size(1) == q->size(1) && v->scalar_type() == q->scalar_type());
    c.like(k, *q, q->scalar_type());
    if (!c.ok)
        return none();
    const int64_t B = q->size(0), H = q->size(1), K = q->size(2), V = v->size(2);
    const int64_t S = pool(c, state, out, slots, B, {H, K, V});
    const double scale = a[5] == Py_None ? 1.0 / std::sqrt((double)K) : PyFloat_Check(a[5]) ? PyFloat_AS_DOUBLE(a[5]) : -1;
    c.need(scale > 0 && H <= INT32_MAX && K <= INT32_MAX && V <= INT32_MAX);
    if (!c.ok)
        return none();
    at::Tensor o = empty({B, H, V}, *q, type);
    const int rc = gla_step(q->data_ptr(), k->data_ptr(), v->data_ptr(), g->data_ptr(), o.data_ptr(), (float)scale,
                            floats(state), floats(out ? out : state), ints(slots), (int)B, (int)S, (int)H, (int)K, (int)V,
                            code, status(c.device), kStatusBytes, c.stream());
    return rc == GLA_OK ? wrap(std::move(o)) : none();
    END_HANDLE_TH_ERRORS
}

// A norm's operands: its code (or -1), columns and rows.
struct Norm {
    int code = -1;
    int64_t D = 0, rows = 0;
};
Norm norm(Call &c, const at::Tensor *x, const at::Tensor *res, const at::Tensor *w)
{
    Norm r;
    r.code = norm_code(x->scalar_type(), res ? res->scalar_type() : x->scalar_type());
    c.need(r.code >= 0 && x->dim() >= 1 && x->size(-1) >= 1 && x->size(-1) <= INT32_MAX);
    if (!c.ok)
        return r;
    r.D = x->size(-1);
    r.rows = x->numel() / r.D;
    if (res)
        c.need(res->sizes() == x->sizes());
    c.shaped(w, {r.D}, at::kFloat);
    return r;
}

double number(PyObject *o, Call &c)
{
    c.need(PyFloat_Check(o));
    return c.ok ? PyFloat_AS_DOUBLE(o) : 0.0;
}

// norm_fwd(x, residual, weight, eps)
PyObject *norm_fwd(PyObject *, PyObject *const *a, Py_ssize_t n)
{
    HANDLE_TH_ERRORS
    Call c;
    if (n != 4)
        return none();
    const at::Tensor *x = c.take(a[0]), *res = c.take(a[1], true), *w = c.take(a[2], true);
    const double eps = number(a[3], c);
    if (!c.ok)
        return none();
    const Norm m = norm(c, x, res, w);
    if (!c.ok)
        return none();
    at::Tensor y = empty(x->sizes(), *x, x->scalar_type()), s;
    if (res)
        s = empty(x->sizes(), *x, res->scalar_type());
    at::Tensor rstd = empty(x->sizes().slice(0, x->dim() - 1), *x, at::kFloat);
    const int rc = gla_norm_fwd(x->data_ptr(), at_of(res), floats(w), y.data_ptr(), res ? s.data_ptr() : nullptr,
                                floats(&rstd), m.rows, (int)m.D, (float)eps, m.code, c.stream());
    return rc == GLA_OK ? tuple_of(std::move(y), res ? std::move(s) : *x, std::move(rstd)) : none();
    END_HANDLE_TH_ERRORS
}

// norm_quant_fwd(x, residual, weight, eps, group)
PyObject *norm_quant_fwd(PyObject *, PyObject *const *a, Py_ssize_t n)
{
    HANDLE_TH_ERRORS
    Call c;
    if (n != 5)
        return none();
    const at::Tensor *x = c.take(a[0]), *res = c.take(a[1], true), *w = c.take(a[2], true);
    const double eps = number(a[3], c);
    const long group = PyLong_Check(a[4]) ? PyLong_AsLong(a[4]) : -1;
    c.need(group == 0 || group == 128);
    if (PyErr_Occurred())
        PyErr_Clear();
    if (!c.ok)
        return none();
    const Norm m = norm(c, x, res, w);
    if (!c.ok)
        return none();
    at::Tensor q = empty(x->sizes(), *x, at::kFloat8_e4m3fn), s;
    if (res)
        s = empty(x->sizes(), *x, res->scalar_type());
    c10::SmallVector<int64_t, 5> sizes(x->sizes().begin(), x->sizes().end());
    at::Tensor rstd = empty(x->sizes().slice(0, x->dim() - 1), *x, at::kFloat);
    sizes.back() = group ? (m.D + group - 1) / group : 1;
    at::Tensor scales = empty(sizes, *x, at::kFloat);
    const int rc = gla_norm_quant_fwd(x->data_ptr(), at_of(res), floats(w), q.data_ptr(), floats(&scales),
                                      res ? s.data_ptr() : nullptr, floats(&rstd), m.rows, (int)m.D, (float)eps, (int)group,
                                      m.code, c.stream());
    return rc == GLA_OK ? tuple_of(std::move(q), std::move(scales), res ? std::move(s) : *x, std::move(rstd)) : none();
    END_HANDLE_TH_ERRORS
}

// norm_bwd(s, rstd, dy, weight, ds, want_dw, workspace or None)
PyObject *norm_bwd(PyObject *, PyObject *const *a, Py_ssize_t n)
{
    HANDLE_TH_ERRORS
    Call c;
    if (n != 7)
        return none();
    const at::Tensor *s = c.take(a[0]), *rstd = c.take(a[1]), *dy = c.take(a[2]), *w = c.take(a[3], true),
                     *ds = c.take(a[4], true), *given = c.take(a[6], true);
    if (!c.ok)
        return none();
    const Norm m = norm(c, dy, s, w);
    if (!c.ok)
        return none();
    c.like(ds, *s, s->scalar_type());
    c.shaped(rstd, s->sizes().slice(0, s->dim() - 1), at::kFloat);
    if (!c.ok)
        return none();
    at::Tensor dx = empty(dy->sizes(), *dy, dy->scalar_type()), dres, dw;
    const bool same = s->scalar_type() == dy->scalar_type();
    if (!same)
        dres = empty(s->sizes(), *s, s->scalar_type());
    if (w && PyObject_IsTrue(a[5]))
        dw = empty({m.D}, *s, at::kFloat);
    // the partial sums' memory is this call's own, as another thread may be between its two launches on this stream
    const at::Tensor ws = given ? *given : empty({(int64_t)gla_norm_bwd_workspace_size(m.rows, (int)m.D)}, *s, at::kByte);
    const int rc = gla_norm_bwd(s->data_ptr(), floats(rstd), floats(w), dy->data_ptr(), at_of(ds), dx.data_ptr(),
                                same ? nullptr : dres.data_ptr(), dw.defined() ? floats(&dw) : nullptr, m.rows, (int)m.D,
                                m.code, ws.data_ptr(), (size_t)ws.numel() * ws.element_size(), c.stream());
    if (rc != GLA_OK)
        return none();
    PyObject *first = wrap(dx), *second = nullptr, *third = first ? wrap(std::move(dw)) : nullptr;
    if (third)
        second = same ? Py_NewRef(first) : wrap(std::move(dres));
    PyObject *out = second ? PyTuple_Pack(3, first, second, third) : nullptr;
    Py_XDECREF(first);
    Py_XDECREF(second);
    Py_XDECREF(third);
    return out;
    END_HANDLE_TH_ERRORS
}

#define CALL(name, f) {name, reinterpret_cast<PyCFunction>(reinterpret_cast<void *>(f)), METH_FASTCALL, nullptr}
PyMethodDef methods[] = {CALL("scan_fwd", scan_fwd), CALL("scan_bwd", scan_bwd), CALL("scan_step", scan_step),
                         CALL("gla_step", step), CALL("norm_fwd", norm_fwd), CALL("norm_quant_fwd", norm_quant_fwd),
                         CALL("norm_bwd", norm_bwd), {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_calls", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__calls() { return PyModule_Create(&module); }
