// Python module over the sequence operators' C ABI (include/seq.h): checks of
// tensors, output allocation and the call, in C++ because a call on single
// tokens takes a few microseconds on the GPU and the same checks in Python
// take more than twice that.  It holds no computation.
#include <Python.h>

#include <ATen/core/Tensor.h>
#include <ATen/cuda/EmptyTensor.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include <string>

#include "seq.h"

namespace {

PyObject *g_error = nullptr;   // DgradError(status, where)

// What a plan's calls are checked against.
struct Spec {
    void *plan;
    int device;
    at::ScalarType type, residual;
    int64_t batch, length, channels, inner, groups;   // inner: kernel width or states; rows: batch
    bool gated;
};

[[noreturn]] void refuse(PyObject *kind, const std::string &what) {
    PyErr_SetString(kind, what.c_str());
    throw python_error();
}

std::string shape_text(at::IntArrayRef s) {
    std::string t = "(";
    for (size_t i = 0; i < s.size(); ++i) t += (i ? ", " : "") + std::to_string(s[i]);
    return t + ")";
}

const Spec &spec_of(PyObject *o) {
    void *p = PyCapsule_GetPointer(o, "seq_plan");
    if (!p) throw python_error();
    return *static_cast<const Spec *>(p);
}

const at::Tensor *given(PyObject *o, const char *name) {
    if (o == Py_None) return nullptr;
    if (!THPVariable_Check(o)) refuse(PyExc_TypeError, std::string(name) + " must be a torch.Tensor");
    return &THPVariable_Unpack(o);
}
const at::Tensor &needed(PyObject *o, const char *name) {
    const at::Tensor *t = given(o, name);
    if (!t) refuse(PyExc_TypeError, std::string(name) + " must be a torch.Tensor");
    return *t;
}

void check(const Spec &s, const at::Tensor &t, const char *name, at::IntArrayRef shape, at::ScalarType type) {
    if (t.scalar_type() != type)
        refuse(PyExc_TypeError, std::string(name) + " must be " + c10::toString(type) + ", got " + c10::toString(t.scalar_type()));
    if (t.sizes() != shape)
        refuse(PyExc_ValueError, std::string(name) + " has shape " + shape_text(t.sizes()) + ", expected " + shape_text(shape));
    if (!t.is_cuda() || t.get_device() != s.device)
        refuse(PyExc_ValueError, std::string(name) + " must be on CUDA device " + std::to_string(s.device) + ", the plan's");
}

// A [.., channels] activation.
seq_ref_t act(const Spec &s, const at::Tensor &t, const char *name, at::IntArrayRef shape, at::ScalarType type) {
    check(s, t, name, shape, type);
    const int64_t n = t.dim();
    if (t.stride(n - 1) != 1 && t.size(n - 1) != 1)
        refuse(PyExc_ValueError, std::string(name) + "'s channels must be contiguous");
    return seq_ref_t{t.data_ptr(), t.stride(0), n > 2 ? t.stride(1) : 0, 0};
}
seq_ref_t act(const Spec &s, const at::Tensor *t, const char *name, at::IntArrayRef shape, at::ScalarType type) {
    return t ? act(s, *t, name, shape, type) : seq_ref_t{nullptr, 0, 0, 0};
}

// A [.., groups, states] tensor.
seq_ref_t grouped(const Spec &s, const at::Tensor &t, const char *name, at::IntArrayRef shape) {
    seq_ref_t r = act(s, t, name, shape, s.type);
    const int64_t n = t.dim();
    r.st = n > 3 ? t.stride(1) : 0;
    r.sg = t.stride(n - 2);
    return r;
}

// Address of a contiguous tensor (absent: NULL).
template <typename X = float>
X *flat(const Spec &s, const at::Tensor *t, const char *name, at::IntArrayRef shape, at::ScalarType type = at::kFloat) {
    if (!t) return nullptr;
    check(s, *t, name, shape, type);
    if (!t->is_contiguous()) refuse(PyExc_ValueError, std::string(name) + " must be contiguous");
    return static_cast<X *>(t->data_ptr());
}

at::Tensor make(const Spec &s, at::IntArrayRef shape, at::ScalarType type) {
    return at::Tensor(at::detail::empty_cuda(shape, type, at::Device(at::kCUDA, static_cast<c10::DeviceIndex>(s.device)), c10::nullopt));
}
at::Tensor given_or_made(const Spec &s, PyObject *o, const char *name, at::IntArrayRef shape, at::ScalarType type) {
    const at::Tensor *t = given(o, name);
    return t ? *t : make(s, shape, type);
}

// A tensor that the call has written counts as changed in place, so that
// autograd notices where its backward pass needed the old values.
void written(const at::Tensor &t) {
    if (t.defined() && !t.is_inference()) t.unsafeGetTensorImpl()->bump_version();
}
void written(PyObject *o) {
    if (o != Py_None) written(THPVariable_Unpack(o));
}

void *stream_of(const Spec &s) {
    return c10::cuda::getCurrentCUDAStream(static_cast<c10::DeviceIndex>(s.device)).stream();
}

void settle(int status, const char *where) {
    if (status == DGRAD_OK) return;
    PyObject *e = PyObject_CallFunction(g_error, "is", status, where);
    if (e) {
        PyErr_SetObject(g_error, e);
        Py_DECREF(e);
    }
    throw python_error();
}

void in_plan(const Spec &s, int64_t b, int64_t l) {
    if (b < 1 || b > s.batch || l < 1 || l > s.length)
        refuse(PyExc_ValueError, "batch " + std::to_string(b) + " and length " + std::to_string(l) + " must be within the plan's " +
                                     std::to_string(s.batch) + " and " + std::to_string(s.length));
}
void at_least(const at::Tensor &t, const char *name, int64_t dims) {
    if (t.dim() < dims) refuse(PyExc_ValueError, std::string(name) + " has shape " + shape_text(t.sizes()) + ": too few dimensions");
}

PyObject *wrapped(const at::Tensor &t) {
    if (!t.defined()) Py_RETURN_NONE;
    return THPVariable_Wrap(t);
}
template <typename... X>
PyObject *tuple_of(const X &...t) {
    PyObject *r = PyTuple_New(sizeof...(t));
    if (!r) throw python_error();
    Py_ssize_t i = 0;
    (PyTuple_SET_ITEM(r, i++, wrapped(t)), ...);
    return r;
}

void expect(Py_ssize_t n, Py_ssize_t want) {
    if (n != want) refuse(PyExc_TypeError, "wrong number of arguments");
}

// ------------------------------------------------------------ plans
// open_plan(handle, device, type, residual type, batch, length, channels, inner, groups, gated)
PyObject *open_plan(PyObject *, PyObject *args) {
    long long h, batch, length, channels, inner, groups;
    int device, type, residual, gated;
    if (!PyArg_ParseTuple(args, "LiiiLLLLLp", &h, &device, &type, &residual, &batch, &length, &channels, &inner, &groups, &gated))
        return nullptr;
    static const at::ScalarType types[] = {at::kFloat, at::kHalf, at::kBFloat16};
    Spec *s = new (std::nothrow) Spec{reinterpret_cast<void *>(h), device, types[type], types[residual], batch, length,
                                      channels, inner, groups, gated != 0};
    if (!s) return PyErr_NoMemory();
    return PyCapsule_New(s, "seq_plan", [](PyObject *c) { delete static_cast<Spec *>(PyCapsule_GetPointer(c, "seq_plan")); });
}

PyObject *set_error(PyObject *, PyObject *cls) {
    Py_XDECREF(g_error);
    Py_INCREF(cls);
    g_error = cls;
    Py_RETURN_NONE;
}

// ------------------------------------------------------------ causal convolution
PyObject *conv_run(PyObject *, PyObject *const *a, Py_ssize_t n) {
    HANDLE_TH_ERRORS
    expect(n, 8);   // plan, x, weight, bias, lengths, state, out, final_state
    const Spec &s = spec_of(a[0]);
    const at::Tensor &x = needed(a[1], "x");
    at_least(x, "x", 2);
    const int64_t b = x.size(0), l = x.size(1), d = s.channels, k = s.inner;
    in_plan(s, b, l);
    const int64_t shape[] = {b, l, d}, state[] = {b, k - 1, d}, w[] = {d, k};
    seq_conv_args_t q{};
    q.batch = b;
    q.length = l;
    q.x = act(s, x, "x", shape, s.type);
    const at::Tensor out = given_or_made(s, a[6], "out", shape, s.type);
    q.y = act(s, out, "out", shape, s.type);
    q.weight = flat(s, &needed(a[2], "weight"), "weight", w);
    q.bias = flat(s, given(a[3], "bias"), "bias", {d});
    q.lengths = flat<int>(s, given(a[4], "lengths"), "lengths", {b}, at::kInt);
    q.state = flat<void>(s, given(a[5], "state"), "state", state, s.type);
    q.final_state = flat<void>(s, given(a[7], "final_state"), "final_state", state, s.type);
    settle(seq_conv_run(static_cast<seq_conv_plan_t>(s.plan), &q, stream_of(s)), "seq_conv_run");
    written(a[6]);
    written(a[7]);
    return wrapped(out);
    END_HANDLE_TH_ERRORS
}

PyObject *conv_backward(PyObject *, PyObject *const *a, Py_ssize_t n) {
    HANDLE_TH_ERRORS
    expect(n, 9);   // plan, grad_out, x, weight, bias, lengths, state, grad_final_state, grad_x
    const Spec &s = spec_of(a[0]);
    const at::Tensor &x = needed(a[2], "x");
    at_least(x, "x", 2);
    const int64_t b = x.size(0), l = x.size(1), d = s.channels, k = s.inner;
    in_plan(s, b, l);
    const int64_t shape[] = {b, l, d}, state[] = {b, k - 1, d}, w[] = {d, k};
    const at::Tensor *bias = given(a[4], "bias"), *st = given(a[6], "state");
    seq_conv_grad_args_t q{};
    q.batch = b;
    q.length = l;
    q.grad_y = act(s, needed(a[1], "grad_out"), "grad_out", shape, s.type);
    q.x = act(s, x, "x", shape, s.type);
    q.weight = flat(s, &needed(a[3], "weight"), "weight", w);
    q.bias = flat(s, bias, "bias", {d});
    q.lengths = flat<int>(s, given(a[5], "lengths"), "lengths", {b}, at::kInt);
    q.state = flat<void>(s, st, "state", state, s.type);
    q.grad_final = flat<void>(s, given(a[7], "grad_final_state"), "grad_final_state", state, s.type);
    const at::Tensor gx = given_or_made(s, a[8], "grad_x", shape, s.type);
    q.grad_x = act(s, gx, "grad_x", shape, s.type);
    const at::Tensor gw = make(s, w, at::kFloat);
    const at::Tensor gb = bias ? make(s, {d}, at::kFloat) : at::Tensor(), gs = st ? make(s, state, s.type) : at::Tensor();
    q.grad_weight = gw.data_ptr<float>();
    q.grad_bias = bias ? gb.data_ptr<float>() : nullptr;
    q.grad_state = st ? gs.data_ptr() : nullptr;
    settle(seq_conv_backward(static_cast<seq_conv_plan_t>(s.plan), &q, stream_of(s)), "seq_conv_backward");
    written(a[8]);
    return tuple_of(gx, gw, gb, gs);
    END_HANDLE_TH_ERRORS
}

PyObject *conv_step(PyObject *, PyObject *const *a, Py_ssize_t n) {
    HANDLE_TH_ERRORS
    expect(n, 8);   // plan, x, weight, cache, bias, slots, write_slots, out
    const Spec &s = spec_of(a[0]);
    const at::Tensor &x = needed(a[1], "x"), &cache = needed(a[3], "cache");
    at_least(x, "x", 1);
    at_least(cache, "cache", 1);
    const int64_t b = x.size(0), d = s.channels, k = s.inner;
    in_plan(s, b, 1);
    const int64_t shape[] = {b, d}, w[] = {d, k}, slots[] = {cache.size(0), k - 1, d};
    seq_conv_step_args_t q{};
    q.batch = b;
    q.n_slots = cache.size(0);
    q.x = act(s, x, "x", shape, s.type);
    const at::Tensor out = given_or_made(s, a[7], "out", shape, s.type);
    q.y = act(s, out, "out", shape, s.type);
    q.weight = flat(s, &needed(a[2], "weight"), "weight", w);
    q.bias = flat(s, given(a[4], "bias"), "bias", {d});
    q.cache = flat<void>(s, &cache, "cache", slots, s.type);
    q.slots = flat<int>(s, given(a[5], "slots"), "slots", {b}, at::kInt);
    q.write_slots = flat<int>(s, given(a[6], "write_slots"), "write_slots", {b}, at::kInt);
    settle(seq_conv_step(static_cast<seq_conv_plan_t>(s.plan), &q, stream_of(s)), "seq_conv_step");
    written(cache);
    written(a[7]);
    return wrapped(out);
    END_HANDLE_TH_ERRORS
}

// ------------------------------------------------------------ selective scan
float *checkpoints_of(const Spec &s, const at::Tensor *t, int64_t b, int64_t l) {
    if (!t) return nullptr;
    const int64_t want = static_cast<int64_t>(seq_scan_checkpoint_bytes(static_cast<seq_scan_plan_t>(s.plan), b, l) / 4);
    if (t->scalar_type() != at::kFloat || !t->is_contiguous() || !t->is_cuda() || t->get_device() != s.device)
        refuse(PyExc_ValueError, "checkpoints must be a contiguous float32 tensor on the plan's device");
    if (t->numel() < want)
        refuse(PyExc_ValueError, "checkpoints has " + std::to_string(t->numel()) + " elements, this batch needs " + std::to_string(want));
    return t->data_ptr<float>();
}

// scan_checkpoints(plan, batch or None, length or None)
PyObject *scan_checkpoints(PyObject *, PyObject *const *a, Py_ssize_t n) {
    HANDLE_TH_ERRORS
    expect(n, 3);
    const Spec &s = spec_of(a[0]);
    int64_t size[2] = {s.batch, s.length};
    for (int i = 0; i < 2; ++i) {
        if (a[1 + i] == Py_None) continue;
        size[i] = PyLong_AsLongLong(a[1 + i]);
        if (size[i] == -1 && PyErr_Occurred()) throw python_error();
    }
    in_plan(s, size[0], size[1]);
    const size_t bytes = seq_scan_checkpoint_bytes(static_cast<seq_scan_plan_t>(s.plan), size[0], size[1]);
    return wrapped(make(s, {static_cast<int64_t>(bytes / 4)}, at::kFloat));
    END_HANDLE_TH_ERRORS
}

PyObject *scan_run(PyObject *, PyObject *const *a, Py_ssize_t n) {
    HANDLE_TH_ERRORS
    expect(n, 14);   // plan, u, dt, A, B, C, D, z, dt_bias, lengths, state, out, final_state, checkpoints
    const Spec &s = spec_of(a[0]);
    const at::Tensor &u = needed(a[1], "u");
    at_least(u, "u", 2);
    const int64_t b = u.size(0), l = u.size(1), d = s.channels, m = s.inner;
    in_plan(s, b, l);
    const int64_t shape[] = {b, l, d}, bc[] = {b, l, s.groups, m}, state[] = {b, d, m}, dn[] = {d, m};
    seq_scan_args_t q{};
    q.batch = b;
    q.length = l;
    q.u = act(s, u, "u", shape, s.type);
    q.dt = act(s, needed(a[2], "dt"), "dt", shape, s.type);
    q.B = grouped(s, needed(a[4], "B"), "B", bc);
    q.C = grouped(s, needed(a[5], "C"), "C", bc);
    q.z = act(s, given(a[7], "z"), "z", shape, s.type);
    const at::Tensor out = given_or_made(s, a[11], "out", shape, s.type);
    q.out = act(s, out, "out", shape, s.type);
    q.A = flat(s, &needed(a[3], "A"), "A", dn);
    q.D = flat(s, given(a[6], "D"), "D", {d});
    q.dt_bias = flat(s, given(a[8], "dt_bias"), "dt_bias", {d});
    q.lengths = flat<int>(s, given(a[9], "lengths"), "lengths", {b}, at::kInt);
    q.state = flat(s, given(a[10], "state"), "state", state);
    q.final_state = flat(s, given(a[12], "final_state"), "final_state", state);
    q.checkpoints = checkpoints_of(s, given(a[13], "checkpoints"), b, l);
    settle(seq_scan_run(static_cast<seq_scan_plan_t>(s.plan), &q, stream_of(s)), "seq_scan_run");
    written(a[11]);
    written(a[12]);
    written(a[13]);
    return wrapped(out);
    END_HANDLE_TH_ERRORS
}

PyObject *scan_backward(PyObject *, PyObject *const *a, Py_ssize_t n) {
    HANDLE_TH_ERRORS
    // plan, grad_out, u, dt, A, B, C, checkpoints, D, z, dt_bias, lengths, state, grad_final_state, grad_u, grad_z
    expect(n, 16);
    const Spec &s = spec_of(a[0]);
    const at::Tensor &u = needed(a[2], "u");
    at_least(u, "u", 2);
    const int64_t b = u.size(0), l = u.size(1), d = s.channels, m = s.inner;
    in_plan(s, b, l);
    const int64_t shape[] = {b, l, d}, bc[] = {b, l, s.groups, m}, state[] = {b, d, m}, dn[] = {d, m};
    const at::Tensor *D = given(a[8], "D"), *z = given(a[9], "z"), *bias = given(a[10], "dt_bias"), *st = given(a[12], "state");
    if (a[7] == Py_None) refuse(PyExc_ValueError, "backward needs the checkpoints that run filled");
    if (!z && a[15] != Py_None) refuse(PyExc_ValueError, "grad_z needs z");
    seq_scan_grad_args_t q{};
    q.batch = b;
    q.length = l;
    q.grad_out = act(s, needed(a[1], "grad_out"), "grad_out", shape, s.type);
    q.u = act(s, u, "u", shape, s.type);
    q.dt = act(s, needed(a[3], "dt"), "dt", shape, s.type);
    q.B = grouped(s, needed(a[5], "B"), "B", bc);
    q.C = grouped(s, needed(a[6], "C"), "C", bc);
    q.z = act(s, z, "z", shape, s.type);
    q.A = flat(s, &needed(a[4], "A"), "A", dn);
    q.D = flat(s, D, "D", {d});
    q.dt_bias = flat(s, bias, "dt_bias", {d});
    q.lengths = flat<int>(s, given(a[11], "lengths"), "lengths", {b}, at::kInt);
    q.state = flat(s, st, "state", state);
    q.checkpoints = checkpoints_of(s, given(a[7], "checkpoints"), b, l);
    q.grad_final = flat(s, given(a[13], "grad_final_state"), "grad_final_state", state);
    const at::Tensor gu = given_or_made(s, a[14], "grad_u", shape, s.type);
    const at::Tensor gz = z ? given_or_made(s, a[15], "grad_z", shape, s.type) : at::Tensor();
    const at::Tensor gdt = make(s, shape, s.type), gB = make(s, bc, s.type), gC = make(s, bc, s.type), gA = make(s, dn, at::kFloat);
    const at::Tensor gD = D ? make(s, {d}, at::kFloat) : at::Tensor(), gb = bias ? make(s, {d}, at::kFloat) : at::Tensor();
    const at::Tensor gs = st ? make(s, state, at::kFloat) : at::Tensor();
    q.grad_u = act(s, gu, "grad_u", shape, s.type);
    q.grad_dt = act(s, gdt, "grad_dt", shape, s.type);
    q.grad_B = grouped(s, gB, "grad_B", bc);
    q.grad_C = grouped(s, gC, "grad_C", bc);
    if (z) q.grad_z = act(s, gz, "grad_z", shape, s.type);
    q.grad_A = gA.data_ptr<float>();
    q.grad_D = D ? gD.data_ptr<float>() : nullptr;
    q.grad_dt_bias = bias ? gb.data_ptr<float>() : nullptr;
    q.grad_state = st ? gs.data_ptr<float>() : nullptr;
    settle(seq_scan_backward(static_cast<seq_scan_plan_t>(s.plan), &q, stream_of(s)), "seq_scan_backward");
    written(a[14]);
    written(a[15]);
    return tuple_of(gu, gdt, gA, gB, gC, gD, gz, gb, gs);
    END_HANDLE_TH_ERRORS
}

PyObject *scan_step(PyObject *, PyObject *const *a, Py_ssize_t n) {
    HANDLE_TH_ERRORS
    expect(n, 13);   // plan, u, dt, A, B, C, cache, D, z, dt_bias, slots, write_slots, out
    const Spec &s = spec_of(a[0]);
    const at::Tensor &u = needed(a[1], "u"), &cache = needed(a[6], "cache");
    at_least(u, "u", 1);
    at_least(cache, "cache", 1);
    const int64_t b = u.size(0), d = s.channels, m = s.inner;
    in_plan(s, b, 1);
    const int64_t shape[] = {b, d}, bc[] = {b, s.groups, m}, slots[] = {cache.size(0), d, m}, dn[] = {d, m};
    seq_scan_step_args_t q{};
    q.batch = b;
    q.n_slots = cache.size(0);
    q.u = act(s, u, "u", shape, s.type);
    q.dt = act(s, needed(a[2], "dt"), "dt", shape, s.type);
    q.B = grouped(s, needed(a[4], "B"), "B", bc);
    q.C = grouped(s, needed(a[5], "C"), "C", bc);
    q.z = act(s, given(a[8], "z"), "z", shape, s.type);
    const at::Tensor out = given_or_made(s, a[12], "out", shape, s.type);
    q.out = act(s, out, "out", shape, s.type);
    q.A = flat(s, &needed(a[3], "A"), "A", dn);
    q.D = flat(s, given(a[7], "D"), "D", {d});
    q.dt_bias = flat(s, given(a[9], "dt_bias"), "dt_bias", {d});
    q.cache = flat(s, &cache, "cache", slots);
    q.slots = flat<int>(s, given(a[10], "slots"), "slots", {b}, at::kInt);
    q.write_slots = flat<int>(s, given(a[11], "write_slots"), "write_slots", {b}, at::kInt);
    settle(seq_scan_step(static_cast<seq_scan_plan_t>(s.plan), &q, stream_of(s)), "seq_scan_step");
    written(cache);
    written(a[12]);
    return wrapped(out);
    END_HANDLE_TH_ERRORS
}

// ------------------------------------------------------------ block norm
int64_t rows_of(const Spec &s, const at::Tensor &y, PyObject *gate) {
    at_least(y, "y", 1);
    const int64_t n = y.size(0);
    if (n < 1 || n > s.batch)
        refuse(PyExc_ValueError, std::to_string(n) + " rows must be within the plan's " + std::to_string(s.batch));
    if ((gate != Py_None) != s.gated) refuse(PyExc_ValueError, "gate must be given exactly if the plan has a gate");
    return n;
}

PyObject *norm_run(PyObject *, PyObject *const *a, Py_ssize_t n) {
    HANDLE_TH_ERRORS
    expect(n, 9);   // plan, y, residual, next_weight, post_weight, gate, scale, residual_out, out
    const Spec &s = spec_of(a[0]);
    const at::Tensor &y = needed(a[1], "y");
    const int64_t d = s.channels, rows = rows_of(s, y, a[5]), shape[] = {rows, d};
    seq_norm_args_t q{};
    q.rows = rows;
    q.y = act(s, y, "y", shape, s.type);
    q.gate = act(s, given(a[5], "gate"), "gate", shape, s.type);
    q.residual = act(s, needed(a[2], "residual"), "residual", shape, s.residual);
    const at::Tensor r = given_or_made(s, a[7], "residual_out", shape, s.residual);
    const at::Tensor out = given_or_made(s, a[8], "out", shape, s.type);
    q.residual_out = act(s, r, "residual_out", shape, s.residual);
    q.x = act(s, out, "out", shape, s.type);
    q.post_weight = flat(s, given(a[4], "post_weight"), "post_weight", {d});
    q.scale = flat(s, given(a[6], "scale"), "scale", {d});
    q.next_weight = flat(s, &needed(a[3], "next_weight"), "next_weight", {d});
    settle(seq_norm_run(static_cast<seq_norm_plan_t>(s.plan), &q, stream_of(s)), "seq_norm_run");
    written(a[7]);
    written(a[8]);
    return tuple_of(r, out);
    END_HANDLE_TH_ERRORS
}

PyObject *norm_backward(PyObject *, PyObject *const *a, Py_ssize_t n) {
    HANDLE_TH_ERRORS
    // plan, grad_residual_out, grad_out, y, residual, next_weight, post_weight, gate, scale, grad_y, grad_gate, grad_residual
    expect(n, 12);
    const Spec &s = spec_of(a[0]);
    const at::Tensor &y = needed(a[3], "y");
    const int64_t d = s.channels, rows = rows_of(s, y, a[7]), shape[] = {rows, d};
    if (!s.gated && a[10] != Py_None) refuse(PyExc_ValueError, "grad_gate needs a gate");
    const at::Tensor *post = given(a[6], "post_weight"), *scale = given(a[8], "scale");
    seq_norm_grad_args_t q{};
    q.rows = rows;
    q.y = act(s, y, "y", shape, s.type);
    q.gate = act(s, given(a[7], "gate"), "gate", shape, s.type);
    q.residual = act(s, needed(a[4], "residual"), "residual", shape, s.residual);
    q.grad_residual_out = act(s, given(a[1], "grad_residual_out"), "grad_residual_out", shape, s.residual);
    q.grad_x = act(s, needed(a[2], "grad_out"), "grad_out", shape, s.type);
    const at::Tensor gy = given_or_made(s, a[9], "grad_y", shape, s.type);
    const at::Tensor gg = s.gated ? given_or_made(s, a[10], "grad_gate", shape, s.type) : at::Tensor();
    const at::Tensor gr = given_or_made(s, a[11], "grad_residual", shape, s.residual);
    const at::Tensor gp = post ? make(s, {d}, at::kFloat) : at::Tensor(), gs = scale ? make(s, {d}, at::kFloat) : at::Tensor();
    const at::Tensor gn = make(s, {d}, at::kFloat);
    q.grad_y = act(s, gy, "grad_y", shape, s.type);
    if (s.gated) q.grad_gate = act(s, gg, "grad_gate", shape, s.type);
    q.grad_residual = act(s, gr, "grad_residual", shape, s.residual);
    q.post_weight = flat(s, post, "post_weight", {d});
    q.scale = flat(s, scale, "scale", {d});
    q.next_weight = flat(s, &needed(a[5], "next_weight"), "next_weight", {d});
    q.grad_post_weight = post ? gp.data_ptr<float>() : nullptr;
    q.grad_scale = scale ? gs.data_ptr<float>() : nullptr;
    q.grad_next_weight = gn.data_ptr<float>();
    settle(seq_norm_backward(static_cast<seq_norm_plan_t>(s.plan), &q, stream_of(s)), "seq_norm_backward");
    written(a[9]);
    written(a[10]);
    written(a[11]);
    return tuple_of(gy, gg, gr, gp, gs, gn);
    END_HANDLE_TH_ERRORS
}

#define FAST(name) {#name, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)(void)>(name)), METH_FASTCALL, nullptr}
PyMethodDef methods[] = {{"open_plan", open_plan, METH_VARARGS, nullptr},
                         {"set_error", set_error, METH_O, nullptr},
                         FAST(conv_run), FAST(conv_backward), FAST(conv_step),
                         FAST(scan_checkpoints), FAST(scan_run), FAST(scan_backward), FAST(scan_step),
                         FAST(norm_run), FAST(norm_backward),
                         {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_seq_bind", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__seq_bind(void) { return PyModule_Create(&module); }
