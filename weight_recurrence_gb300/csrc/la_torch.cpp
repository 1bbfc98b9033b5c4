// la_torch.cpp - the Python binding of the operators around the attention:
// checks of shapes, types and devices, views, and the memory that a call
// returns or needs, on the stream that it launches on.
//
// A decoded token's call is 2 us of GPU time.  Marshalled in Python with ctypes
// (as the attention's own calls are) it took 13 us of host time, most of it in
// allocating tensors and reading their properties one by one; here it takes 4.
//
// The library itself stays free of PyTorch: its entry points are looked up in
// whichever build use() was given.
#include <Python.h>
#include <dlfcn.h>

#include <string>
#include <vector>

#include <ATen/ATen.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include "../../include/la.h"

namespace {

struct Error {   // becomes a Python exception
    PyObject *type;
    std::string what;
};
[[noreturn]] void bad_value(const std::string &what) { throw Error{PyExc_ValueError, what}; }
[[noreturn]] void bad_type(const std::string &what) { throw Error{PyExc_TypeError, what}; }

struct Calls {
    decltype(&la_recurrence_workspace_bytes) recurrence_workspace_bytes;
    decltype(&la_recurrence_forward) recurrence_forward;
    decltype(&la_recurrence_step) recurrence_step;
    decltype(&la_recurrence_backward) recurrence_backward;
    decltype(&la_layernorm_forward) layernorm_forward;
    decltype(&la_layernorm_workspace_bytes) layernorm_workspace_bytes;
    decltype(&la_layernorm_backward) layernorm_backward;
    decltype(&la_grad_workspace_bytes) grad_workspace_bytes;
    decltype(&la_grad_norm) grad_norm;
    decltype(&la_grad_clip) grad_clip;
    decltype(&la_decay_workspace_bytes) decay_workspace_bytes;
    decltype(&la_decay_forward) decay_forward;
    decltype(&la_decay_step) decay_step;
    decltype(&la_decay_backward) decay_backward;
    decltype(&la_qk_rotate_forward) qk_rotate_forward;
    decltype(&la_qk_rotate_workspace_bytes) qk_rotate_workspace_bytes;
    decltype(&la_qk_rotate_backward) qk_rotate_backward;
} calls;

std::string shape_text(at::IntArrayRef s) {
    std::string t = "(";
    for (size_t i = 0; i < s.size(); i++) t += (i ? ", " : "") + std::to_string(s[i]);
    return t + (s.size() == 1 ? ",)" : ")");
}
const char *type_text(at::ScalarType t) {
    return t == at::kFloat ? "torch.float32" : t == at::kBFloat16 ? "torch.bfloat16" : "torch.int32";
}

// The tensor, or an undefined one for None.
const at::Tensor &tensor(const char *name, PyObject *o) {
    static const at::Tensor none;
    if (o == Py_None) return none;
    if (!THPVariable_Check(o)) bad_type(std::string(name) + " must be a tensor");
    return THPVariable_Unpack(o);
}
const at::Tensor &required(const char *name, PyObject *o) {
    const at::Tensor &t = tensor(name, o);
    if (!t.defined()) bad_value(std::string(name) + " is required");
    return t;
}

la_dtype dtype_of(const at::Tensor &t) {
    if (t.scalar_type() == at::kFloat) return LA_DTYPE_F32;
    if (t.scalar_type() == at::kBFloat16) return LA_DTYPE_BF16;
    bad_type(std::string("unsupported dtype ") + c10::toString(t.scalar_type()) + " (float32 or bfloat16)");
}

// t (or undefined) has this shape, type and device.
void like(const char *name, const at::Tensor &t, at::IntArrayRef shape, at::ScalarType type, at::Device device) {
    if (!t.defined()) return;
    if (t.sizes() != shape) bad_value(std::string(name) + " must have shape " + shape_text(shape));
    if (t.scalar_type() != type) bad_type(std::string(name) + " must be " + type_text(type));
    if (t.device() != device) bad_value(std::string(name) + " must be on the same device as the rest");
}
// ... and is taken as a plain fp32 (or int32) array.
void array(const char *name, const at::Tensor &t, at::IntArrayRef shape, at::Device device,
           at::ScalarType type = at::kFloat) {
    like(name, t, shape, type, device);
    if (t.defined() && !t.is_contiguous()) bad_value(std::string(name) + " must be contiguous");
}
template <typename T = float> T *data(const at::Tensor &t) {
    return t.defined() ? static_cast<T *>(t.data_ptr()) : nullptr;
}

// The stream of a call (None: the current one, else its handle), and the place
// where the call allocates.  The caller's tensors may be memory of another stream:
// on a stream that was given, the allocator is told that they are in use there, so
// that one freed right after the call is not handed out again too early.
class Place {
  public:
    Place(PyObject *stream, at::Device device, std::initializer_list<const at::Tensor *> used) {
        if (!device.is_cuda()) bad_value("tensors must be on a CUDA device");
        if (device.index() != c10::cuda::current_device()) bad_value("tensors must be on the current CUDA device");
        if (stream == Py_None) {
            stream_ = c10::cuda::getCurrentCUDAStream(device.index()).stream();
        } else {
            stream_ = reinterpret_cast<cudaStream_t>(PyLong_AsVoidPtr(stream));
            if (PyErr_Occurred()) throw Error{nullptr, ""};
            const auto given = c10::cuda::getStreamFromExternal(stream_, device.index());
            for (const at::Tensor *t : used)
                if (t->defined()) t->record_stream(given);
            guard_.reset_stream(given);
        }
    }
    la_stream_t stream() const { return reinterpret_cast<la_stream_t>(stream_); }
    void use(const at::Tensor &t) const { t.record_stream(*guard_.current_stream()); }

  private:
    cudaStream_t stream_;
    c10::cuda::OptionalCUDAStreamGuard guard_;
};

at::Tensor out_like(const at::Tensor &given, const at::Tensor &ref) {
    return given.defined() ? given : at::empty(ref.sizes(), ref.options());
}
at::Tensor out_float(const at::Tensor &given, const at::Tensor &ref, at::IntArrayRef shape) {
    return given.defined() ? given : at::empty(shape, ref.options().dtype(at::kFloat));
}
at::Tensor workspace(const at::Tensor &ref, size_t bytes) {
    return bytes ? at::empty({(int64_t)bytes}, ref.options().dtype(at::kByte)) : at::Tensor();
}

// Rows of [B,N,D] or [B,H,N,D] ([B,D] or [B,H,D] for a step).
la_view view_of(const char *name, const at::Tensor &t, bool step) {
    if (!t.defined()) return {nullptr, 0, 0, 0};
    const auto st = t.strides();
    const size_t n = st.size();
    if (st[n - 1] != 1 && t.size(n - 1) > 1) bad_value(std::string(name) + ": the channels must be contiguous");
    if (step) return {t.data_ptr(), st[0], n == 3 ? st[1] : 0, 0};
    return {t.data_ptr(), st[0], n == 4 ? st[1] : 0, st[n - 2]};
}

int small(int64_t n) {
    if (n > 0x7fffffff) bad_value("a dimension is larger than 2^31 - 1");
    return (int)n;
}

la_shape rec_shape(const at::Tensor &x, bool step) {
    const auto sh = x.sizes();
    const int lead = (int)sh.size() - (step ? 1 : 2);
    if (lead != 1 && lead != 2)
        bad_value(step ? "x must be [B,D] or [B,H,D]" : "x must be [B,N,D] or [B,H,N,D]");
    if (sh.back() < 1) bad_value("x must have a channel");
    return {small(sh[0]), lead == 2 ? small(sh[1]) : 1, step ? 1 : small(sh[sh.size() - 2]), small(sh.back()), 0,
            dtype_of(x)};
}
c10::SmallVector<int64_t, 3> state_shape(const at::Tensor &x) {
    const auto sh = x.sizes();
    c10::SmallVector<int64_t, 3> s(sh.begin(), sh.end() - 2);
    s.push_back(sh.back());
    return s;
}

// All rows (last dimension) of t as one strided list.
la_rows rows_of(const char *name, const at::Tensor &t) {
    if (!t.defined()) return {nullptr, 0};
    const auto st = t.strides(), sh = t.sizes();
    const int64_t C = sh.back();
    if (t.is_contiguous()) return {t.data_ptr(), C};
    if (st.back() != 1 && C > 1) bad_value(std::string(name) + ": the last dimension must be contiguous");
    int64_t stride = -1, extent = 0;
    for (int64_t d = (int64_t)sh.size() - 2; d >= 0; d--) {
        if (sh[d] == 1) continue;
        if (stride < 0) stride = st[d];
        else if (st[d] != extent) bad_value(std::string(name) + ": the rows must share one stride");
        extent = st[d] * sh[d];
    }
    return {t.data_ptr(), stride < 0 ? C : stride};
}

PyObject *wrap(const at::Tensor &t) { return THPVariable_Wrap(t); }
PyObject *result(la_status st, std::initializer_list<at::Tensor> outs) {   // (status, tensors...)
    PyObject *r = PyTuple_New(1 + (Py_ssize_t)outs.size());
    if (!r) throw Error{nullptr, ""};
    PyTuple_SET_ITEM(r, 0, PyLong_FromLong(st));
    Py_ssize_t i = 1;
    for (const at::Tensor &t : outs) {
        if (t.defined()) {
            PyTuple_SET_ITEM(r, i++, wrap(t));
        } else {
            Py_INCREF(Py_None);
            PyTuple_SET_ITEM(r, i++, Py_None);
        }
    }
    return r;
}

constexpr size_t kInvalid = (size_t)-1;

// (x, g, gate, out, h0, hN, lens, stream) -> (status, out)
PyObject *recurrence_forward(PyObject *const *a) {
    const at::Tensor &x = required("x", a[0]), &g = required("g", a[1]), &given = tensor("out", a[3]);
    const at::Tensor &h0 = tensor("h0", a[4]), &hN = tensor("hN", a[5]), &lens = tensor("lens", a[6]);
    const la_shape s = rec_shape(x, false);
    const auto device = x.device();
    like("g", g, x.sizes(), x.scalar_type(), device);
    like("out", given, x.sizes(), x.scalar_type(), device);
    const auto state = state_shape(x);
    array("h0", h0, state, device);
    array("hN", hN, state, device);
    array("lens", lens, {s.B}, device, at::kInt);
    const Place place(a[7], device, {&x, &g, &given, &h0, &hN, &lens});
    const at::Tensor out = out_like(given, x);
    const size_t need = calls.recurrence_workspace_bytes(s);
    const at::Tensor ws = workspace(x, need == kInvalid ? 0 : need);   // the call itself says what is wrong
    return result(calls.recurrence_forward(view_of("x", x, false), view_of("g", g, false), view_of("out", out, false),
                                           data<int>(lens), s, (la_gate)PyLong_AsLong(a[2]), data(h0), data(hN),
                                           data<void>(ws), need, place.stream()),
                  {out});
}

// (x, g, h, gate, y, stream) -> (status, y)
PyObject *recurrence_step(PyObject *const *a) {
    const at::Tensor &x = required("x", a[0]), &g = required("g", a[1]), &h = required("h", a[2]);
    const at::Tensor &given = tensor("y", a[4]);
    const la_shape s = rec_shape(x, true);
    const auto device = x.device();
    like("g", g, x.sizes(), x.scalar_type(), device);
    like("y", given, x.sizes(), x.scalar_type(), device);
    array("h", h, x.sizes(), device);
    const Place place(a[5], device, {&x, &g, &h, &given});
    const at::Tensor y = out_like(given, x);
    return result(calls.recurrence_step(view_of("x", x, true), view_of("g", g, true), view_of("y", y, true), s,
                                        (la_gate)PyLong_AsLong(a[3]), data(h), place.stream()),
                  {y});
}

// (x, g, out, dout, gate, h0, dhN, dh0, lens, dx, dg, stream) -> (status, dx, dg)
PyObject *recurrence_backward(PyObject *const *a) {
    const at::Tensor &x = tensor("x", a[0]), &g = required("g", a[1]), &out = required("out", a[2]);
    const at::Tensor &dout = required("dout", a[3]), &h0 = tensor("h0", a[5]), &dhN = tensor("dhN", a[6]);
    const at::Tensor &dh0 = tensor("dh0", a[7]), &lens = tensor("lens", a[8]);
    const at::Tensor &given_x = tensor("dx", a[9]), &given_g = tensor("dg", a[10]);
    const la_gate gate = (la_gate)PyLong_AsLong(a[4]);
    const la_shape s = rec_shape(g, false);
    if (gate == LA_GATE_SIGMOID && !x.defined()) bad_value("the sigmoid gate needs x");
    const auto device = g.device();
    like("x", x, g.sizes(), g.scalar_type(), device);
    like("out", out, g.sizes(), g.scalar_type(), device);
    like("dout", dout, g.sizes(), g.scalar_type(), device);
    like("dx", given_x, g.sizes(), g.scalar_type(), device);
    like("dg", given_g, g.sizes(), g.scalar_type(), device);
    const auto state = state_shape(g);
    array("h0", h0, state, device);
    array("dhN", dhN, state, device);
    array("dh0", dh0, state, device);
    array("lens", lens, {s.B}, device, at::kInt);
    const Place place(a[11], device, {&x, &g, &out, &dout, &h0, &dhN, &dh0, &lens, &given_x, &given_g});
    const at::Tensor dx = out_like(given_x, g), dg = out_like(given_g, g);
    const size_t need = calls.recurrence_workspace_bytes(s);
    const at::Tensor ws = workspace(g, need == kInvalid ? 0 : need);
    return result(calls.recurrence_backward(view_of("x", x, false), view_of("g", g, false), view_of("out", out, false),
                                            view_of("dout", dout, false), view_of("dx", dx, false),
                                            view_of("dg", dg, false), data<int>(lens), s, gate, data(h0), data(dhN),
                                            data(dh0), data<void>(ws), need, place.stream()),
                  {dx, dg});
}

// (x, w, b, eps, res, y, sum, mean, rstd, stats, stream) -> (status, y, sum, mean, rstd)
PyObject *layernorm_forward(PyObject *const *a) {
    const at::Tensor &x = required("x", a[0]), &w = tensor("w", a[1]), &b = tensor("b", a[2]);
    const at::Tensor &res = tensor("res", a[4]), &given_y = tensor("y", a[5]), &given_sum = tensor("sum", a[6]);
    const at::Tensor &given_mean = tensor("mean", a[7]), &given_rstd = tensor("rstd", a[8]);
    const bool stats = PyObject_IsTrue(a[9]);
    if (x.dim() < 1 || x.sizes().back() < 1) bad_value("x must have rows of at least one value");
    const la_dtype dtype = dtype_of(x);
    const auto sh = x.sizes(), lead = sh.slice(0, sh.size() - 1);
    const int64_t C = sh.back();
    const auto device = x.device();
    if (given_sum.defined() && !res.defined()) bad_value("sum needs res");
    if (!stats && (given_mean.defined() || given_rstd.defined())) bad_value("mean and rstd need stats");
    like("res", res, sh, x.scalar_type(), device);
    like("sum", given_sum, sh, x.scalar_type(), device);
    like("y", given_y, sh, x.scalar_type(), device);
    array("w", w, {C}, device);
    array("b", b, {C}, device);
    array("mean", given_mean, lead, device);
    array("rstd", given_rstd, lead, device);
    const double eps = PyFloat_AsDouble(a[3]);
    if (PyErr_Occurred()) throw Error{nullptr, ""};
    const Place place(a[10], device, {&x, &w, &b, &res, &given_y, &given_sum, &given_mean, &given_rstd});
    const at::Tensor y = out_like(given_y, x);
    at::Tensor sum, mean, rstd;
    if (res.defined()) sum = out_like(given_sum, x);
    if (stats) mean = out_float(given_mean, x, lead), rstd = out_float(given_rstd, x, lead);
    return result(calls.layernorm_forward(rows_of("x", x), rows_of("res", res), rows_of("sum", sum), rows_of("y", y),
                                          data(w), data(b), data(mean), data(rstd), x.numel() / C, small(C), dtype,
                                          (float)eps, place.stream()),
                  {y, res.defined() ? sum : x, mean, rstd});
}

// (dy, s, w, mean, rstd, dsum, ds, dw, db, stream) -> (status, ds, dw, db)
PyObject *layernorm_backward(PyObject *const *a) {
    const at::Tensor &dy = required("dy", a[0]), &s = required("s", a[1]), &w = tensor("w", a[2]);
    const at::Tensor &mean = required("mean", a[3]), &rstd = required("rstd", a[4]), &dsum = tensor("dsum", a[5]);
    const at::Tensor &given = tensor("ds", a[6]), &given_w = tensor("dw", a[7]), &given_b = tensor("db", a[8]);
    if (dy.dim() < 1 || dy.sizes().back() < 1) bad_value("dy must have rows of at least one value");
    const la_dtype dtype = dtype_of(dy);
    const auto sh = dy.sizes(), lead = sh.slice(0, sh.size() - 1);
    const int64_t C = sh.back(), rows = dy.numel() / C;
    const auto device = dy.device();
    like("s", s, sh, dy.scalar_type(), device);
    like("dsum", dsum, sh, dy.scalar_type(), device);
    like("ds", given, sh, dy.scalar_type(), device);
    array("w", w, {C}, device);
    array("mean", mean, lead, device);
    array("rstd", rstd, lead, device);
    array("dw", given_w, {C}, device);
    array("db", given_b, {C}, device);
    const Place place(a[9], device, {&dy, &s, &w, &mean, &rstd, &dsum, &given, &given_w, &given_b});
    const at::Tensor ds = out_like(given, dy), dw = out_float(given_w, dy, {C}), db = out_float(given_b, dy, {C});
    const size_t need = calls.layernorm_workspace_bytes(rows, small(C), dtype);
    const at::Tensor ws = workspace(dy, need == kInvalid ? 0 : need);
    return result(calls.layernorm_backward(rows_of("dy", dy), rows_of("s", s), rows_of("dsum", dsum),
                                           rows_of("ds", ds), data(w), data(mean), data(rstd), data(dw), data(db),
                                           rows, small(C), dtype, data<void>(ws), need, place.stream()),
                  {ds, dw, db});
}

// (grads, max_norm or None for the norm alone, out or None for in place, norm, stream) -> (status, norm)
PyObject *grad(PyObject *const *a) {
    struct List {   // a list or tuple, held while it is read
        PyObject *seq;
        explicit List(PyObject *o) : seq(PySequence_Fast(o, "a list of tensors is wanted")) {
            if (!seq) throw Error{nullptr, ""};
        }
        ~List() { Py_DECREF(seq); }
        Py_ssize_t size() const { return PySequence_Fast_GET_SIZE(seq); }
        PyObject *operator[](Py_ssize_t i) const { return PySequence_Fast_GET_ITEM(seq, i); }
    };
    const List grads(a[0]);
    const Py_ssize_t n = grads.size();
    if (n == 0) bad_value("no tensors");
    if (n > 0x7fffffff) bad_value("too many tensors");
    const bool clip = a[1] != Py_None;
    const at::Tensor first = required("grads", grads[0]);
    std::vector<la_tensor> table((size_t)n);
    for (Py_ssize_t i = 0; i < n; i++) {
        const at::Tensor &t = required("grads", grads[i]);
        if (!t.is_contiguous()) bad_value("tensors must be contiguous");
        table[i] = {t.data_ptr(), clip ? t.data_ptr() : nullptr, t.numel(), dtype_of(t)};
        if (t.device() != first.device()) bad_value("all tensors must be on one device");
    }
    if (clip && a[2] != Py_None) {
        const List out(a[2]);
        if (out.size() != n) bad_value("out must have one tensor per gradient");
        for (Py_ssize_t i = 0; i < n; i++) {
            const at::Tensor &t = required("out", out[i]);
            if (t.sizes() != required("grads", grads[i]).sizes() || dtype_of(t) != table[i].dtype)
                bad_value("out must have the gradients' shapes and types");
            if (!t.is_contiguous()) bad_value("out must be contiguous");
            if (t.device() != first.device()) bad_value("all tensors must be on one device");
            table[i].dst = t.data_ptr();
        }
    }
    const at::Tensor &given = tensor("norm", a[3]);
    array("norm", given, {}, first.device());
    const double max_norm = clip ? PyFloat_AsDouble(a[1]) : 0.0;
    if (PyErr_Occurred()) throw Error{nullptr, ""};
    const Place place(a[4], first.device(), {&given});
    if (a[4] != Py_None)
        for (Py_ssize_t i = 0; i < n; i++) place.use(required("grads", grads[i]));
    if (a[4] != Py_None && clip && a[2] != Py_None) {
        const List out(a[2]);
        for (Py_ssize_t i = 0; i < n; i++) place.use(required("out", out[i]));
    }
    const at::Tensor norm = out_float(given, first, {});
    const size_t need = calls.grad_workspace_bytes((int)n);
    const at::Tensor ws = workspace(first, need);
    return result(clip ? calls.grad_clip(table.data(), (int)n, (float)max_norm, data(norm), data<void>(ws), need,
                                         place.stream())
                       : calls.grad_norm(table.data(), (int)n, data(norm), data<void>(ws), need, place.stream()),
                  {norm});
}

float number(PyObject *o) {
    const double v = PyFloat_AsDouble(o);
    if (PyErr_Occurred()) throw Error{nullptr, ""};
    return (float)v;
}

// Shape of the attention with decays: k [B,H,N,D] and v [B,H,N,M] (no N for a step).
la_shape decay_shape(const at::Tensor &k, const at::Tensor &v, bool step) {
    const auto a = k.sizes(), b = v.sizes();
    const size_t dims = step ? 3 : 4;
    if (a.size() != dims || b.size() != dims)
        bad_value(step ? "k must be [B,H,D] and v [B,H,M]" : "k must be [B,H,N,D] and v [B,H,N,M]");
    if (a.slice(0, dims - 1) != b.slice(0, dims - 1)) bad_value("k and v must agree in all but the last dimension");
    if (a.back() < 1 || b.back() < 1) bad_value("k and v must have a channel");
    return {small(a[0]), small(a[1]), step ? 1 : small(a[2]), small(a.back()), small(b.back()), dtype_of(k)};
}
c10::SmallVector<int64_t, 4> with_last(const at::Tensor &x, int64_t n) {
    c10::SmallVector<int64_t, 4> s(x.sizes().begin(), x.sizes().end());
    s.back() = n;
    return s;
}

// (q, k, v, log_decay, scale, S0, SN, lens, out, want_out, stream) -> (status, out)
PyObject *decay_forward(PyObject *const *a) {
    const at::Tensor &q = tensor("q", a[0]), &k = required("k", a[1]), &v = required("v", a[2]);
    const at::Tensor &g = required("log_decay", a[3]), &S0 = tensor("S0", a[5]), &SN = tensor("SN", a[6]);
    const at::Tensor &lens = tensor("lens", a[7]), &given = tensor("out", a[8]);
    const bool want = PyObject_IsTrue(a[9]);
    const la_shape s = decay_shape(k, v, false);
    const auto device = k.device();
    if (want && !q.defined()) bad_value("q is required");
    if (!want && given.defined()) bad_value("out needs want_out");
    if (!want && !SN.defined()) bad_value("nothing is wanted: want_out or SN");
    like("q", q, k.sizes(), k.scalar_type(), device);
    like("v", v, v.sizes(), k.scalar_type(), device);
    like("out", given, v.sizes(), k.scalar_type(), device);
    array("log_decay", g, {s.H}, device);
    array("S0", S0, {s.B, s.H, s.D, s.M}, device);
    array("SN", SN, {s.B, s.H, s.D, s.M}, device);
    array("lens", lens, {s.B}, device, at::kInt);
    const float scale = number(a[4]);
    const Place place(a[10], device, {&q, &k, &v, &g, &S0, &SN, &lens, &given});
    at::Tensor out;
    if (want) out = out_like(given, v);
    const size_t need = calls.decay_workspace_bytes(s, 0);
    const at::Tensor ws = workspace(k, need == kInvalid ? 0 : need);
    return result(calls.decay_forward(view_of("q", q, false), view_of("k", k, false), view_of("v", v, false),
                                      view_of("out", out, false), data(g), data<int>(lens), s, scale, data(S0), data(SN),
                                      data<void>(ws), need, place.stream()),
                  {out});
}

// (q, k, v, S, log_decay, scale, y, stream) -> (status, y)
PyObject *decay_step(PyObject *const *a) {
    const at::Tensor &q = required("q", a[0]), &k = required("k", a[1]), &v = required("v", a[2]);
    const at::Tensor &S = required("S", a[3]), &g = required("log_decay", a[4]), &given = tensor("y", a[6]);
    const la_shape s = decay_shape(k, v, true);
    const auto device = k.device();
    like("q", q, k.sizes(), k.scalar_type(), device);
    like("v", v, v.sizes(), k.scalar_type(), device);
    like("y", given, v.sizes(), k.scalar_type(), device);
    array("log_decay", g, {s.H}, device);
    array("S", S, {s.B, s.H, s.D, s.M}, device);
    const float scale = number(a[5]);
    const Place place(a[7], device, {&q, &k, &v, &S, &g, &given});
    const at::Tensor y = out_like(given, v);
    return result(calls.decay_step(view_of("q", q, true), view_of("k", k, true), view_of("v", v, true),
                                   view_of("y", y, true), data(g), s, scale, data(S), place.stream()),
                  {y});
}

// (q, k, v, dout, log_decay, scale, S0, dSN, dS0, lens, dq, dk, dv, stream) -> (status, dq, dk, dv)
PyObject *decay_backward(PyObject *const *a) {
    const at::Tensor &q = required("q", a[0]), &k = required("k", a[1]), &v = required("v", a[2]);
    const at::Tensor &dout = required("dout", a[3]), &g = required("log_decay", a[4]), &S0 = tensor("S0", a[6]);
    const at::Tensor &dSN = tensor("dSN", a[7]), &dS0 = tensor("dS0", a[8]), &lens = tensor("lens", a[9]);
    const at::Tensor &gq = tensor("dq", a[10]), &gk = tensor("dk", a[11]), &gv = tensor("dv", a[12]);
    const la_shape s = decay_shape(k, v, false);
    const auto device = k.device();
    like("q", q, k.sizes(), k.scalar_type(), device);
    like("v", v, v.sizes(), k.scalar_type(), device);
    like("dout", dout, v.sizes(), k.scalar_type(), device);
    like("dq", gq, k.sizes(), k.scalar_type(), device);
    like("dk", gk, k.sizes(), k.scalar_type(), device);
    like("dv", gv, v.sizes(), k.scalar_type(), device);
    array("log_decay", g, {s.H}, device);
    for (const auto &st : {std::make_pair("S0", &S0), std::make_pair("dSN", &dSN), std::make_pair("dS0", &dS0)})
        array(st.first, *st.second, {s.B, s.H, s.D, s.M}, device);
    array("lens", lens, {s.B}, device, at::kInt);
    const float scale = number(a[5]);
    const Place place(a[13], device, {&q, &k, &v, &dout, &g, &S0, &dSN, &dS0, &lens, &gq, &gk, &gv});
    const at::Tensor dq = out_like(gq, k), dk = out_like(gk, k), dv = out_like(gv, v);
    const size_t need = calls.decay_workspace_bytes(s, 1);
    const at::Tensor ws = workspace(k, need == kInvalid ? 0 : need);
    return result(calls.decay_backward(view_of("q", q, false), view_of("k", k, false), view_of("v", v, false),
                                       view_of("dout", dout, false), view_of("dq", dq, false), view_of("dk", dk, false),
                                       view_of("dv", dv, false), data(g), data<int>(lens), s, scale, data(S0), data(dSN),
                                       data(dS0), data<void>(ws), need, place.stream()),
                  {dq, dk, dv});
}

// What the rotation's two calls take alike: q [B,Hq,N,D], k [B,Hk,N,D] or none, positions, frequencies, axes.
struct Rotation {
    la_qk_shape s;
    la_rotation r;
    Rotation(const at::Tensor &q, const at::Tensor &k, const at::Tensor &pos, const at::Tensor &freq, PyObject *pairs,
             PyObject *axes) {
        const auto sh = q.sizes();
        if (sh.size() != 4 || sh[3] < 1) bad_value("q must be [B,Hq,N,D]");
        if (k.defined() && (k.dim() != 4 || k.size(0) != sh[0] || k.size(2) != sh[2] || k.size(3) != sh[3]))
            bad_value("k must be [B,Hk,N,D] with q's B, N and D");
        const auto device = q.device();
        like("k", k, k.sizes(), q.scalar_type(), device);
        s = {small(sh[0]), small(sh[2]), small(sh[1]), k.defined() ? small(k.size(1)) : 0, small(sh[3]), dtype_of(q)};
        if (freq.dim() != 1) bad_value("freq must be [P]");
        array("freq", freq, freq.sizes(), device);
        const int64_t d = pos.dim();
        if (d < 1 || d > 3 || pos.size(d - 1) != sh[2] || (d > 1 && pos.size(d - 2) != sh[0]))
            bad_value("pos must be [N], [B,N] or [A,B,N]");
        like("pos", pos, pos.sizes(), at::kInt, device);
        const auto st = pos.strides();
        r.pos = data<int>(pos), r.freq = data(freq);
        r.sn = st[d - 1], r.sb = d > 1 ? st[d - 2] : 0, r.sa = d > 2 ? st[0] : 0;
        r.A = d > 2 ? small(pos.size(0)) : 1, r.P = small(freq.numel());
        if (2 * (int64_t)r.P > sh[3]) bad_value("freq has more pairs than a head has");
        r.pairs = (la_pairs)PyLong_AsLong(pairs), r.axes = nullptr;
        if (axes != Py_None) {
            char *bytes;
            Py_ssize_t n;
            if (PyBytes_AsStringAndSize(axes, &bytes, &n) < 0) throw Error{nullptr, ""};
            if (n != r.P) bad_value("axes must have one entry per pair");
            r.axes = reinterpret_cast<const unsigned char *>(bytes);
        }
    }
};

// (q, k, pos, freq, wq, wk, eps, norm, pairs, axes, qo, ko, stream) -> (status, qo, ko)
PyObject *qk_rotate_forward(PyObject *const *a) {
    const at::Tensor &q = required("q", a[0]), &k = tensor("k", a[1]), &pos = required("pos", a[2]);
    const at::Tensor &freq = required("freq", a[3]), &wq = tensor("wq", a[4]), &wk = tensor("wk", a[5]);
    const at::Tensor &gq = tensor("qo", a[10]), &gk = tensor("ko", a[11]);
    const Rotation rot(q, k, pos, freq, a[8], a[9]);
    const auto device = q.device();
    const bool norm = PyObject_IsTrue(a[7]);
    if (!norm && (wq.defined() || wk.defined())) bad_value("wq and wk need the norm");
    if (!k.defined() && (wk.defined() || gk.defined())) bad_value("wk and ko need k");
    array("wq", wq, {rot.s.D}, device);
    array("wk", wk, {rot.s.D}, device);
    like("qo", gq, q.sizes(), q.scalar_type(), device);
    if (k.defined()) like("ko", gk, k.sizes(), k.scalar_type(), device);
    const float eps = number(a[6]);
    const Place place(a[12], device, {&q, &k, &pos, &freq, &wq, &wk, &gq, &gk});
    const at::Tensor qo = out_like(gq, q);
    at::Tensor ko;
    if (k.defined()) ko = out_like(gk, k);
    return result(calls.qk_rotate_forward(view_of("q", q, false), view_of("k", k, false), view_of("qo", qo, false),
                                          view_of("ko", ko, false), data(wq), data(wk), rot.r, rot.s, norm, eps,
                                          place.stream()),
                  {qo, ko});
}

// (dqo, dko, q, k, pos, freq, wq, wk, eps, norm, pairs, axes, dq, dk, dwq, dwk, stream) -> (status, dq, dk, dwq, dwk)
PyObject *qk_rotate_backward(PyObject *const *a) {
    const at::Tensor &dqo = required("dqo", a[0]), &dko = tensor("dko", a[1]), &q = required("q", a[2]);
    const at::Tensor &k = tensor("k", a[3]), &pos = required("pos", a[4]), &freq = required("freq", a[5]);
    const at::Tensor &wq = tensor("wq", a[6]), &wk = tensor("wk", a[7]), &gq = tensor("dq", a[12]);
    const at::Tensor &gk = tensor("dk", a[13]), &gwq = tensor("dwq", a[14]), &gwk = tensor("dwk", a[15]);
    const Rotation rot(q, k, pos, freq, a[10], a[11]);
    const auto device = q.device();
    const bool norm = PyObject_IsTrue(a[9]);
    if (!norm && (wq.defined() || wk.defined() || gwq.defined() || gwk.defined()))
        bad_value("weights and their gradients need the norm");
    if (k.defined() != dko.defined()) bad_value("dko and k go together");
    if (!k.defined() && (wk.defined() || gk.defined() || gwk.defined())) bad_value("wk, dk and dwk need k");
    like("dqo", dqo, q.sizes(), q.scalar_type(), device);
    like("dq", gq, q.sizes(), q.scalar_type(), device);
    if (k.defined()) {
        like("dko", dko, k.sizes(), k.scalar_type(), device);
        like("dk", gk, k.sizes(), k.scalar_type(), device);
    }
    array("wq", wq, {rot.s.D}, device);
    array("wk", wk, {rot.s.D}, device);
    array("dwq", gwq, {rot.s.D}, device);
    array("dwk", gwk, {rot.s.D}, device);
    const float eps = number(a[8]);
    const Place place(a[16], device, {&dqo, &dko, &q, &k, &pos, &freq, &wq, &wk, &gq, &gk, &gwq, &gwk});
    const at::Tensor dq = out_like(gq, q);
    at::Tensor dk, dwq, dwk;
    if (k.defined()) dk = out_like(gk, k);
    if (norm) dwq = out_float(gwq, q, {rot.s.D});
    if (norm && k.defined()) dwk = out_float(gwk, q, {rot.s.D});
    const size_t need = calls.qk_rotate_workspace_bytes(rot.s);
    const at::Tensor ws = workspace(q, norm && need != kInvalid ? need : 0);
    return result(calls.qk_rotate_backward(view_of("dqo", dqo, false), view_of("dko", dko, false), view_of("q", q, false),
                                           view_of("k", k, false), view_of("dq", dq, false), view_of("dk", dk, false),
                                           data(wq), data(wk), rot.r, rot.s, norm, eps, data(dwq), data(dwk),
                                           data<void>(ws), need, place.stream()),
                  {dq, dk, dwq, dwk});
}

// (tensor, step) -> (address, sb, sh, sn) and (tensor) -> (address, stride): what a call hands to the library.
PyObject *view(PyObject *const *a) {
    const la_view v = view_of("x", required("x", a[0]), PyObject_IsTrue(a[1]));
    return Py_BuildValue("NLLL", PyLong_FromVoidPtr(v.data), v.sb, v.sh, v.sn);
}
PyObject *rows(PyObject *const *a) {
    const la_rows r = rows_of("x", required("x", a[0]));
    return Py_BuildValue("NL", PyLong_FromVoidPtr(r.data), r.stride);
}

// (path of a build of the library)
PyObject *use(PyObject *const *a) {
    const char *path = PyUnicode_AsUTF8(a[0]);
    if (!path) throw Error{nullptr, ""};
    void *h = dlopen(path, RTLD_NOW | RTLD_LOCAL);
    if (!h) throw Error{PyExc_RuntimeError, dlerror()};
    Calls c;
    auto get = [&](auto &f, const char *name) {
        f = reinterpret_cast<std::decay_t<decltype(f)>>(dlsym(h, name));
        if (!f) throw Error{PyExc_RuntimeError, std::string(path) + " has no " + name};
    };
    get(c.recurrence_workspace_bytes, "la_recurrence_workspace_bytes");
    get(c.recurrence_forward, "la_recurrence_forward");
    get(c.recurrence_step, "la_recurrence_step");
    get(c.recurrence_backward, "la_recurrence_backward");
    get(c.layernorm_forward, "la_layernorm_forward");
    get(c.layernorm_workspace_bytes, "la_layernorm_workspace_bytes");
    get(c.layernorm_backward, "la_layernorm_backward");
    get(c.grad_workspace_bytes, "la_grad_workspace_bytes");
    get(c.grad_norm, "la_grad_norm");
    get(c.grad_clip, "la_grad_clip");
    get(c.decay_workspace_bytes, "la_decay_workspace_bytes");
    get(c.decay_forward, "la_decay_forward");
    get(c.decay_step, "la_decay_step");
    get(c.decay_backward, "la_decay_backward");
    get(c.qk_rotate_forward, "la_qk_rotate_forward");
    get(c.qk_rotate_workspace_bytes, "la_qk_rotate_workspace_bytes");
    get(c.qk_rotate_backward, "la_qk_rotate_backward");
    calls = c;
    Py_RETURN_NONE;
}

// Runs a function that takes exactly N arguments; no C++ exception leaves it.
template <PyObject *(*F)(PyObject *const *), int N>
PyObject *entry(PyObject *, PyObject *const *args, Py_ssize_t n) {
    if (n != N) return PyErr_Format(PyExc_TypeError, "%d arguments are wanted, not %zd", N, n);
    HANDLE_TH_ERRORS   // PyTorch's own exceptions become the Python ones they are elsewhere
    try {
        return F(args);
    } catch (const Error &e) {
        if (e.type) PyErr_SetString(e.type, e.what.c_str());
        return nullptr;
    }
    END_HANDLE_TH_ERRORS
}
#define ENTRY(f, n) {#f, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(&entry<f, n>)), METH_FASTCALL, nullptr}

PyMethodDef methods[] = {ENTRY(use, 1),
                         ENTRY(view, 2),
                         ENTRY(rows, 1),
                         ENTRY(recurrence_forward, 8),
                         ENTRY(recurrence_step, 6),
                         ENTRY(recurrence_backward, 12),
                         ENTRY(layernorm_forward, 11),
                         ENTRY(layernorm_backward, 10),
                         ENTRY(grad, 5),
                         ENTRY(decay_forward, 11),
                         ENTRY(decay_step, 8),
                         ENTRY(decay_backward, 14),
                         ENTRY(qk_rotate_forward, 13),
                         ENTRY(qk_rotate_backward, 17),
                         {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_la_torch", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__la_torch(void) { return PyModule_Create(&module); }
