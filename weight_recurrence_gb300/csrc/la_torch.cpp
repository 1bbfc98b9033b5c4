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
                         {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_la_torch", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__la_torch(void) { return PyModule_Create(&module); }
