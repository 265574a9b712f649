// The torch front ends of the slot and convolution operators: checks of their tensors, the current
// stream, allocation of what the caller does not give, and the call of the C entry point
// (include/ssm_scan.h).  They run once per layer and step, so they are compiled: checked and passed
// from Python, the dozen tensors of a decode step cost three times what its kernel does (13.0 us a
// call against 3.4 us of kernel).
//
// The entry points are bound by address (bind), so that they are those of the library that the
// package has loaded, whichever build that is.
#define PY_SSIZE_T_CLEAN
#include <Python.h>

#include <ATen/ATen.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include <algorithm>
#include <cstring>
#include <initializer_list>
#include <string>

#include "ssm_scan.h"

namespace {

using at::Tensor;

struct Entries {
    decltype(&ssm_causal_conv1d_fwd) conv_fwd;
    decltype(&ssm_causal_conv1d_bwd_workspace_size) conv_bwd_size;
    decltype(&ssm_causal_conv1d_bwd) conv_bwd;
    decltype(&ssm_causal_conv1d_packed_fwd) conv_packed;
    decltype(&ssm_causal_conv1d_update) conv_update;
    decltype(&ssm_selective_scan_packed_workspace_size) scan_packed_size;
    decltype(&ssm_selective_scan_packed_fwd) scan_packed;
    decltype(&ssm_selective_state_update_slots) state_update;
    decltype(&ssm_state_slots_copy) slots_copy;
} entry;
PyObject* error_class = nullptr;      // called with (status, where), gives the exception to raise

// A refusal: the Python error is set.
struct Refused {};
[[noreturn]] void refuse(const char* format, const char* name, const char* what = "") {
    PyErr_Format(PyExc_ValueError, format, name, what);
    throw Refused();
}

// A tensor argument, or nothing for None.
struct Arg {
    const char* name;
    const Tensor* t = nullptr;
    Arg(const char* n, PyObject* o) : name(n) {
        if (o == Py_None) return;
        if (!THPVariable_Check(o)) {
            PyErr_Format(PyExc_TypeError, "%s must be a tensor", n);
            throw Refused();
        }
        t = &THPVariable_Unpack(o);
    }
    explicit operator bool() const { return t != nullptr; }
    const Tensor& operator*() const { return *t; }
    const Tensor* operator->() const { return t; }
    void* ptr() const { return t ? t->data_ptr() : nullptr; }
};

// An argument that cannot be None and whose rank says the other shapes.
void need_rank(const Arg& a, int64_t dims) {
    if (!a) refuse("%s must be a tensor%s", a.name);
    if (a->dim() != dims) {
        PyErr_Format(PyExc_ValueError, "%s must have %lld dimensions", a.name, (long long)dims);
        throw Refused();
    }
}
int need_cuda(const Arg& a, int64_t dims) {
    need_rank(a, dims);
    if (!a->is_cuda()) refuse("%s must be a CUDA tensor%s", a.name);
    if (!a->is_contiguous()) refuse("%s must be contiguous%s", a.name);
    return a->get_device();
}
int32_t io_code(const Arg& a) {
    if (a->scalar_type() == at::kBFloat16) return SSM_BF16;
    if (a->scalar_type() == at::kFloat) return SSM_F32;
    refuse("%s must be bfloat16 or float32%s", a.name);
}
// None, or a contiguous tensor of this type and shape on this device
void need(const Arg& a, at::ScalarType type, at::IntArrayRef shape, int device, bool may_be_none = true) {
    if (!a) {
        if (may_be_none) return;
        refuse("%s must be a tensor%s", a.name);
    }
    if (a->scalar_type() != type) refuse("%s must be %s", a.name, at::toString(type));
    if (a->sizes() != shape) {
        std::string want = "(", got = "(";
        for (auto v : shape) want += std::to_string(v) + ",";
        for (auto v : a->sizes()) got += std::to_string(v) + ",";
        PyErr_Format(PyExc_ValueError, "%s must have shape %s), not %s)", a.name, want.c_str(), got.c_str());
        throw Refused();
    }
    if (!a->is_cuda() || a->get_device() != device) refuse("%s must be on the device of the other tensors%s", a.name);
    if (!a->is_contiguous()) refuse("%s must be contiguous%s", a.name);
}

// Whether the dimensions from `first` on are laid out without gaps.
bool inner_contiguous(const Tensor& t, int64_t first) {
    int64_t want = 1;
    for (int64_t i = t.dim() - 1; i >= first; --i) {
        if (t.size(i) != 1 && t.stride(i) != want) return false;
        want *= t.size(i);
    }
    return true;
}
// A pool (n_slots, n, last) whose slots are contiguous and may lie apart; the elements from one to the next.
int64_t pool_stride(const Arg& a, at::ScalarType type, int64_t n, int64_t last, int device) {
    need_rank(a, 3);
    if (a->scalar_type() != type) refuse("%s must be %s", a.name, at::toString(type));
    if (a->size(1) != n || a->size(2) != last) {
        PyErr_Format(PyExc_ValueError, "%s must have shape (n_slots, %lld, %lld)", a.name, (long long)n, (long long)last);
        throw Refused();
    }
    if (!a->is_cuda() || a->get_device() != device) refuse("%s must be on the device of the other tensors%s", a.name);
    if (a->is_contiguous()) return n * last;
    if (!inner_contiguous(*a, 1)) refuse("every slot of %s must be contiguous%s", a.name);
    // a single slot's stride says nothing
    return a->size(0) > 1 ? a->stride(0) : n * last;
}
void need_indices(int64_t n, int device, const Arg& cu, const Arg& slots, const Arg& has) {
    need(cu, at::kInt, {n + 1}, device, false);
    need(slots, at::kInt, {n}, device);
    if (has) need(has, has->scalar_type() == at::kBool ? at::kBool : at::kByte, {n}, device);
}
int64_t n_seq(const Arg& cu) {
    need_rank(cu, 1);
    if (cu->size(0) < 1) refuse("%s must have n_seq + 1 entries%s", cu.name);
    return cu->size(0) - 1;
}
// the width of taps (dim, width)
int64_t need_taps(const Arg& w, const Arg& bias, int64_t dim, int device, bool check_width) {
    need_rank(w, 2);
    const int64_t width = w->size(1);
    if (check_width && (width < 1 || width > 4)) refuse("%s must have a width of 1 to 4%s", w.name);
    need(w, at::kFloat, {dim, width}, device);
    need(bias, at::kFloat, {dim}, device);
    return width;
}
void need_workspace(const Arg& ws, int device) {
    if (ws && (!ws->is_cuda() || ws->get_device() != device || !ws->is_contiguous()))
        refuse("%s must be contiguous and on the device of the other tensors%s", ws.name);
}
// The bytes from a tensor's first element to behind its last one, wherever its dimensions lie.
struct Span {
    const char *lo, *hi;
    explicit Span(const Tensor& t) : lo(static_cast<const char*>(t.data_ptr())), hi(lo) {
        if (t.numel() == 0) return;
        int64_t last = 0;
        for (int64_t i = 0; i < t.dim(); ++i) last += (t.size(i) - 1) * t.stride(i);
        hi = lo + (last + 1) * t.element_size();
    }
    bool meets(const Span& o) const { return lo < o.hi && o.lo < hi; }
};
// What is written must share no byte with what is read (`out` given: an output of the call's own never does).
// `in_place`: it may be that very tensor, where each thread reads its elements before it writes them.
void need_apart(const Arg& out, std::initializer_list<const Arg*> read, bool in_place = false) {
    if (!out) return;
    const Span o(*out);
    for (const Arg* in : read)
        if (*in && !(in_place && out.ptr() == in->ptr()) && o.meets(Span(**in)))
            refuse(in_place ? "%s must not overlap %s but for being the same tensor" : "%s must not overlap %s", out.name, in->name);
}
size_t bytes_of(const Tensor& t) { return (size_t)t.numel() * t.element_size(); }

// The device's current stream, with the device current for as long as this lives.
struct Launch {
    c10::cuda::CUDAGuard guard;
    ssm_stream_t stream;
    explicit Launch(int device)
        : guard((c10::DeviceIndex)device),
          stream(reinterpret_cast<ssm_stream_t>(c10::cuda::getCurrentCUDAStream((c10::DeviceIndex)device).stream())) {}
};
void check(int rc, const char* where) {
    if (rc == SSM_OK) return;
    PyObject* e = PyObject_CallFunction(error_class, "is", rc, where);
    if (e) {
        PyErr_SetObject((PyObject*)Py_TYPE(e), e);
        Py_DECREF(e);
    }
    throw Refused();
}
// `zeroed`: the call may leave some of it unwritten (padding, which only slots can name in a call of single tokens).
Tensor out_or(const Arg& out, const Tensor& like, bool zeroed) {
    return out ? *out : zeroed ? at::zeros_like(like) : at::empty_like(like);
}
bool truth(PyObject* o) {
    const int v = PyObject_IsTrue(o);
    if (v < 0) throw Refused();
    return v != 0;
}
int64_t whole(PyObject* o) {
    const long long v = PyLong_AsLongLong(o);
    if (v == -1 && PyErr_Occurred()) throw Refused();
    return v;
}
const float* f32(const Arg& a) { return static_cast<const float*>(a.ptr()); }
const int32_t* i32(const Arg& a) { return static_cast<const int32_t*>(a.ptr()); }
const uint8_t* u8(const Arg& a) { return static_cast<const uint8_t*>(a.ptr()); }

// (x, w, bias, silu, out)
PyObject* conv_fwd(PyObject* const* v) {
    const Arg x("x", v[0]), w("w", v[1]), bias("bias", v[2]), out("out", v[4]);
    const bool silu = truth(v[3]);
    const int dev = need_cuda(x, 3);
    const int64_t width = need_taps(w, bias, x->size(1), dev, false);
    const int32_t io = io_code(x);
    need(out, x->scalar_type(), x->sizes(), dev);
    need_apart(out, {&x, &w, &bias});
    const Launch on(dev);
    Tensor o = out_or(out, *x, false);
    check(entry.conv_fwd(x->size(0), x->size(1), x->size(2), (int32_t)width, io, x.ptr(), f32(w), f32(bias), silu,
                         o.data_ptr(), on.stream),
          "ssm_causal_conv1d_fwd");
    return THPVariable_Wrap(o);
}

// (x, w, dout, bias, silu, workspace) -> (dx, dw, dbias)
PyObject* conv_bwd(PyObject* const* v) {
    const Arg x("x", v[0]), w("w", v[1]), dout("dout", v[2]), bias("bias", v[3]), ws("workspace", v[5]);
    const bool silu = truth(v[4]);
    const int dev = need_cuda(x, 3);
    const int64_t b = x->size(0), d = x->size(1), l = x->size(2), width = need_taps(w, bias, d, dev, false);
    const int32_t io = io_code(x);
    need(dout, x->scalar_type(), x->sizes(), dev, false);
    need_workspace(ws, dev);
    const Launch on(dev);
    size_t bytes = 0;
    check(entry.conv_bwd_size(b, d, l, (int32_t)width, io, &bytes), "ssm_causal_conv1d_bwd_workspace_size");
    const Tensor work = ws ? *ws : at::empty({(int64_t)bytes}, x->options().dtype(at::kByte));
    Tensor dx = at::empty_like(*x), dw = at::empty_like(*w), db = at::empty({d}, w->options());
    check(entry.conv_bwd(b, d, l, (int32_t)width, io, x.ptr(), f32(w), f32(bias), silu, dout.ptr(), dx.data_ptr(),
                         dw.data_ptr<float>(), db.data_ptr<float>(), work.data_ptr(), bytes_of(work), on.stream),
          "ssm_causal_conv1d_bwd");
    return Py_BuildValue("(NNN)", THPVariable_Wrap(dx), THPVariable_Wrap(dw), THPVariable_Wrap(db));
}

// (x, w, cu_seqlens, conv_states, slots, has_state, bias, silu, out)
PyObject* conv_packed(PyObject* const* v) {
    const Arg x("x", v[0]), w("w", v[1]), cu("cu_seqlens", v[2]), states("conv_states", v[3]), slots("slots", v[4]),
        has("has_state", v[5]), bias("bias", v[6]), out("out", v[8]);
    const bool silu = truth(v[7]);
    const int dev = need_cuda(x, 2);
    const int64_t dim = x->size(0), total = x->size(1), n = n_seq(cu), width = need_taps(w, bias, dim, dev, true);
    const int32_t io = io_code(x);
    need(out, x->scalar_type(), x->sizes(), dev);
    const int64_t stride = pool_stride(states, x->scalar_type(), dim, width - 1, dev);
    need_indices(n, dev, cu, slots, has);
    need_apart(out, {&x, &w, &bias, &states, &cu, &slots, &has});
    const Launch on(dev);
    Tensor o = out_or(out, *x, true);
    check(entry.conv_packed(dim, total, n, (int32_t)width, io, x.ptr(), f32(w), f32(bias), silu, i32(cu), i32(slots), u8(has),
                            states.ptr(), states->size(0), stride, o.data_ptr(), on.stream),
          "ssm_causal_conv1d_packed_fwd");
    return THPVariable_Wrap(o);
}

// (x, w, conv_states, slots, bias, silu, out)
PyObject* conv_update(PyObject* const* v) {
    const Arg x("x", v[0]), w("w", v[1]), states("conv_states", v[2]), slots("slots", v[3]), bias("bias", v[4]), out("out", v[6]);
    const bool silu = truth(v[5]);
    const int dev = need_cuda(x, 2);
    const int64_t batch = x->size(0), dim = x->size(1), width = need_taps(w, bias, dim, dev, true);
    const int32_t io = io_code(x);
    need(out, x->scalar_type(), x->sizes(), dev);
    const int64_t stride = pool_stride(states, x->scalar_type(), dim, width - 1, dev);
    need(slots, at::kInt, {batch}, dev);
    need_apart(out, {&x}, true);
    need_apart(out, {&w, &bias, &states, &slots});
    const Launch on(dev);
    Tensor o = out_or(out, *x, (bool)slots);
    check(entry.conv_update(batch, dim, (int32_t)width, io, x.ptr(), f32(w), f32(bias), silu, i32(slots), states.ptr(),
                            states->size(0), stride, o.data_ptr(), on.stream),
          "ssm_causal_conv1d_update");
    return THPVariable_Wrap(o);
}

// (u, delta, A, B, C, cu_seqlens, states, slots, has_state, D, z, delta_bias, softplus, max_seqlen, out, workspace)
PyObject* scan_packed(PyObject* const* v) {
    const Arg u("u", v[0]), delta("delta", v[1]), A("A", v[2]), B("B", v[3]), C("C", v[4]), cu("cu_seqlens", v[5]),
        states("states", v[6]), slots("slots", v[7]), has("has_state", v[8]), D("D", v[9]), z("z", v[10]),
        bias("delta_bias", v[11]), out("out", v[14]), ws("workspace", v[15]);
    const bool softplus = truth(v[12]);
    const int64_t longest = v[13] == Py_None ? 0 : std::max<int64_t>(whole(v[13]), 0);
    const int dev = need_cuda(u, 2);
    need_rank(delta, 2);
    need_rank(B, 3);
    const int64_t dim = u->size(0), total = u->size(1), heads = delta->size(0), groups = B->size(0), N = B->size(1);
    const at::ScalarType type = u->scalar_type();
    const int32_t io = io_code(u);
    const int64_t n = n_seq(cu);
    need(delta, type, {heads, total}, dev);
    if (heads == dim) need(A, at::kFloat, {dim, N}, dev, false);
    else need(A, at::kFloat, {heads}, dev, false);
    need(B, type, {groups, N, total}, dev);
    need(C, type, {groups, N, total}, dev, false);
    need(D, at::kFloat, {dim}, dev);
    need(z, type, {dim, total}, dev);
    need(bias, at::kFloat, {heads}, dev);
    need(out, type, {dim, total}, dev);
    const int64_t stride = pool_stride(states, at::kFloat, dim, N, dev);
    need_indices(n, dev, cu, slots, has);
    need_workspace(ws, dev);
    need_apart(out, {&u, &delta, &B, &C, &z, &A, &D, &bias, &states, &cu, &slots, &has, &ws});
    const ssm_dims_t d = {n, dim, total, N, heads, groups, io, 0};
    const Launch on(dev);
    size_t bytes = 0;
    check(entry.scan_packed_size(&d, longest, &bytes), "ssm_selective_scan_packed_workspace_size");
    Tensor work;
    if (ws) work = *ws;
    else if (bytes) work = at::empty({(int64_t)bytes}, u->options().dtype(at::kByte));
    Tensor o = out_or(out, *u, true);
    check(entry.scan_packed(&d, u.ptr(), delta.ptr(), f32(A), B.ptr(), C.ptr(), f32(D), z.ptr(), f32(bias), softplus, i32(cu),
                            i32(slots), u8(has), static_cast<float*>(states.ptr()), states->size(0), stride, longest,
                            o.data_ptr(), work.defined() ? work.data_ptr() : nullptr, work.defined() ? bytes_of(work) : 0,
                            on.stream),
          "ssm_selective_scan_packed_fwd");
    return THPVariable_Wrap(o);
}

// (states, u, delta, A, B, C, slots, D, z, delta_bias, softplus, out)
PyObject* state_update(PyObject* const* v) {
    const Arg states("states", v[0]), u("u", v[1]), delta("delta", v[2]), A("A", v[3]), B("B", v[4]), C("C", v[5]),
        slots("slots", v[6]), D("D", v[7]), z("z", v[8]), bias("delta_bias", v[9]), out("out", v[11]);
    const bool softplus = truth(v[10]);
    const int dev = need_cuda(u, 2);
    need_rank(delta, 2);
    need_rank(B, 3);
    const int64_t batch = u->size(0), dim = u->size(1), heads = delta->size(1), groups = B->size(1), N = B->size(2);
    const at::ScalarType type = u->scalar_type();
    const int32_t io = io_code(u);
    need(delta, type, {batch, heads}, dev);
    if (heads == dim) need(A, at::kFloat, {dim, N}, dev, false);
    else need(A, at::kFloat, {heads}, dev, false);
    need(B, type, {batch, groups, N}, dev);
    need(C, type, {batch, groups, N}, dev, false);
    need(D, at::kFloat, {dim}, dev);
    need(z, type, {batch, dim}, dev);
    need(bias, at::kFloat, {heads}, dev);
    need(out, type, {batch, dim}, dev);
    need(slots, at::kInt, {batch}, dev);
    const int64_t stride = pool_stride(states, at::kFloat, dim, N, dev);
    need_apart(out, {&u, &z}, true);
    need_apart(out, {&delta, &B, &C, &A, &D, &bias, &states, &slots});
    const ssm_dims_t d = {batch, dim, 1, N, heads, groups, io, 0};
    const Launch on(dev);
    Tensor o = out_or(out, *u, (bool)slots);
    check(entry.state_update(&d, static_cast<float*>(states.ptr()), i32(slots), states->size(0), stride, u.ptr(), delta.ptr(),
                             f32(A), B.ptr(), C.ptr(), f32(D), z.ptr(), f32(bias), softplus, o.data_ptr(), on.stream),
          "ssm_selective_state_update_slots");
    return THPVariable_Wrap(o);
}

// (pool, src, dst, slot_dim)
PyObject* slots_copy(PyObject* const* v) {
    const Arg pool("pool", v[0]), src("src", v[1]), dst("dst", v[2]);
    const int64_t at_dim = whole(v[3]);
    if (!pool || !pool->is_cuda()) refuse("%s must be a CUDA tensor%s", pool.name);
    if (at_dim < 0 || at_dim > 1 || pool->dim() <= at_dim) refuse("%s must be 0, or 1 behind a dimension of layers%s", "slot_dim");
    if (!pool->is_contiguous() && !inner_contiguous(*pool, at_dim + 1)) refuse("every slot of %s must be contiguous%s", pool.name);
    need_rank(src, 1);
    const int dev = pool->get_device();
    const int64_t n = src->size(0), e = pool->element_size(), slots = pool->size(at_dim);
    need(src, at::kInt, {n}, dev);
    need(dst, at::kInt, {n}, dev, false);
    int64_t slot_bytes = e;
    for (int64_t i = at_dim + 1; i < pool->dim(); ++i) slot_bytes *= pool->size(i);
    const Launch on(dev);
    // a single slot's stride says nothing
    check(entry.slots_copy(pool.ptr(), at_dim ? pool->size(0) : 1, slots, slot_bytes,
                           slots > 1 ? pool->stride(at_dim) * e : slot_bytes, at_dim ? pool->stride(0) * e : 0, i32(src),
                           i32(dst), n, on.stream),
          "ssm_state_slots_copy");
    Py_INCREF(v[0]);
    return v[0];
}

// ({entry point: address}, exception class)
PyObject* bind(PyObject* const* v) {
    const struct {
        const char* name;
        void* to;
    } all[] = {{"ssm_causal_conv1d_fwd", &entry.conv_fwd},
               {"ssm_causal_conv1d_bwd_workspace_size", &entry.conv_bwd_size},
               {"ssm_causal_conv1d_bwd", &entry.conv_bwd},
               {"ssm_causal_conv1d_packed_fwd", &entry.conv_packed},
               {"ssm_causal_conv1d_update", &entry.conv_update},
               {"ssm_selective_scan_packed_workspace_size", &entry.scan_packed_size},
               {"ssm_selective_scan_packed_fwd", &entry.scan_packed},
               {"ssm_selective_state_update_slots", &entry.state_update},
               {"ssm_state_slots_copy", &entry.slots_copy}};
    for (const auto& a : all) {
        PyObject* o = PyMapping_GetItemString(v[0], a.name);
        if (!o) throw Refused();
        void* p = PyLong_AsVoidPtr(o);
        Py_DECREF(o);
        if (!p) throw Refused();
        std::memcpy(a.to, &p, sizeof p);
    }
    Py_INCREF(v[1]);
    Py_XSETREF(error_class, v[1]);
    Py_RETURN_NONE;
}

// torch's exceptions (out of memory among them) become Python's here; none crosses into Python.
template <PyObject* (*F)(PyObject* const*), int N>
PyObject* entry_point(PyObject*, PyObject* const* args, Py_ssize_t n) {
    HANDLE_TH_ERRORS
    if (n != N) {
        PyErr_Format(PyExc_TypeError, "%d arguments wanted, %zd given", N, n);
        return nullptr;
    }
    try {
        return F(args);
    } catch (const Refused&) {
        return nullptr;
    }
    END_HANDLE_TH_ERRORS
}

#define METHOD(f, n) {#f, (PyCFunction)(void (*)(void)) & entry_point<f, n>, METH_FASTCALL, nullptr}
PyMethodDef methods[] = {METHOD(bind, 2),       METHOD(conv_fwd, 5),     METHOD(conv_bwd, 6),
                         METHOD(conv_packed, 9), METHOD(conv_update, 7),  METHOD(scan_packed, 16),
                         METHOD(state_update, 12), METHOD(slots_copy, 4), {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_front", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__front() { return PyModule_Create(&module); }
