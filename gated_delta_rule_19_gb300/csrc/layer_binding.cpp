// layer_binding.cpp -- the Python binding of the linear-attention layer's calls and of those
// around it in its block (include/gdn.h) on torch tensors: the same checks, allocations and errors as gdn.py's,
// in C++.  A decode step's kernel takes a few microseconds; marshalling one call in
// Python took 13 us on the benchmark's host, here it takes 3.4 (the launch is 2.5 of them;
// 4.2 with a program's own Python between the calls).
//
// The functions take positional arguments only; gdn.py has their signatures and
// documentation.  An argument that may be left out is None.

#include <Python.h>

#include <ATen/EmptyTensor.h>
#include <ATen/core/Tensor.h>
#include <c10/core/DeviceGuard.h>
#include <c10/core/impl/VirtualGuardImpl.h>
#include <c10/cuda/CUDACachingAllocator.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <dlfcn.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include <cstdarg>
#include <cstdio>
#include <memory>
#include <optional>
#include <string>
#include <vector>

#include "gdn.h"

namespace {

// The library's entry points, looked up by load().
struct Api {
#define GDN_LAYER_CALLS(F)                                                                                      \
    F(gdn_last_error) F(gdn_la_fwd_workspace_bytes) F(gdn_la_saved_bytes) F(gdn_la_bwd_workspace_bytes)          \
    F(gdn_la_fwd) F(gdn_la_bwd) F(gdn_la_decode) F(gdn_qk_norm_rope_fwd)                                         \
    F(gdn_qk_norm_rope_bwd_workspace_bytes) F(gdn_qk_norm_rope_bwd) F(gdn_gated_norm_fwd)                        \
    F(gdn_gated_norm_bwd_workspace_bytes) F(gdn_gated_norm_bwd)
// The block's, which a library of the layer alone lacks: their calls then raise.
#define GDN_BLOCK_CALLS(F)                                                                                      \
    F(gdn_qk_norm_rope_axes_fwd_workspace_bytes) F(gdn_qk_norm_rope_axes_fwd)                                    \
    F(gdn_qk_norm_rope_axes_bwd_workspace_bytes) F(gdn_qk_norm_rope_axes_bwd)                                    \
    F(gdn_add_norm_fwd) F(gdn_add_norm_quant)                                                                   \
    F(gdn_add_norm_bwd_workspace_bytes) F(gdn_add_norm_bwd) F(gdn_grad_workspace_bytes) F(gdn_grad_norm)         \
    F(gdn_clip_grads) F(gdn_state_store) F(gdn_state_load)
#define GDN_FIELD(name) decltype(&::name) name = nullptr;
    GDN_LAYER_CALLS(GDN_FIELD) GDN_BLOCK_CALLS(GDN_FIELD)
#undef GDN_FIELD
} api;

PyObject* error_type = nullptr;  // gdn.GdnError

struct Error {
    int status;
    std::string text;
};
struct PythonError {};  // a Python exception is set

[[noreturn]] void fail(int status, const char* fmt, ...) {
    char s[512];
    va_list ap;
    va_start(ap, fmt);
    vsnprintf(s, sizeof(s), fmt, ap);
    va_end(ap);
    throw Error{status, s};
}
[[noreturn]] void invalid(const std::string& text) { throw Error{GDN_ERR_INVALID_ARG, text}; }

std::string shape_text(at::IntArrayRef s) {
    std::string t = "(";
    for (size_t i = 0; i < s.size(); ++i) t += (i ? ", " : "") + std::to_string(s[i]);
    return t + (s.size() == 1 ? ",)" : ")");
}

// A tensor argument; NULL for None where that is allowed.
const at::Tensor* tensor(PyObject* o, const char* name, bool optional = false) {
    if (o == Py_None) {
        if (optional) return nullptr;
        invalid(std::string(name) + " is required");
    }
    if (!THPVariable_Check(o)) {
        PyErr_Format(PyExc_TypeError, "%s must be a torch.Tensor", name);
        throw PythonError{};
    }
    return &THPVariable_Unpack(o);
}

// What every tensor of a call has in common: the first one's device and type.
struct Like {
    at::Device device;
    at::ScalarType type;
    int code;
    Like(const at::Tensor& t, const char* name) : Like(t, name, t.dim() == 4, "four dimensions") {}
    Like(const at::Tensor& t, const char* name, bool shaped, const char* expected)
        : device(t.device()), type(t.scalar_type()) {
        if (!t.is_cuda()) invalid("inputs must be CUDA tensors");
        if (!shaped) invalid(std::string(name) + " has shape " + shape_text(t.sizes()) + ", expected " + expected);
        if (type == at::kFloat) code = GDN_F32;
        else if (type == at::kBFloat16) code = GDN_BF16;
        else fail(GDN_ERR_UNSUPPORTED, "dtype %s (use float32 or bfloat16)", c10::toString(type));
    }
    // at::empty's own steps without its dispatch: a call makes four to six tensors.  Under an
    // OnStream, whose device and stream they belong to.
    at::Tensor empty(at::IntArrayRef shape, at::ScalarType t) const {
        return at::Tensor(at::detail::empty_generic(shape, c10::cuda::CUDACachingAllocator::get(),
                                                    c10::DispatchKeySet(c10::DispatchKey::CUDA), t, std::nullopt));
    }
};

void check(const at::Tensor& t, const char* name, at::IntArrayRef shape, at::ScalarType type, at::Device device) {
    if (t.scalar_type() != type)
        fail(GDN_ERR_INVALID_ARG, "%s has dtype %s, expected %s", name, c10::toString(t.scalar_type()),
             c10::toString(type));
    if (t.sizes() != shape)
        invalid(std::string(name) + " has shape " + shape_text(t.sizes()) + ", expected " + shape_text(shape));
    if (t.device() != device)
        invalid(std::string(name) + " is on " + t.device().str() + ", expected " + device.str());
}

// A [B, T, H, D] tensor whose tokens lie a fixed stride apart: that stride in elements
// (0: dense).
int64_t rows(const at::Tensor& t, const char* name, at::IntArrayRef s, const Like& like) {
    check(t, name, s, like.type, like.device);
    if (t.is_contiguous() || t.numel() == 0) return 0;
    const int64_t token = s[1] > 1 ? t.stride(1) : t.stride(0);
    if ((s[3] > 1 && t.stride(3) != 1) || (s[2] > 1 && t.stride(2) != s[3]) ||
        (s[0] > 1 && s[1] > 1 && t.stride(0) != s[1] * t.stride(1)) || (s[0] * s[1] > 1 && token < s[2] * s[3]))
        invalid(std::string(name) + " must be dense in its last two dimensions and its tokens a fixed stride apart, " +
                "got strides " + shape_text(t.strides()));
    return s[0] * s[1] > 1 ? token : 0;
}

const at::Tensor& dense(const at::Tensor& t, const char* name, at::IntArrayRef shape, at::ScalarType type,
                        const Like& like) {
    check(t, name, shape, type, like.device);
    if (!t.is_contiguous()) invalid(std::string(name) + " must be contiguous");
    return t;
}

// A dense input's address (NULL for None where that is allowed).
void* input(PyObject* o, const char* name, at::IntArrayRef shape, at::ScalarType type, const Like& like,
            bool optional = false) {
    const at::Tensor* t = tensor(o, name, optional);
    return t ? dense(*t, name, shape, type, like).data_ptr() : nullptr;
}

// An output to fill: the caller's, or a new one.
at::Tensor output(PyObject* o, const char* name, at::IntArrayRef shape, at::ScalarType type, const Like& like) {
    const at::Tensor* t = tensor(o, name, true);
    return t ? dense(*t, name, shape, type, like) : like.empty(shape, type);
}

// A state to fill: True a new one, False or None none.
std::optional<at::Tensor> state_output(PyObject* o, const char* name, at::IntArrayRef shape, const Like& like) {
    if (o == Py_None || o == Py_False) return std::nullopt;
    return output(o == Py_True ? Py_None : o, name, shape, at::kFloat, like);
}

// A caller's buffer of bytes.
const at::Tensor& bytes_of(const at::Tensor& t, const char* name, const Like& like) {
    if (t.device() != like.device || !t.is_contiguous())
        invalid(std::string(name) + " must be a contiguous tensor on " + like.device.str());
    return t;
}

// The workspace: the caller's, or (None) memory of `need()` bytes for the time of the call.
struct Workspace {
    c10::DataPtr own;
    void* at;
    size_t bytes;
    template <typename Need>
    Workspace(PyObject* o, const Like& like, Need&& need) {
        if (const at::Tensor* given = tensor(o, "workspace", true)) {
            const at::Tensor& t = bytes_of(*given, "workspace", like);
            at = t.data_ptr();
            bytes = (size_t)t.numel() * t.element_size();
        } else {
            bytes = need();
            if (bytes) own = c10::cuda::CUDACachingAllocator::get()->allocate(bytes);
            at = own.get();
        }
    }
};

// The call's device, which is the tensors' (the library launches on the current one), and
// its stream: the given one, or that device's current one.  What the call makes belongs to
// them: a workspace that goes back to the current stream would be handed out again while
// the given one still has to run.
struct OnStream {
    c10::DeviceGuard device;
    void* raw;
    std::optional<c10::cuda::CUDAStreamGuard> guard;
    OnStream(PyObject* o, const Like& like) : device(like.device) {
        const c10::cuda::CUDAStream now(c10::impl::VirtualGuardImpl(like.device.type()).getStream(like.device));
        raw = now.stream();
        if (o == Py_None) return;
        raw = PyLong_AsVoidPtr(o);
        if (!raw && PyErr_Occurred()) throw PythonError{};
        if (raw != now.stream())
            guard.emplace(c10::cuda::getStreamFromExternal((cudaStream_t)raw, like.device.index()));
    }
};

void done(gdn_status st) {
    if (st != GDN_OK) throw Error{(int)st, api.gdn_last_error()};
}

float* data(const std::optional<at::Tensor>& t) { return t ? t->data_ptr<float>() : nullptr; }

PyObject* wrap(const at::Tensor& t) { return THPVariable_Wrap(t); }
PyObject* wrap(const std::optional<at::Tensor>& t) {
    if (t) return THPVariable_Wrap(*t);
    Py_RETURN_NONE;
}
// What the call wrote counts as changed, so that autograd sees a saved state that was
// overwritten (tensors of inference mode have no count).
void changed(const at::Tensor& t) {
    if (!t.is_inference()) t.unsafeGetTensorImpl()->bump_version();
}
void changed(const std::optional<at::Tensor>& t) {
    if (t) changed(*t);
}
template <typename... T>
PyObject* results(const T&... t) {
    (changed(t), ...);
    PyObject* r = PyTuple_New(sizeof...(T));
    Py_ssize_t i = 0;
    (PyTuple_SET_ITEM(r, i++, wrap(t)), ...);
    return r;
}

float as_float(PyObject* o) {
    const double x = PyFloat_AsDouble(o);
    if (x == -1.0 && PyErr_Occurred()) throw PythonError{};
    return (float)x;
}

// Runs a call's body; its C++ exceptions become Python's.
template <typename F>
PyObject* call(Py_ssize_t given, Py_ssize_t want, F&& body) {
    if (given != want) {
        PyErr_Format(PyExc_TypeError, "expected %zd arguments, got %zd", want, given);
        return nullptr;
    }
    if (!api.gdn_la_fwd) {
        PyErr_SetString(PyExc_RuntimeError, "the library is not loaded");
        return nullptr;
    }
    try {
        return body();
    } catch (const Error& e) {
        if (PyObject* x = PyObject_CallFunction(error_type, "is", e.status, e.text.c_str())) {
            PyErr_SetObject(error_type, x);
            Py_DECREF(x);
        }
    } catch (const PythonError&) {
    } catch (const std::exception&) {  // torch's own: an allocation that failed is its OutOfMemoryError
        torch::translate_exception_to_python(std::current_exception());
    }
    return nullptr;
}

// --------------------------------------------------------- linear attention

struct La {
    const at::Tensor &q, &k, &v;
    Like like;
    int64_t B, T, H, K, V;
    gdn_la_problem p;
    const float* log_decay;
    La(PyObject* const* a)
        : q(*tensor(a[0], "q")), k(*tensor(a[1], "k")), v(*tensor(a[2], "v")), like(q, "q") {
        Like(v, "v");
        B = q.size(0), T = q.size(1), H = q.size(2), K = q.size(3), V = v.size(3);
        p = {B, T, H, K, V, rows(q, "q", q.sizes(), like), rows(k, "k", q.sizes(), like),
             rows(v, "v", {B, T, H, V}, like), like.code};
        log_decay = (const float*)input(a[3], "log_decay", {H}, at::kFloat, like);
    }
};

// q, k, v, log_decay, initial_state, o, final_state, saved, workspace, stream
PyObject* la_fwd(PyObject*, PyObject* const* a, Py_ssize_t n) {
    return call(n, 10, [&] {
        La c(a);
        const OnStream stream(a[9], c.like);
        const at::DimVector state{c.B, c.H, c.V, c.K};
        const void* s0 = input(a[4], "initial_state", state, at::kFloat, c.like, true);
        const at::Tensor o = output(a[5], "o", {c.B, c.T, c.H, c.V}, c.like.type, c.like);
        const auto sT = state_output(a[6], "final_state", state, c.like);
        std::optional<at::Tensor> saved;
        if (a[7] != Py_None && a[7] != Py_False) {
            const size_t need = api.gdn_la_saved_bytes(&c.p);
            if (a[7] == Py_True) saved = c.like.empty({(int64_t)need}, at::kByte);
            else saved = bytes_of(*tensor(a[7], "saved"), "saved", c.like);
            if ((size_t)saved->nbytes() < need) invalid("saved buffer is smaller than gdn_la_saved_bytes()");
        }
        const Workspace ws(a[8], c.like, [&] { return api.gdn_la_fwd_workspace_bytes(&c.p); });
        done(api.gdn_la_fwd(&c.p, c.q.data_ptr(), c.k.data_ptr(), c.v.data_ptr(), c.log_decay, (const float*)s0,
                            o.data_ptr(), data(sT), saved ? saved->data_ptr() : nullptr, ws.at, ws.bytes,
                            stream.raw));
        return results(o, sT, saved);
    });
}

// q, k, v, log_decay, initial_state, d_o, d_final_state, saved, dq, dk, dv, d_initial_state,
// workspace, stream
PyObject* la_bwd(PyObject*, PyObject* const* a, Py_ssize_t n) {
    return call(n, 14, [&] {
        La c(a);
        const OnStream stream(a[13], c.like);
        const at::DimVector state{c.B, c.H, c.V, c.K}, vs{c.B, c.T, c.H, c.V};
        const void* s0 = input(a[4], "initial_state", state, at::kFloat, c.like, true);
        const void* d_o = input(a[5], "d_o", vs, c.like.type, c.like);
        const void* dS = input(a[6], "d_final_state", state, at::kFloat, c.like, true);
        const void* saved = nullptr;
        if (a[7] != Py_None) {
            const at::Tensor& b = bytes_of(*tensor(a[7], "saved"), "saved", c.like);
            if ((size_t)b.nbytes() < api.gdn_la_saved_bytes(&c.p))
                invalid("saved buffer is smaller than gdn_la_saved_bytes()");
            saved = b.data_ptr();
        }
        const at::Tensor dq = output(a[8], "dq", c.q.sizes(), c.like.type, c.like),
                         dk = output(a[9], "dk", c.q.sizes(), c.like.type, c.like),
                         dv = output(a[10], "dv", vs, c.like.type, c.like);
        const auto ds0 = state_output(a[11], "d_initial_state", state, c.like);
        const Workspace ws(a[12], c.like, [&] { return api.gdn_la_bwd_workspace_bytes(&c.p); });
        done(api.gdn_la_bwd(&c.p, c.q.data_ptr(), c.k.data_ptr(), c.v.data_ptr(), c.log_decay, (const float*)s0, saved,
                            d_o, (const float*)dS, dq.data_ptr(), dk.data_ptr(), dv.data_ptr(), data(ds0), ws.at,
                            ws.bytes, stream.raw));
        return results(dq, dk, dv, ds0);
    });
}

// q, k, v, log_decay, state, o, stream
PyObject* la_decode(PyObject*, PyObject* const* a, Py_ssize_t n) {
    return call(n, 7, [&] {
        La c(a);
        const OnStream stream(a[6], c.like);
        const at::Tensor& state = *tensor(a[4], "state");
        dense(state, "state", {c.B, c.H, c.V, c.K}, at::kFloat, c.like);
        const at::Tensor o = output(a[5], "o", {c.B, c.T, c.H, c.V}, c.like.type, c.like);
        done(api.gdn_la_decode(&c.p, c.q.data_ptr(), c.k.data_ptr(), c.v.data_ptr(), c.log_decay,
                               state.data_ptr<float>(), o.data_ptr(), stream.raw));
        return results(o, state);
    });
}

// ------------------------------------------------ norm and rotation of q and k

struct Rope {
    const at::Tensor &q, &k;
    Like like;
    at::DimVector ks;
    gdn_rope_problem p;
    const void *wq, *wk;
    const float *cos = nullptr, *sin = nullptr;
    const int32_t* positions;
    // q, k, q_weight, k_weight, cos, sin, positions, then eps, interleaved
    Rope(PyObject* const* a, PyObject* eps, PyObject* interleaved)
        : q(*tensor(a[0], "q")), k(*tensor(a[1], "k")), like(q, "q") {
        Like(k, "k");
        const int64_t B = q.size(0), T = q.size(1), D = q.size(3);
        ks = {B, T, k.size(2), D};
        int64_t table = 0, pairs = 0;
        if (a[4] != Py_None || a[5] != Py_None) {
            const at::Tensor& c = *tensor(a[4], "cos");
            if (c.dim() != 2) invalid("cos must be a [table_rows, R/2] tensor");
            table = c.size(0), pairs = c.size(1);
            cos = (const float*)input(a[4], "cos", {table, pairs}, at::kFloat, like);
            sin = (const float*)input(a[5], "sin", {table, pairs}, at::kFloat, like);
        }
        wq = input(a[2], "q_weight", {D}, like.type, like);
        wk = input(a[3], "k_weight", {D}, like.type, like);
        positions = (const int32_t*)input(a[6], "positions", {B, T}, at::kInt, like, true);
        const int inter = PyObject_IsTrue(interleaved);
        if (inter < 0) throw PythonError{};
        p = {B, T, q.size(2), k.size(2), D, 2 * pairs, table, rows(q, "q", q.sizes(), like), rows(k, "k", ks, like),
             as_float(eps), inter, like.code};
    }
};

// q, k, q_weight, k_weight, cos, sin, positions, eps, interleaved, q_out, k_out, stream
PyObject* rope_fwd(PyObject*, PyObject* const* a, Py_ssize_t n) {
    return call(n, 12, [&] {
        Rope c(a, a[7], a[8]);
        const OnStream stream(a[11], c.like);
        const at::Tensor qo = output(a[9], "q_out", c.q.sizes(), c.like.type, c.like),
                         ko = output(a[10], "k_out", c.ks, c.like.type, c.like);
        done(api.gdn_qk_norm_rope_fwd(&c.p, c.q.data_ptr(), c.k.data_ptr(), c.wq, c.wk, c.cos, c.sin, c.positions,
                                      qo.data_ptr(), ko.data_ptr(), stream.raw));
        return results(qo, ko);
    });
}

// q, k, q_weight, k_weight, cos, sin, positions, dq_out, dk_out, eps, interleaved, dq, dk,
// dq_weight, dk_weight, workspace, stream
PyObject* rope_bwd(PyObject*, PyObject* const* a, Py_ssize_t n) {
    return call(n, 17, [&] {
        Rope c(a, a[9], a[10]);
        const OnStream stream(a[16], c.like);
        const at::DimVector width{c.p.D};
        const void *dqo = input(a[7], "dq_out", c.q.sizes(), c.like.type, c.like),
                   *dko = input(a[8], "dk_out", c.ks, c.like.type, c.like);
        const at::Tensor dq = output(a[11], "dq", c.q.sizes(), c.like.type, c.like),
                         dk = output(a[12], "dk", c.ks, c.like.type, c.like),
                         dwq = output(a[13], "dq_weight", width, c.like.type, c.like),
                         dwk = output(a[14], "dk_weight", width, c.like.type, c.like);
        const Workspace ws(a[15], c.like, [&] { return api.gdn_qk_norm_rope_bwd_workspace_bytes(&c.p); });
        done(api.gdn_qk_norm_rope_bwd(&c.p, c.q.data_ptr(), c.k.data_ptr(), c.wq, c.wk, c.cos, c.sin, c.positions, dqo,
                                      dko, dq.data_ptr(), dk.data_ptr(), dwq.data_ptr(), dwk.data_ptr(), ws.at,
                                      ws.bytes, stream.raw));
        return results(dq, dk, dwq, dwk);
    });
}

// ----------------------------------------------------------------- gated norm

struct Gated {
    const at::Tensor &x, &gate;
    Like like;
    gdn_gated_norm_problem p;
    const void* weight;
    Gated(PyObject* const* a, PyObject* eps)
        : x(*tensor(a[0], "x")), gate(*tensor(a[1], "gate")), like(x, "x") {
        weight = input(a[2], "weight", {x.size(3)}, like.type, like);
        p = {x.size(0), x.size(1), x.size(2), x.size(3), rows(x, "x", x.sizes(), like),
             rows(gate, "gate", x.sizes(), like), as_float(eps), like.code};
    }
};

// x, gate, weight, eps, y, stream
PyObject* gated_fwd(PyObject*, PyObject* const* a, Py_ssize_t n) {
    return call(n, 6, [&] {
        Gated c(a, a[3]);
        const OnStream stream(a[5], c.like);
        const at::Tensor y = output(a[4], "y", c.x.sizes(), c.like.type, c.like);
        done(api.gdn_gated_norm_fwd(&c.p, c.x.data_ptr(), c.gate.data_ptr(), c.weight, y.data_ptr(),
                                    stream.raw));
        changed(y);
        return wrap(y);
    });
}

// x, gate, weight, dy, eps, dx, dgate, dweight, workspace, stream
PyObject* gated_bwd(PyObject*, PyObject* const* a, Py_ssize_t n) {
    return call(n, 10, [&] {
        Gated c(a, a[4]);
        const OnStream stream(a[9], c.like);
        const void* dy = input(a[3], "dy", c.x.sizes(), c.like.type, c.like);
        const at::Tensor dx = output(a[5], "dx", c.x.sizes(), c.like.type, c.like),
                         dz = output(a[6], "dgate", c.x.sizes(), c.like.type, c.like),
                         dw = output(a[7], "dweight", {c.p.D}, c.like.type, c.like);
        const Workspace ws(a[8], c.like, [&] { return api.gdn_gated_norm_bwd_workspace_bytes(&c.p); });
        done(api.gdn_gated_norm_bwd(&c.p, c.x.data_ptr(), c.gate.data_ptr(), c.weight, dy, dx.data_ptr(),
                                    dz.data_ptr(), dw.data_ptr(), ws.at, ws.bytes, stream.raw));
        return results(dx, dz, dw);
    });
}

// ------------------------------------------- norm and rotation by several positions

struct RopeAxes {
    const at::Tensor &q, &k;
    Like like;
    at::DimVector ks;
    gdn_rope_axes_problem p{};
    const void *wq, *wk;
    const float *cos = nullptr, *sin = nullptr;
    const int32_t* positions;
    // q, k, q_weight, k_weight, cos, sin, positions, sections, then eps, interleaved, alternating
    RopeAxes(PyObject* const* a, PyObject* eps, PyObject* interleaved, PyObject* alternating)
        : q(*tensor(a[0], "q")), k(*tensor(a[1], "k")), like(q, "q") {
        Like(k, "k");
        const int64_t B = q.size(0), T = q.size(1), D = q.size(3);
        ks = {B, T, k.size(2), D};
        const at::Tensor& c = *tensor(a[4], "cos");
        if (c.dim() != 2) invalid("cos must be a [table_rows, R/2] tensor");
        const int64_t table = c.size(0), pairs = c.size(1);
        cos = (const float*)input(a[4], "cos", {table, pairs}, at::kFloat, like);
        sin = (const float*)input(a[5], "sin", {table, pairs}, at::kFloat, like);
        wq = input(a[2], "q_weight", {D}, like.type, like);
        wk = input(a[3], "k_weight", {D}, like.type, like);
        PyObject* parts = PySequence_Fast(a[7], "sections must be a sequence of whole numbers");
        if (!parts) throw PythonError{};
        const Py_ssize_t n = PySequence_Fast_GET_SIZE(parts);
        bool whole = true;
        for (Py_ssize_t i = 0; i < n && i < 4; ++i) {
            const long x = PyLong_AsLong(PySequence_Fast_GET_ITEM(parts, i));
            whole = whole && !(x == -1 && PyErr_Occurred());
            p.sections[i] = x < -1 || x > 1 << 20 ? -1 : (int32_t)x;
            if (!whole) break;
        }
        Py_DECREF(parts);
        if (!whole) throw PythonError{};
        if (n < 1 || n > 4) fail(GDN_ERR_UNSUPPORTED, "sections has %zd entries, expected 1 to 4", n);
        p.axes = (int32_t)n;
        positions = (const int32_t*)input(a[6], "positions", {(int64_t)n, B, T}, at::kInt, like);
        const int inter = PyObject_IsTrue(interleaved), alt = PyObject_IsTrue(alternating);
        if (inter < 0 || alt < 0) throw PythonError{};
        p.alternating = alt;
        p.rope = {B, T, q.size(2), k.size(2), D, 2 * pairs, table, rows(q, "q", q.sizes(), like),
                  rows(k, "k", ks, like), as_float(eps), inter, like.code};
    }
};

bool have_block() {
    if (api.gdn_state_load) return true;
    PyErr_SetString(PyExc_RuntimeError, "the library lacks the block's calls: build it again");
    return false;
}

// q, k, q_weight, k_weight, cos, sin, positions, sections, eps, interleaved, alternating, q_out,
// k_out, workspace, stream
PyObject* rope_axes_fwd(PyObject*, PyObject* const* a, Py_ssize_t n) {
    return !have_block() ? nullptr : call(n, 15, [&] {
        RopeAxes c(a, a[8], a[9], a[10]);
        const OnStream stream(a[14], c.like);
        const at::Tensor qo = output(a[11], "q_out", c.q.sizes(), c.like.type, c.like),
                         ko = output(a[12], "k_out", c.ks, c.like.type, c.like);
        const Workspace ws(a[13], c.like, [&] { return api.gdn_qk_norm_rope_axes_fwd_workspace_bytes(&c.p); });
        done(api.gdn_qk_norm_rope_axes_fwd(&c.p, c.q.data_ptr(), c.k.data_ptr(), c.wq, c.wk, c.cos, c.sin, c.positions,
                                           qo.data_ptr(), ko.data_ptr(), ws.at, ws.bytes, stream.raw));
        return results(qo, ko);
    });
}

// q, k, q_weight, k_weight, cos, sin, positions, sections, dq_out, dk_out, eps, interleaved,
// alternating, dq, dk, dq_weight, dk_weight, workspace, stream
PyObject* rope_axes_bwd(PyObject*, PyObject* const* a, Py_ssize_t n) {
    return !have_block() ? nullptr : call(n, 19, [&] {
        RopeAxes c(a, a[10], a[11], a[12]);
        const OnStream stream(a[18], c.like);
        const at::DimVector width{c.p.rope.D};
        const void *dqo = input(a[8], "dq_out", c.q.sizes(), c.like.type, c.like),
                   *dko = input(a[9], "dk_out", c.ks, c.like.type, c.like);
        const at::Tensor dq = output(a[13], "dq", c.q.sizes(), c.like.type, c.like),
                         dk = output(a[14], "dk", c.ks, c.like.type, c.like),
                         dwq = output(a[15], "dq_weight", width, c.like.type, c.like),
                         dwk = output(a[16], "dk_weight", width, c.like.type, c.like);
        const Workspace ws(a[17], c.like, [&] { return api.gdn_qk_norm_rope_axes_bwd_workspace_bytes(&c.p); });
        done(api.gdn_qk_norm_rope_axes_bwd(&c.p, c.q.data_ptr(), c.k.data_ptr(), c.wq, c.wk, c.cos, c.sin, c.positions,
                                           dqo, dko, dq.data_ptr(), dk.data_ptr(), dwq.data_ptr(), dwk.data_ptr(),
                                           ws.at, ws.bytes, stream.raw));
        return results(dq, dk, dwq, dwk);
    });
}

// ------------------------------------------------- residual addition and norm

// A [..., D] tensor whose rows lie a fixed stride apart: that stride in elements (0: dense).
int64_t row_step(const at::Tensor& t, const char* name, at::IntArrayRef shape, at::ScalarType type, const Like& like) {
    check(t, name, shape, type, like.device);
    if (t.is_contiguous() || t.numel() == 0) return 0;
    const int64_t D = t.size(-1);
    int64_t step = 0, count = 1;  // of the rows seen so far
    bool even = D == 1 || t.stride(-1) == 1;
    for (int64_t i = t.dim() - 2; i >= 0; --i) {
        if (t.size(i) == 1) continue;
        if (count == 1) step = t.stride(i);
        even = even && t.stride(i) == step * count;
        count *= t.size(i);
    }
    if (!even || (count > 1 && step < D))
        invalid(std::string(name) + " must be dense in its last dimension and its rows a fixed stride apart, got strides " +
                shape_text(t.strides()));
    return count > 1 ? step : 0;
}

at::ScalarType stream_type(const at::Tensor& t, const char* name, const Like& like) {
    if (t.scalar_type() != like.type && t.scalar_type() != at::kFloat)
        fail(GDN_ERR_UNSUPPORTED, "%s has dtype %s, expected %s or Float", name, c10::toString(t.scalar_type()),
             c10::toString(like.type));
    return t.scalar_type();
}

// x, residual, weight, and the call's problem.
struct AddNorm {
    const at::Tensor& x;
    const at::Tensor* residual;
    Like like;
    at::ScalarType kept;  // h's type
    const void* weight;
    gdn_add_norm_problem p;
    AddNorm(PyObject* const* a, PyObject* eps)
        : x(*tensor(a[0], "x")), residual(tensor(a[1], "residual", true)),
          like(x, "x", x.dim() > 0 && x.size(-1) > 0, "rows in the last dimension") {
        kept = residual ? stream_type(*residual, "residual", like) : like.type;
        const int64_t D = x.size(-1);
        weight = input(a[2], "weight", {D}, like.type, like);
        p = {x.numel() / D, D, row_step(x, "x", x.sizes(), like.type, like),
             residual ? row_step(*residual, "residual", x.sizes(), kept, like) : 0, as_float(eps), like.code,
             kept == at::kFloat ? GDN_F32 : GDN_BF16};
    }
    // The sum: none without a residual; the caller's, or a new one.
    std::optional<at::Tensor> sum(PyObject* o) const {
        if (!residual) {
            if (o != Py_None) invalid("h is given without a residual: it would be x");
            return std::nullopt;
        }
        return output(o, "h", x.sizes(), kept, like);
    }
};

void* address(const std::optional<at::Tensor>& t) { return t ? t->data_ptr() : nullptr; }

// x, residual, weight, eps, h, y, stream
PyObject* add_norm_fwd(PyObject*, PyObject* const* a, Py_ssize_t n) {
    return !have_block() ? nullptr : call(n, 7, [&] {
        AddNorm c(a, a[3]);
        const OnStream stream(a[6], c.like);
        const auto h = c.sum(a[4]);
        const at::Tensor y = output(a[5], "y", c.x.sizes(), c.like.type, c.like);
        done(api.gdn_add_norm_fwd(&c.p, c.x.data_ptr(), c.residual ? c.residual->data_ptr() : nullptr, c.weight,
                                  address(h), y.data_ptr(), stream.raw));
        return results(y, h);
    });
}

// x, residual, weight, eps, group, h, y, scales, stream
PyObject* add_norm_quant(PyObject*, PyObject* const* a, Py_ssize_t n) {
    return !have_block() ? nullptr : call(n, 9, [&] {
        AddNorm c(a, a[3]);
        const OnStream stream(a[8], c.like);
        const long group = PyLong_AsLong(a[4]);
        if (group == -1 && PyErr_Occurred()) throw PythonError{};
        if (group < 0 || group > 128 || (group && c.p.D % group))
            fail(GDN_ERR_UNSUPPORTED, "group=%ld: must be 0, 32, 64 or 128 and divide D=%ld", group, (long)c.p.D);
        const auto h = c.sum(a[5]);
        const at::Tensor y = output(a[6], "y", c.x.sizes(), at::kFloat8_e4m3fn, c.like);
        at::DimVector parts(c.x.sizes().begin(), c.x.sizes().end());
        parts.back() = group ? c.p.D / group : 1;
        const at::Tensor scales = output(a[7], "scales", parts, at::kFloat, c.like);
        done(api.gdn_add_norm_quant(&c.p, (int32_t)group, c.x.data_ptr(), c.residual ? c.residual->data_ptr() : nullptr,
                                    c.weight, address(h), y.data_ptr(), scales.data_ptr<float>(), stream.raw));
        return results(y, scales, h);
    });
}

// h, weight, dy, dh, eps, dx, d_residual, dweight, workspace, stream
PyObject* add_norm_bwd(PyObject*, PyObject* const* a, Py_ssize_t n) {
    return !have_block() ? nullptr : call(n, 10, [&] {
        const at::Tensor &h = *tensor(a[0], "h"), &dy = *tensor(a[2], "dy");
        const Like like(dy, "dy", dy.dim() > 0 && dy.size(-1) > 0, "rows in the last dimension");
        const at::ScalarType kept = stream_type(h, "h", like);
        const OnStream stream(a[9], like);
        const int64_t D = dy.size(-1);
        const gdn_add_norm_problem p = {dy.numel() / D, D, 0, row_step(h, "h", dy.sizes(), kept, like), as_float(a[4]),
                                        like.code, kept == at::kFloat ? GDN_F32 : GDN_BF16};
        dense(dy, "dy", dy.sizes(), like.type, like);
        const void *w = input(a[1], "weight", {D}, like.type, like), *dh = input(a[3], "dh", dy.sizes(), kept, like, true);
        const bool apart = kept != like.type;
        const at::Tensor dx = output(a[5], "dx", dy.sizes(), like.type, like);
        if (!apart && a[6] != Py_None && !tensor(a[6], "d_residual")->is_same(dx))
            invalid("d_residual is given where the types agree: dx is both gradients");
        const at::Tensor dr = apart ? output(a[6], "d_residual", dy.sizes(), kept, like) : dx;
        const at::Tensor dw = output(a[7], "dweight", {D}, like.type, like);
        const Workspace ws(a[8], like, [&] { return api.gdn_add_norm_bwd_workspace_bytes(&p); });
        done(api.gdn_add_norm_bwd(&p, h.data_ptr(), w, dy.data_ptr(), dh, dx.data_ptr(), apart ? dr.data_ptr() : nullptr,
                                  dw.data_ptr(), ws.at, ws.bytes, stream.raw));
        return results(dx, dr, dw);
    });
}

// ------------------------------------------------------- the gradients' norm

// A reference of its own to a Python object: a member, so that a constructor that throws gives
// it back.
struct Release {
    void operator()(PyObject* o) const { Py_DECREF(o); }
};
using Owned = std::unique_ptr<PyObject, Release>;

// The tensors of a list (None is left out), with their outputs where there are some.
struct Grads {
    std::vector<gdn_grad> list;
    std::vector<const at::Tensor*> written;
    std::optional<Like> like;
    Owned seq, outs;
    const at::Tensor& one(PyObject* o, const char* what) {
        const at::Tensor& t = *tensor(o, what);
        if (t.layout() != at::kStrided || !t.is_non_overlapping_and_dense())
            invalid(std::string(what) + " must be dense in memory, got strides " +
                    (t.layout() == at::kStrided ? shape_text(t.strides()) : "of another layout"));
        const Like l(t, what, true, "");
        if (!like) like = l;
        else if (like->device != l.device) invalid(std::string(what) + " is on " + l.device.str() + ", expected " + like->device.str());
        return t;
    }
    static int32_t code(const at::Tensor& t) { return t.scalar_type() == at::kFloat ? GDN_F32 : GDN_BF16; }
    Grads(PyObject* tensors, PyObject* out, bool write) {
        if (THPVariable_Check(tensors)) invalid("grads must be a sequence of tensors");
        seq.reset(PySequence_Fast(tensors, "grads must be a sequence of tensors"));
        if (!seq) throw PythonError{};
        const Py_ssize_t n = PySequence_Fast_GET_SIZE(seq.get());
        if (out != Py_None) {
            if (THPVariable_Check(out)) invalid("out must be a sequence of tensors");
            outs.reset(PySequence_Fast(out, "out must be a sequence of tensors"));
            if (!outs) throw PythonError{};
            if (PySequence_Fast_GET_SIZE(outs.get()) != n)
                fail(GDN_ERR_INVALID_ARG, "out has %zd tensors, expected %zd", PySequence_Fast_GET_SIZE(outs.get()), n);
        }
        list.reserve(n);
        for (Py_ssize_t i = 0; i < n; ++i) {
            PyObject* o = PySequence_Fast_GET_ITEM(seq.get(), i);
            if (o == Py_None) continue;
            const at::Tensor& g = one(o, "a gradient");
            const at::Tensor& to = outs ? one(PySequence_Fast_GET_ITEM(outs.get(), i), "an output") : g;
            if (outs && (to.sizes() != g.sizes() || !(to.strides() == g.strides() || (to.is_contiguous() && g.is_contiguous()))))
                invalid("an output has shape " + shape_text(to.sizes()) + " and strides " + shape_text(to.strides()) +
                        ", its gradient " + shape_text(g.sizes()) + " and " + shape_text(g.strides()));
            list.push_back({g.data_ptr(), to.data_ptr(), g.numel(), code(g), code(to)});
            if (write) written.push_back(&to);
        }
    }
};

// The norm to fill: the caller's, or a new one on the gradients' device.
at::Tensor norm_output(PyObject* o, const Grads& g) {
    if (o != Py_None) {
        const at::Tensor& t = *tensor(o, "norm");
        const Like l(t, "norm", t.numel() == 1, "one element");
        if (l.type != at::kFloat) fail(GDN_ERR_INVALID_ARG, "norm has dtype %s, expected Float", c10::toString(l.type));
        if (g.like && g.like->device != l.device) invalid("norm is on " + l.device.str() + ", expected " + g.like->device.str());
        return t;
    }
    if (!g.like) invalid("no gradients: their device is not known (give norm)");
    return g.like->empty({}, at::kFloat);
}

PyObject* grads_call(PyObject* tensors, PyObject* out, const float* max_norm, PyObject* norm, PyObject* workspace,
                     PyObject* on) {
    Grads g(tensors, out, max_norm != nullptr);
    if (!g.like && norm != Py_None) {
        const at::Tensor& t = *tensor(norm, "norm");
        g.like.emplace(t, "norm", true, "");
    }
    if (!g.like) invalid("no gradients: their device is not known (give norm)");
    const OnStream stream(on, *g.like);
    const at::Tensor to = norm_output(norm, g);
    const int64_t count = (int64_t)g.list.size();
    const Workspace ws(workspace, *g.like, [&] { return api.gdn_grad_workspace_bytes(g.list.data(), count); });
    done(max_norm ? api.gdn_clip_grads(g.list.data(), count, *max_norm, to.data_ptr<float>(), ws.at, ws.bytes, stream.raw)
                  : api.gdn_grad_norm(g.list.data(), count, to.data_ptr<float>(), ws.at, ws.bytes, stream.raw));
    for (const at::Tensor* t : g.written) changed(*t);
    changed(to);
    return wrap(to);
}

// grads, norm, workspace, stream
PyObject* grad_norm(PyObject*, PyObject* const* a, Py_ssize_t n) {
    return !have_block() ? nullptr : call(n, 4, [&] { return grads_call(a[0], Py_None, nullptr, a[1], a[2], a[3]); });
}

// grads, max_norm, out, norm, workspace, stream
PyObject* clip_grads(PyObject*, PyObject* const* a, Py_ssize_t n) {
    return !have_block() ? nullptr : call(n, 6, [&] {
        const float most = as_float(a[1]);
        return grads_call(a[0], a[2], &most, a[3], a[4], a[5]);
    });
}

// ------------------------------------------------------- the cache of states

struct StateCache {
    const at::Tensor &cache, &scales, &slots;
    Like like;
    gdn_state_cache_problem p;
    StateCache(PyObject* cache_, PyObject* scales_, PyObject* slots_)
        : cache(*tensor(cache_, "cache")), scales(*tensor(scales_, "scales")), slots(*tensor(slots_, "slots")),
          like(scales, "scales", scales.dim() == 3, "[slots, H, V]") {
        if (cache.dim() != 4) invalid("cache has shape " + shape_text(cache.sizes()) + ", expected [slots, H, V, K]");
        if (slots.dim() != 1) invalid("slots has shape " + shape_text(slots.sizes()) + ", expected [B]");
        p = {slots.size(0), cache.size(1), cache.size(3), cache.size(2), cache.size(0)};
        dense(cache, "cache", cache.sizes(), at::kChar, like);
        dense(scales, "scales", {p.slots, p.H, p.V}, at::kFloat, like);
        dense(slots, "slots", {p.B}, at::kInt, like);
    }
};

// states, slots, cache, scales, stream
PyObject* state_store(PyObject*, PyObject* const* a, Py_ssize_t n) {
    return !have_block() ? nullptr : call(n, 5, [&] {
        const StateCache c(a[2], a[3], a[1]);
        const OnStream stream(a[4], c.like);
        const void* states = input(a[0], "states", {c.p.B, c.p.H, c.p.V, c.p.K}, at::kFloat, c.like);
        done(api.gdn_state_store(&c.p, (const float*)states, c.slots.data_ptr<int32_t>(), c.cache.data_ptr(),
                                 c.scales.data_ptr<float>(), stream.raw));
        return results(c.cache, c.scales);
    });
}

// cache, scales, slots, states, stream
PyObject* state_load(PyObject*, PyObject* const* a, Py_ssize_t n) {
    return !have_block() ? nullptr : call(n, 5, [&] {
        const StateCache c(a[0], a[1], a[2]);
        const OnStream stream(a[4], c.like);
        const at::Tensor states = output(a[3], "states", {c.p.B, c.p.H, c.p.V, c.p.K}, at::kFloat, c.like);
        done(api.gdn_state_load(&c.p, c.cache.data_ptr(), c.scales.data_ptr<float>(), c.slots.data_ptr<int32_t>(),
                                states.data_ptr<float>(), stream.raw));
        changed(states);
        return wrap(states);
    });
}

// load(path of libgdn.so, GdnError)
PyObject* load(PyObject*, PyObject* const* a, Py_ssize_t n) {
    if (n != 2 || !PyUnicode_Check(a[0]) || !PyType_Check(a[1])) {
        PyErr_SetString(PyExc_TypeError, "load(path, error type)");
        return nullptr;
    }
    void* lib = dlopen(PyUnicode_AsUTF8(a[0]), RTLD_NOW);
    Api found;
    const char* missing = lib ? nullptr : "the library";
#define GDN_LOOK(name)                                                            \
    if (lib && !(found.name = (decltype(found.name))dlsym(lib, #name))) missing = #name;
    GDN_LAYER_CALLS(GDN_LOOK)
#undef GDN_LOOK
#define GDN_LOOK(name) \
    if (lib) found.name = (decltype(found.name))dlsym(lib, #name);
    GDN_BLOCK_CALLS(GDN_LOOK)
#undef GDN_LOOK
    if (missing) {
        PyErr_Format(PyExc_RuntimeError, "%s: %s not found", PyUnicode_AsUTF8(a[0]), missing);
        return nullptr;
    }
    Py_INCREF(a[1]);
    Py_XDECREF(error_type);
    error_type = a[1];
    api = found;
    Py_RETURN_NONE;
}

#define GDN_METHOD(name) {#name, (PyCFunction)(void*)name, METH_FASTCALL, nullptr}
PyMethodDef methods[] = {GDN_METHOD(load),      GDN_METHOD(la_fwd),   GDN_METHOD(la_bwd),
                         GDN_METHOD(la_decode), GDN_METHOD(rope_fwd), GDN_METHOD(rope_bwd),
                         GDN_METHOD(gated_fwd), GDN_METHOD(gated_bwd), GDN_METHOD(rope_axes_fwd),
                         GDN_METHOD(rope_axes_bwd), GDN_METHOD(add_norm_fwd), GDN_METHOD(add_norm_quant),
                         GDN_METHOD(add_norm_bwd), GDN_METHOD(grad_norm), GDN_METHOD(clip_grads),
                         GDN_METHOD(state_store), GDN_METHOD(state_load), {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_layer", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__layer() { return PyModule_Create(&module); }
