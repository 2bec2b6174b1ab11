// Binding of the operators on tokens (mdcn_rotary_*, mdcn_attention_*): checks
// torch tensors, allocates outputs and workspaces that were not given, and
// calls the C ABI on the tensors' device and the current stream. Marshalling
// only, as in the ctypes binding of the other entry points; in C++ because a
// call on few tokens costs little more on the GPU than its launch, and reading
// ten tensors from Python takes several times as long.
//
// Every function returns its outputs, or the C call's status as an int where
// that is not MDCN_OK; what the binding itself finds wrong raises ValueError or
// TypeError before anything is called.
#include <Python.h>

#include <ATen/core/Tensor.h>
#include <ATen/cuda/EmptyTensor.h>
#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/autograd/python_variable.h>

#include <cmath>
#include <cstdint>
#include <optional>
#include <stdexcept>
#include <string>

#include "mdcn.h"

namespace {

// The library's functions, handed over by the package once it is loaded.
struct Library {
    decltype(&mdcn_rotary_forward) rotary_forward;
    decltype(&mdcn_rotary_backward) rotary_backward;
    decltype(&mdcn_rotary_backward_workspace_size) rotary_backward_size;
    decltype(&mdcn_attention_forward) attention_forward;
    decltype(&mdcn_attention_workspace_size) attention_size;
    decltype(&mdcn_attention_backward) attention_backward;
    decltype(&mdcn_attention_backward_workspace_size) attention_backward_size;
} lib;

// A check that failed: raised as ValueError, or TypeError.
struct Refusal {
    PyObject* type;
    std::string what;
};
[[noreturn]] void refuse(const std::string& what) { throw Refusal{PyExc_ValueError, what}; }
[[noreturn]] void refuse_type(const std::string& what) { throw Refusal{PyExc_TypeError, what}; }
struct Raised {};  // a Python exception is set

using Shape = c10::IntArrayRef;

std::string text(Shape s) {
    std::string t = "(";
    for (size_t i = 0; i < s.size(); ++i) t += (i ? ", " : "") + std::to_string(s[i]);
    return t + ")";
}

const at::Tensor& tensor(const char* name, PyObject* o) {
    if (!THPVariable_Check(o)) refuse_type(std::string(name) + " must be a tensor");
    return THPVariable_Unpack(o);
}

mdcn_dtype dtype_of(const at::Tensor& t) {
    switch (t.scalar_type()) {
        case at::kFloat: return MDCN_F32;
        case at::kHalf: return MDCN_F16;
        case at::kBFloat16: return MDCN_BF16;
        default: refuse_type("unsupported dtype (float32, float16 or bfloat16)");
    }
}

// What every other tensor of a call has to match.
struct Call {
    at::ScalarType type;
    c10::Device device = c10::Device(c10::kCPU);
    mdcn_dtype code;

    Call(const char* name, const at::Tensor& t) {
        if (t.dim() != 3) refuse(std::string(name) + " must be [tokens, heads, head_dim]");
        if (!t.is_cuda()) refuse(std::string(name) + " must be on a CUDA device");
        type = t.scalar_type();
        device = t.device();
        code = dtype_of(t);
    }
    // A [tokens][heads][head_dim] tensor of the given shape: its address, and its strides into s.
    void* view(const char* name, const at::Tensor& t, Shape shape, mdcn_strides& s) const {
        if (t.scalar_type() != type) refuse_type(std::string(name) + " must have the dtype of the other tensors");
        if (t.sizes() != shape) refuse(std::string(name) + " must have the shape " + text(shape) + ", not " + text(t.sizes()));
        if (t.device() != device) refuse(std::string(name) + " must be on the device of the other tensors");
        if (t.stride(2) != 1 && shape[2] > 1) refuse("the last index of " + std::string(name) + " must be contiguous");
        s.token = t.stride(0);
        s.head = t.stride(1);
        return t.data_ptr();
    }
    // A contiguous tensor of another kind (NULL for None).
    void* flat(const char* name, PyObject* o, at::ScalarType want, Shape shape) const {
        if (o == Py_None) return nullptr;
        const at::Tensor& t = tensor(name, o);
        if (t.scalar_type() != want) refuse_type(std::string(name) + " has the wrong dtype");
        if (t.sizes() != shape) refuse(std::string(name) + " must have the shape " + text(shape) + ", not " + text(t.sizes()));
        if (t.device() != device || !t.is_contiguous())
            refuse(std::string(name) + " must be contiguous and on the device of the other tensors");
        return t.data_ptr();
    }
    // From the caching allocator straight away: two outputs by way of the dispatcher take longer than
    // the rest of a call.
    at::Tensor make(Shape shape, at::ScalarType t) const {
        return at::Tensor(at::detail::empty_cuda(shape, t, device, std::nullopt));
    }
    // The workspace given (None: none) where it has the bytes, else a new one; its address and size.
    void* workspace(PyObject* o, size_t need, at::Tensor& keep, size_t& bytes, bool grow) const {
        bytes = 0;
        if (o != Py_None) {
            const at::Tensor& t = tensor("workspace", o);
            if (t.device() != device || !t.is_contiguous())
                refuse("workspace must be contiguous and on the device of the other tensors");
            bytes = static_cast<size_t>(t.numel()) * t.element_size();
            if (!grow || bytes >= need) return t.data_ptr();
        }
        if (!grow || need == 0) return nullptr;
        keep = make({static_cast<int64_t>(need)}, at::kByte);
        bytes = need;
        return keep.data_ptr();
    }
    void* stream(PyObject* o) const {
        if (o == Py_None) return c10::cuda::getCurrentCUDAStream(device.index()).stream();
        PyObject* v = PyObject_GetAttrString(o, "cuda_stream");
        if (!v) {
            PyErr_Clear();
            Py_INCREF(o);
            v = o;
        }
        void* p = PyLong_AsVoidPtr(v);
        Py_DECREF(v);
        if (!p && PyErr_Occurred()) throw Raised{};
        return p;
    }
};

double number(PyObject* o) {
    const double v = PyFloat_AsDouble(o);
    if (v == -1.0 && PyErr_Occurred()) throw Raised{};
    return v;
}
int64_t whole(PyObject* o) {
    const int64_t v = PyLong_AsLongLong(o);
    if (v == -1 && PyErr_Occurred()) throw Raised{};
    return v;
}
bool truth(PyObject* o) {
    const int v = PyObject_IsTrue(o);
    if (v < 0) throw Raised{};
    return v != 0;
}

PyObject* wrap(const at::Tensor& t) { return THPVariable_Wrap(t); }

// What given output is: o itself, or a new tensor where it is None.
struct Output {
    at::Tensor t;
    PyObject* given;
    PyObject* result() const {
        if (given) {
            Py_INCREF(given);
            return given;
        }
        if (!t.defined()) Py_RETURN_NONE;
        return wrap(t);
    }
};
Output output(const char* name, PyObject* o, const Call& c, Shape shape) {
    if (o == Py_None) return {c.make(shape, c.type), nullptr};
    return {tensor(name, o), o};
}

template <typename F>
PyObject* guarded(Py_ssize_t got, Py_ssize_t want, F body) {
    if (got != want) {
        PyErr_SetString(PyExc_TypeError, "wrong number of arguments");
        return nullptr;
    }
    try {
        return body();
    } catch (const Refusal& r) {
        PyErr_SetString(r.type, r.what.c_str());
    } catch (const Raised&) {
    } catch (const std::exception& e) {
        PyErr_SetString(PyExc_RuntimeError, e.what());
    }
    return nullptr;
}

PyObject* pack(std::initializer_list<const Output*> outs) {
    PyObject* r = PyTuple_New(static_cast<Py_ssize_t>(outs.size()));
    Py_ssize_t i = 0;
    for (const Output* o : outs) {
        PyObject* v = r ? o->result() : nullptr;
        if (!v) {
            Py_XDECREF(r);
            return nullptr;
        }
        PyTuple_SET_ITEM(r, i++, v);
    }
    return r;
}

// ---------------------------------------------------------------- rotary
struct Rotary {
    Call call;
    mdcn_rotary_attrs attrs{};
    mdcn_rotary_dims dims{};
    void *pos, *freq, *qw, *kw;
    Shape qshape, kshape;

    // q and k (or their outputs' gradients) give the shapes
    Rotary(const at::Tensor& q, const at::Tensor* k, PyObject* positions, PyObject* inv_freq, PyObject* sections,
           PyObject* layout, PyObject* norm, PyObject* q_weight, PyObject* k_weight, PyObject* eps)
        : call("q", q) {
        attrs.layout = static_cast<int32_t>(whole(layout));
        attrs.norm = truth(norm) ? 1 : 0;
        attrs.eps = static_cast<float>(number(eps));
        qshape = q.sizes();
        dims.tokens = qshape[0];
        dims.q_heads = qshape[1];
        dims.head_dim = qshape[2];
        if (k) {
            kshape = k->sizes();
            if (kshape.size() != 3 || kshape[0] != qshape[0] || kshape[2] != qshape[2])
                refuse("k must be [tokens, heads, head_dim] with the tokens and head_dim of q");
            dims.k_heads = kshape[1];
        } else if (k_weight != Py_None) {
            refuse("k_weight without k");
        }
        PyObject* s = PySequence_Fast(sections, "sections must be a sequence");
        if (!s) throw Raised{};
        const Py_ssize_t n = PySequence_Fast_GET_SIZE(s);
        int64_t pairs = 0;
        try {
            if (n < 1 || n > 4) refuse("1 to 4 sections");
            for (Py_ssize_t i = 0; i < n; ++i) {
                dims.sections[i] = whole(PySequence_Fast_GET_ITEM(s, i));
                pairs += dims.sections[i];
            }
        } catch (...) {
            Py_DECREF(s);
            throw;
        }
        Py_DECREF(s);
        dims.axes = n;
        if (positions == Py_None || inv_freq == Py_None) refuse_type("positions and inv_freq must be tensors");
        pos = call.flat("positions", positions, at::kInt, {dims.tokens, static_cast<int64_t>(n)});
        freq = call.flat("inv_freq", inv_freq, at::kFloat, {pairs});
        qw = call.flat("q_weight", q_weight, call.type, {dims.head_dim});
        kw = call.flat("k_weight", k_weight, call.type, {dims.head_dim});
    }
};

const at::Tensor* maybe(const char* name, PyObject* o) { return o == Py_None ? nullptr : &tensor(name, o); }

// (q, k, positions, inv_freq, sections, q_out, k_out, layout, norm, q_weight, k_weight, eps, stream) -> (q_out, k_out)
PyObject* rotary_forward(PyObject*, PyObject* const* a, Py_ssize_t n) {
    return guarded(n, 13, [&]() -> PyObject* {
        const at::Tensor& q = tensor("q", a[0]);
        const at::Tensor* k = maybe("k", a[1]);
        Rotary p(q, k, a[2], a[3], a[4], a[7], a[8], a[9], a[10], a[11]);
        if (!k && a[6] != Py_None) refuse("k_out is given exactly when k is");
        const Output qo = output("q_out", a[5], p.call, p.qshape);
        Output ko{at::Tensor(), nullptr};
        void* const qp = p.call.view("q", q, p.qshape, p.dims.q);
        void* const yp = p.call.view("q_out", qo.t, p.qshape, p.dims.q_out);
        void *kp = nullptr, *zp = nullptr;
        if (k) {
            ko = output("k_out", a[6], p.call, p.kshape);
            kp = p.call.view("k", *k, p.kshape, p.dims.k);
            zp = p.call.view("k_out", ko.t, p.kshape, p.dims.k_out);
        }
        const c10::cuda::OptionalCUDAGuard guard(p.call.device);
        const mdcn_status s = lib.rotary_forward(&p.attrs, &p.dims, p.call.code, qp, kp, p.pos, p.freq, p.qw, p.kw, yp,
                                                 zp, p.call.stream(a[12]));
        return s == MDCN_OK ? pack({&qo, &ko}) : PyLong_FromLong(s);
    });
}

// (grad_q_out, grad_k_out, q, k, positions, inv_freq, sections, grad_q, grad_k, grad_q_weight, grad_k_weight,
//  workspace, grow, layout, norm, q_weight, k_weight, eps, stream) -> (grad_q, grad_k, grad_q_weight, grad_k_weight);
// grow: allocate what is None, and a workspace that is too small
PyObject* rotary_backward(PyObject*, PyObject* const* a, Py_ssize_t n) {
    return guarded(n, 19, [&]() -> PyObject* {
        const at::Tensor& gy = tensor("grad_q_out", a[0]);
        const at::Tensor* gz = maybe("grad_k_out", a[1]);
        Rotary p(gy, gz, a[4], a[5], a[6], a[13], a[14], a[15], a[16], a[17]);
        const bool grow = truth(a[12]), norm = p.attrs.norm != 0;
        if (norm && (a[2] == Py_None || (a[3] == Py_None) != (gz == nullptr))) refuse("with norm, q and k are needed");
        if (!grow) {
            if ((a[8] == Py_None) != (gz == nullptr)) refuse("grad_k is given exactly when grad_k_out is");
            if ((a[9] == Py_None) != (a[15] == Py_None) || (a[10] == Py_None) != (a[16] == Py_None))
                refuse("a weight's gradient is given exactly when the weight is");
        }
        void* const yp = p.call.view("grad_q_out", gy, p.qshape, p.dims.q_out);
        const Output gq = output("grad_q", a[7], p.call, p.qshape);
        Output gk{at::Tensor(), nullptr}, gqw{at::Tensor(), nullptr}, gkw{at::Tensor(), nullptr};
        void* const gp = p.call.view("grad_q", gq.t, p.qshape, p.dims.q_grad);
        void *zp = nullptr, *hp = nullptr, *qp = nullptr, *kp = nullptr;
        if (norm) qp = p.call.view("q", tensor("q", a[2]), p.qshape, p.dims.q);
        if (gz) {
            zp = p.call.view("grad_k_out", *gz, p.kshape, p.dims.k_out);
            gk = output("grad_k", a[8], p.call, p.kshape);
            hp = p.call.view("grad_k", gk.t, p.kshape, p.dims.k_grad);
            if (norm) kp = p.call.view("k", tensor("k", a[3]), p.kshape, p.dims.k);
        }
        const Shape one = p.qshape.slice(2, 1);
        auto weight = [&](const char* name, PyObject* o, const void* w, Output& out) -> void* {
            if (!w) return nullptr;
            if (o != Py_None) {
                out = {tensor(name, o), o};
                return p.call.flat(name, o, p.call.type, one);
            }
            out.t = p.call.make(one, p.call.type);
            return out.t.data_ptr();
        };
        void* const wq = weight("grad_q_weight", a[9], p.qw, gqw);
        void* const wk = weight("grad_k_weight", a[10], p.kw, gkw);
        size_t need = 0, bytes = 0;
        if (grow && (wq || wk)) {
            const mdcn_status s = lib.rotary_backward_size(&p.attrs, &p.dims, p.call.code, &need);
            if (s != MDCN_OK) return PyLong_FromLong(s);
        }
        at::Tensor keep;
        void* const ws = p.call.workspace(a[11], need, keep, bytes, grow);
        const c10::cuda::OptionalCUDAGuard guard(p.call.device);
        const mdcn_status s =
            lib.rotary_backward(&p.attrs, &p.dims, p.call.code, yp, zp, qp, kp, p.pos, p.freq, p.qw, p.kw, gp, hp, wq,
                                wk, ws, bytes, p.call.stream(a[18]));
        return s == MDCN_OK ? pack({&gq, &gk, &gqw, &gkw}) : PyLong_FromLong(s);
    });
}

// (grad_q_out, grad_k_out, positions, inv_freq, sections, layout, norm, eps) -> (status, bytes)
PyObject* rotary_backward_size(PyObject*, PyObject* const* a, Py_ssize_t n) {
    return guarded(n, 8, [&]() -> PyObject* {
        const at::Tensor& gy = tensor("grad_q_out", a[0]);
        Rotary p(gy, maybe("grad_k_out", a[1]), a[2], a[3], a[4], a[5], a[6], Py_None, Py_None, a[7]);
        mdcn_strides* all[] = {&p.dims.q, &p.dims.k, &p.dims.q_out, &p.dims.k_out, &p.dims.q_grad, &p.dims.k_grad};
        for (mdcn_strides* s : all) s->token = s->head = 1;  // sizes do not depend on the strides
        size_t bytes = 0;
        const mdcn_status s = lib.rotary_backward_size(&p.attrs, &p.dims, p.call.code, &bytes);
        return Py_BuildValue("iK", static_cast<int>(s), static_cast<unsigned long long>(bytes));
    });
}

// ---------------------------------------------------------------- attention
struct Attention {
    Call call;
    mdcn_attention_attrs attrs{};
    mdcn_attention_dims dims{};
    void *q, *k, *v, *q_starts, *k_starts, *k_lengths;
    Shape qshape, kshape;

    // a: q, k, v, q_starts, k_starts, k_lengths, causal, scale
    explicit Attention(PyObject* const* a) : call("q", tensor("q", a[0])) {
        const at::Tensor &tq = tensor("q", a[0]), &tk = tensor("k", a[1]), &tv = tensor("v", a[2]);
        qshape = tq.sizes();
        kshape = tk.sizes();
        if (kshape.size() != 3 || kshape[2] != qshape[2])
            refuse("k must be [tokens, heads, head_dim] with the head_dim of q");
        q = call.view("q", tq, qshape, dims.q);
        k = call.view("k", tk, kshape, dims.k);
        v = call.view("v", tv, kshape, dims.v);
        const at::Tensor& starts = tensor("q_starts", a[3]);
        tensor("k_starts", a[4]);
        if (starts.dim() != 1 || starts.size(0) < 1) refuse("q_starts must be [sequences + 1]");
        dims.batch = starts.size(0) - 1;
        q_starts = call.flat("q_starts", a[3], at::kInt, {dims.batch + 1});
        k_starts = call.flat("k_starts", a[4], at::kInt, {dims.batch + 1});
        k_lengths = call.flat("k_lengths", a[5], at::kInt, {dims.batch});
        dims.q_tokens = qshape[0];
        dims.q_heads = qshape[1];
        dims.head_dim = qshape[2];
        dims.k_tokens = kshape[0];
        dims.k_heads = kshape[1];
        attrs.causal = truth(a[6]) ? 1 : 0;
        attrs.scale = static_cast<float>(a[7] == Py_None ? 1.0 / std::sqrt(static_cast<double>(dims.head_dim))
                                                         : number(a[7]));
    }
    float* lse(PyObject* o) const { return static_cast<float*>(call.flat("lse", o, at::kFloat, {qshape[1], qshape[0]})); }
};

// (q, k, v, q_starts, k_starts, k_lengths, causal, scale, out, lse, workspace, grow, stream) -> (out, lse)
PyObject* attention_forward(PyObject*, PyObject* const* a, Py_ssize_t n) {
    return guarded(n, 13, [&]() -> PyObject* {
        Attention p(a);
        const bool grow = truth(a[11]);
        const Output out = output("out", a[8], p.call, p.qshape);
        void* const op = p.call.view("out", out.t, p.qshape, p.dims.out);
        Output lse{at::Tensor(), a[9] == Py_None ? nullptr : a[9]};
        void* lp;
        if (a[9] == Py_None) {
            lse.t = p.call.make({p.qshape[1], p.qshape[0]}, at::kFloat);
            lp = lse.t.data_ptr();
        } else {
            lp = p.lse(a[9]);
        }
        size_t need = 0, bytes = 0;
        if (grow) {
            const mdcn_status s = lib.attention_size(&p.attrs, &p.dims, p.call.code, &need);
            if (s != MDCN_OK) return PyLong_FromLong(s);
        }
        at::Tensor keep;
        void* const ws = p.call.workspace(a[10], need, keep, bytes, grow);
        const c10::cuda::OptionalCUDAGuard guard(p.call.device);
        const mdcn_status s = lib.attention_forward(&p.attrs, &p.dims, p.call.code, p.q, p.k, p.v, p.q_starts,
                                                    p.k_starts, p.k_lengths, op, lp, ws, bytes, p.call.stream(a[12]));
        return s == MDCN_OK ? pack({&out, &lse}) : PyLong_FromLong(s);
    });
}

// (q, k, v, q_starts, k_starts, k_lengths, causal, scale, out) -> (status, bytes)
PyObject* attention_size(PyObject*, PyObject* const* a, Py_ssize_t n) {
    return guarded(n, 9, [&]() -> PyObject* {
        Attention p(a);
        p.call.view("out", tensor("out", a[8]), p.qshape, p.dims.out);
        size_t bytes = 0;
        const mdcn_status s = lib.attention_size(&p.attrs, &p.dims, p.call.code, &bytes);
        return Py_BuildValue("iK", static_cast<int>(s), static_cast<unsigned long long>(bytes));
    });
}

struct Gradients {
    Output q, k, v;
    void *g, *out, *gq, *gk, *gv;
    // a: grad_out, out, grad_q, grad_k, grad_v
    Gradients(Attention& p, PyObject* const* a)
        : q(output("grad_q", a[2], p.call, p.qshape)),
          k(output("grad_k", a[3], p.call, p.kshape)),
          v(output("grad_v", a[4], p.call, p.kshape)) {
        g = p.call.view("grad_out", tensor("grad_out", a[0]), p.qshape, p.dims.grad_out);
        out = p.call.view("out", tensor("out", a[1]), p.qshape, p.dims.out);
        gq = p.call.view("grad_q", q.t, p.qshape, p.dims.grad_q);
        gk = p.call.view("grad_k", k.t, p.kshape, p.dims.grad_k);
        gv = p.call.view("grad_v", v.t, p.kshape, p.dims.grad_v);
    }
};

// (q, k, v, q_starts, k_starts, k_lengths, causal, scale, grad_out, out, grad_q, grad_k, grad_v, lse, workspace, grow,
//  stream) -> (grad_q, grad_k, grad_v)
PyObject* attention_backward(PyObject*, PyObject* const* a, Py_ssize_t n) {
    return guarded(n, 17, [&]() -> PyObject* {
        Attention p(a);
        const Gradients g(p, a + 8);
        const bool grow = truth(a[15]);
        tensor("lse", a[13]);
        const float* lse = p.lse(a[13]);
        size_t need = 0, bytes = 0;
        if (grow) {
            const mdcn_status s = lib.attention_backward_size(&p.attrs, &p.dims, p.call.code, &need);
            if (s != MDCN_OK) return PyLong_FromLong(s);
        }
        at::Tensor keep;
        void* const ws = p.call.workspace(a[14], need, keep, bytes, grow);
        const c10::cuda::OptionalCUDAGuard guard(p.call.device);
        const mdcn_status s =
            lib.attention_backward(&p.attrs, &p.dims, p.call.code, g.g, p.q, p.k, p.v, g.out, lse, p.q_starts,
                                   p.k_starts, p.k_lengths, g.gq, g.gk, g.gv, ws, bytes, p.call.stream(a[16]));
        return s == MDCN_OK ? pack({&g.q, &g.k, &g.v}) : PyLong_FromLong(s);
    });
}

// (q, k, v, q_starts, k_starts, k_lengths, causal, scale, grad_out, out, grad_q, grad_k, grad_v) -> (status, bytes)
PyObject* attention_backward_size(PyObject*, PyObject* const* a, Py_ssize_t n) {
    return guarded(n, 13, [&]() -> PyObject* {
        Attention p(a);
        const Gradients g(p, a + 8);
        size_t bytes = 0;
        const mdcn_status s = lib.attention_backward_size(&p.attrs, &p.dims, p.call.code, &bytes);
        return Py_BuildValue("iK", static_cast<int>(s), static_cast<unsigned long long>(bytes));
    });
}

// The addresses of the seven library functions, in Library's order.
PyObject* bind(PyObject*, PyObject* const* a, Py_ssize_t n) {
    return guarded(n, 7, [&]() -> PyObject* {
        void* p[7];
        for (int i = 0; i < 7; ++i) {
            p[i] = PyLong_AsVoidPtr(a[i]);
            if (!p[i]) throw Raised{};
        }
        lib.rotary_forward = reinterpret_cast<decltype(lib.rotary_forward)>(p[0]);
        lib.rotary_backward = reinterpret_cast<decltype(lib.rotary_backward)>(p[1]);
        lib.rotary_backward_size = reinterpret_cast<decltype(lib.rotary_backward_size)>(p[2]);
        lib.attention_forward = reinterpret_cast<decltype(lib.attention_forward)>(p[3]);
        lib.attention_size = reinterpret_cast<decltype(lib.attention_size)>(p[4]);
        lib.attention_backward = reinterpret_cast<decltype(lib.attention_backward)>(p[5]);
        lib.attention_backward_size = reinterpret_cast<decltype(lib.attention_backward_size)>(p[6]);
        Py_RETURN_NONE;
    });
}

#define METHOD(f) {#f, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(f)), METH_FASTCALL, nullptr}
PyMethodDef methods[] = {METHOD(bind),
                         METHOD(rotary_forward),
                         METHOD(rotary_backward),
                         METHOD(rotary_backward_size),
                         METHOD(attention_forward),
                         METHOD(attention_size),
                         METHOD(attention_backward),
                         METHOD(attention_backward_size),
                         {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_token_binding", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__token_binding(void) { return PyModule_Create(&module); }
