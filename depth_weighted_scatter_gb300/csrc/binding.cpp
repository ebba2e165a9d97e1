// binding.cpp -- the tensor-level helpers of the token operators
// (attention.py) as a native Python module: checks of types and shapes,
// allocation of outputs and workspaces with PyTorch, the current stream, and
// the call of the C entry point (include/bevpool.h).  A decoding step makes
// these calls for every layer with microseconds of work each, which the same
// code in Python does not keep up with.
#define PY_SSIZE_T_CLEAN
#include <Python.h>

#include <ATen/core/Tensor.h>
#include <ATen/core/grad_mode.h>
#include <ATen/ops/empty.h>
#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include <cmath>
#include <string>

#include "../../include/bevpool.h"

namespace {

PyObject *g_error = nullptr;               // BevpoolError(status, what)

struct Refusal {
    int status;
    std::string what;
};

[[noreturn]] void refuse(const std::string &what, int status = BEVPOOL_ERR_INVALID_ARG) { throw Refusal{status, what}; }

// Positional arguments of a call.
class Args {
public:
    Args(PyObject *const *a, Py_ssize_t n, Py_ssize_t want) : a_(a) {
        if (n != want) refuse("wrong number of arguments");
    }
    PyObject *next() { return a_[i_++]; }
    at::Tensor tensor(const char *name) {
        PyObject *o = next();
        if (!THPVariable_Check(o)) refuse(std::string(name) + ": a tensor is wanted");
        return plain(name, THPVariable_Unpack(o));
    }
    at::Tensor maybe(const char *name) {   // None: undefined
        PyObject *o = next();
        if (o == Py_None) return at::Tensor();
        if (!THPVariable_Check(o)) refuse(std::string(name) + ": a tensor or None is wanted");
        return plain(name, THPVariable_Unpack(o));
    }
    int32_t i32(const char *name) {
        const long long v = PyLong_AsLongLong(next());
        if (v == -1 && PyErr_Occurred()) throw python_error();
        if (v < INT32_MIN || v > INT32_MAX) refuse(std::string(name) + ": out of 32-bit range");
        return static_cast<int32_t>(v);
    }
    float f32() {
        const double v = PyFloat_AsDouble(next());
        if (v == -1.0 && PyErr_Occurred()) throw python_error();
        return static_cast<float>(v);
    }
    bool flag() {
        const int v = PyObject_IsTrue(next());
        if (v < 0) throw python_error();
        return v != 0;
    }

private:
    // The helpers record no gradients, so a tensor that would lose its own is refused.
    const at::Tensor &plain(const char *name, const at::Tensor &t) const {
        if ((grad_ && t.requires_grad()) || t._fw_grad(0).defined())
            refuse(std::string(name) + ": gradients are not recorded through this call; make it under torch.no_grad() or on "
                                       "detached tensors (qk_norm_rope_backward computes those of qk_norm_rope)");
        return t;
    }

    const bool grad_ = at::GradMode::is_enabled();
    PyObject *const *a_;
    Py_ssize_t i_ = 0;
};

// The tensor that the others are checked against.
struct Like {
    int64_t T, H, D;
    at::ScalarType type;
    bevpool_dtype code;
    c10::Device device;
    void *stream;
};

Like like(const char *name, const at::Tensor &t) {
    if (t.dim() != 3) refuse(std::string(name) + ": a [tokens, heads, head_dim] tensor is wanted");
    const auto type = t.scalar_type();
    if (type != at::kHalf && type != at::kBFloat16) refuse(std::string(name) + ": fp16 or bf16 is wanted", BEVPOOL_ERR_UNSUPPORTED);
    if (!t.is_cuda() || t.device().index() != c10::cuda::current_device())
        refuse(std::string(name) + ": tensors must be on the current CUDA device");
    if (t.size(0) > INT32_MAX || t.size(1) > INT32_MAX || t.size(2) > INT32_MAX) refuse(std::string(name) + ": too large");
    return {t.size(0), t.size(1), t.size(2), type, type == at::kHalf ? BEVPOOL_F16 : BEVPOOL_BF16, t.device(),
            c10::cuda::getCurrentCUDAStream(t.device().index()).stream()};
}

struct Rows {
    void *p;
    int64_t ts, hs;
};

// A [tokens, heads, head_dim] tensor of the same tokens, head_dim, type and
// device; heads < 0: any number.
Rows rows(const char *name, const at::Tensor &t, const Like &l, int64_t heads) {
    if (t.dim() != 3 || t.size(0) != l.T || t.size(2) != l.D || (heads >= 0 && t.size(1) != heads) ||
        t.scalar_type() != l.type || t.device() != l.device)
        refuse(std::string(name) + ": tokens, heads, head_dim, type or device does not match");
    if (t.stride(2) != 1) refuse(std::string(name) + ": the last axis must be contiguous");
    if (t.size(1) > INT32_MAX) refuse(std::string(name) + ": too many heads");
    // the stride of an axis of one entry is never used
    return {t.data_ptr(), t.size(0) > 1 ? t.stride(0) : 0, t.size(1) > 1 ? t.stride(1) : 0};
}

void *vector(const char *name, const at::Tensor &t, int64_t n, at::ScalarType type, const c10::Device &device) {
    if (!t.defined()) return nullptr;
    if (t.scalar_type() != type || t.device() != device || t.numel() != n || !t.is_contiguous())
        refuse(std::string(name) + ": a contiguous " + c10::toString(type) + " tensor of " + std::to_string(n) +
               " entries on the same device is wanted");
    return t.data_ptr();
}

at::Tensor fresh(at::IntArrayRef sizes, at::ScalarType type, const c10::Device &device) {
    return at::empty(sizes, at::TensorOptions().dtype(type).device(device));
}

// A caller's workspace (undefined: none): the kernels write all of its bytes, so
// it has to own them, where they run.
void workspace_ok(const at::Tensor &ws) {
    if (!ws.defined()) return;
    if (!ws.is_contiguous()) refuse("workspace: a contiguous tensor is wanted");
    if (!ws.is_cuda() || ws.device().index() != c10::cuda::current_device())
        refuse("workspace: a tensor on the current CUDA device is wanted");
}

struct Positions {
    const int32_t *p;
    int32_t axes, sections[4], rotary_dim, interleaved;
    const float *inv_freq;
};

// positions, inv_freq, sections (None or a sequence), interleaved
Positions positions(Args &a, const Like &l) {
    Positions r;
    const at::Tensor p = a.tensor("positions"), f = a.tensor("inv_freq");
    PyObject *sec = a.next();
    r.interleaved = a.flag();
    const int64_t axes = p.dim() == 2 ? p.size(1) : 1;
    if (p.dim() < 1 || p.dim() > 2 || p.size(0) != l.T || axes < 1 || axes > 4)
        refuse("positions: int32 [tokens] or [tokens, axes <= 4] is wanted");
    if (f.numel() > 1 << 20) refuse("inv_freq: too long");
    r.axes = static_cast<int32_t>(axes);
    r.rotary_dim = static_cast<int32_t>(2 * f.numel());
    r.p = static_cast<const int32_t *>(vector("positions", p, l.T * axes, at::kInt, l.device));
    r.inv_freq = static_cast<const float *>(vector("inv_freq", f, f.numel(), at::kFloat, l.device));
    if (sec == Py_None) {
        if (axes != 1) refuse("sections: one entry an axis is wanted");
        r.sections[0] = r.rotary_dim / 2;
    } else {
        PyObject *s = PySequence_Fast(sec, "sections: a sequence is wanted");
        if (!s) throw python_error();
        const bool fits = PySequence_Fast_GET_SIZE(s) == axes;
        for (int i = 0; fits && i < axes; ++i) {
            const long long v = PyLong_AsLongLong(PySequence_Fast_GET_ITEM(s, i));
            r.sections[i] = v < -1 || v > INT32_MAX ? -1 : static_cast<int32_t>(v);
        }
        Py_DECREF(s);
        if (PyErr_Occurred()) throw python_error();
        if (!fits) refuse("sections: one entry an axis is wanted");
    }
    return r;
}

struct Cache {
    bevpool_dtype code;
    void *k, *v;
    int64_t ps, ss, hs;
    int32_t n_pages, heads, page, table_pages, n_seqs;
    const int32_t *table, *kv_len, *cu_q;
};

// k_cache, v_cache, block_table, kv_len, cu_q
Cache cache(Args &a, const Like &l, int64_t heads) {
    const at::Tensor k = a.tensor("k_cache"), v = a.tensor("v_cache"), t = a.tensor("block_table"), n = a.tensor("kv_len"),
                     cu = a.tensor("cu_q");
    bool alike = k.dim() == 4 && k.sizes() == v.sizes() && k.scalar_type() == v.scalar_type();
    for (int64_t i = 0; alike && i < 4; ++i) alike = k.size(i) == 1 || k.stride(i) == v.stride(i);
    if (!alike)
        refuse("caches: two [n_pages, n_k_heads, page_size, head_dim] tensors of one type and layout are wanted");
    Cache c;
    switch (k.scalar_type()) {
        case at::kHalf: c.code = BEVPOOL_F16; break;
        case at::kBFloat16: c.code = BEVPOOL_BF16; break;
        case at::kFloat8_e4m3fn:
        case at::kByte: c.code = BEVPOOL_E4M3; break;
        default: refuse("caches: fp16, bf16 or E4M3 codes are wanted", BEVPOOL_ERR_UNSUPPORTED);
    }
    if ((heads >= 0 && k.size(1) != heads) || k.size(3) != l.D || k.device() != l.device || v.device() != l.device)
        refuse("caches: heads, head_dim or device does not match");
    if (k.stride(3) != 1) refuse("caches: the last axis must be contiguous");
    if (t.dim() != 2) refuse("block_table: [n_seqs, pages] is wanted");
    for (const int64_t x : {k.size(0), k.size(1), k.size(2), t.size(0), t.size(1)})
        if (x > INT32_MAX) refuse("caches: too large");
    c.k = k.data_ptr();
    c.v = v.data_ptr();
    c.n_pages = static_cast<int32_t>(k.size(0));
    c.heads = static_cast<int32_t>(k.size(1));
    c.page = static_cast<int32_t>(k.size(2));
    c.ps = c.n_pages > 1 ? k.stride(0) : 0;
    c.hs = c.heads > 1 ? k.stride(1) : 0;
    c.ss = k.stride(2);
    c.n_seqs = static_cast<int32_t>(t.size(0));
    c.table_pages = static_cast<int32_t>(t.size(1));
    c.table = static_cast<const int32_t *>(vector("block_table", t, t.size(0) * t.size(1), at::kInt, l.device));
    c.kv_len = static_cast<const int32_t *>(vector("kv_len", n, t.size(0), at::kInt, l.device));
    c.cu_q = static_cast<const int32_t *>(vector("cu_q", cu, t.size(0) + 1, at::kInt, l.device));
    return c;
}

void done(bevpool_status st, const char *what) {
    if (st != BEVPOOL_OK) refuse(what, st);
}

const float *weight(const char *name, const at::Tensor &w, const Like &l) {
    return static_cast<const float *>(vector(name, w, l.D, at::kFloat, l.device));
}

// q, k, q_weight, k_weight, q_out, k_out, eps, positions..
PyObject *qk_norm_rope(Args a) {
    const at::Tensor q = a.tensor("q"), k = a.tensor("k"), qw = a.maybe("q_weight"), kw = a.maybe("k_weight");
    at::Tensor qo = a.maybe("q_out"), ko = a.maybe("k_out");
    const float eps = a.f32();
    const Like l = like("q", q);
    const Rows qr = rows("q", q, l, l.H), kr = rows("k", k, l, -1);
    const Positions p = positions(a, l);
    const float *w0 = weight("q_weight", qw, l), *w1 = weight("k_weight", kw, l);
    if (!qo.defined()) qo = fresh(q.sizes(), l.type, l.device);
    if (!ko.defined()) ko = fresh(k.sizes(), l.type, l.device);
    const Rows qor = rows("q_out", qo, l, l.H), kor = rows("k_out", ko, l, k.size(1));
    done(bevpool_qk_norm_rope(l.code, qr.p, qr.ts, qr.hs, kr.p, kr.ts, kr.hs, l.T, l.H, k.size(1), l.D, w0, w1, eps, p.p, p.axes,
                              p.sections, p.rotary_dim, p.inv_freq, p.interleaved, qor.p, qor.ts, qor.hs, kor.p, kor.ts,
                              kor.hs, l.stream),
         "bevpool_qk_norm_rope");
    return Py_BuildValue("NN", THPVariable_Wrap(qo), THPVariable_Wrap(ko));
}

// dq_out, dk_out, q, k, q_weight, k_weight, dq, dk, workspace, eps, positions..
PyObject *qk_norm_rope_backward(Args a) {
    const at::Tensor gq = a.tensor("dq_out"), gk = a.tensor("dk_out"), q = a.tensor("q"), k = a.tensor("k"),
                     qw = a.maybe("q_weight"), kw = a.maybe("k_weight");
    at::Tensor dq = a.maybe("dq"), dk = a.maybe("dk"), ws = a.maybe("workspace"), dqw, dkw;
    workspace_ok(ws);
    const float eps = a.f32();
    const Like l = like("q", q);
    const Rows qr = rows("q", q, l, l.H), kr = rows("k", k, l, -1);
    const Rows gqr = rows("dq_out", gq, l, l.H), gkr = rows("dk_out", gk, l, k.size(1));
    const Positions p = positions(a, l);
    const float *w0 = weight("q_weight", qw, l), *w1 = weight("k_weight", kw, l);
    if (!dq.defined()) dq = fresh(q.sizes(), l.type, l.device);
    if (!dk.defined()) dk = fresh(k.sizes(), l.type, l.device);
    const Rows dqr = rows("dq", dq, l, l.H), dkr = rows("dk", dk, l, k.size(1));
    if (w0) dqw = fresh({l.D}, at::kFloat, l.device);
    if (w1) dkw = fresh({l.D}, at::kFloat, l.device);
    if (!ws.defined() && (w0 || w1)) {
        const size_t n = bevpool_qk_norm_rope_backward_workspace_size(l.T, l.H, k.size(1), l.D);
        ws = fresh({static_cast<int64_t>(n ? n : 1)}, at::kByte, l.device);
    }
    done(bevpool_qk_norm_rope_backward(
             l.code, gqr.p, gqr.ts, gqr.hs, gkr.p, gkr.ts, gkr.hs, qr.p, qr.ts, qr.hs, kr.p, kr.ts, kr.hs, l.T, l.H, k.size(1),
             l.D, w0, w1, eps, p.p, p.axes, p.sections, p.rotary_dim, p.inv_freq, p.interleaved, dqr.p, dqr.ts, dqr.hs, dkr.p,
             dkr.ts, dkr.hs, w0 ? static_cast<float *>(dqw.data_ptr()) : nullptr,
             w1 ? static_cast<float *>(dkw.data_ptr()) : nullptr, ws.defined() ? ws.data_ptr() : nullptr,
             ws.defined() ? ws.nbytes() : 0, l.stream),
         "bevpool_qk_norm_rope_backward");
    return Py_BuildValue("NNNN", THPVariable_Wrap(dq), THPVariable_Wrap(dk), THPVariable_Wrap(dqw), THPVariable_Wrap(dkw));
}

// k, v, q, k_weight, q_weight, q_out, k_scale, v_scale, k_cache.. , eps, positions..
PyObject *kv_append(Args a) {
    const at::Tensor k = a.tensor("k"), v = a.tensor("v"), q = a.maybe("q"), kw = a.maybe("k_weight"), qw = a.maybe("q_weight");
    at::Tensor qo = a.maybe("q_out");
    const float ks = a.f32(), vs = a.f32();
    const Like l = like("k", k);
    const Rows kr = rows("k", k, l, l.H), vr = rows("v", v, l, l.H);
    const Cache c = cache(a, l, l.H);
    const float eps = a.f32();
    const Positions p = positions(a, l);
    const float *w0 = weight("q_weight", qw, l), *w1 = weight("k_weight", kw, l);
    Rows qr = {nullptr, 0, 0}, qor = {nullptr, 0, 0};
    int64_t Hq = 0;
    if (q.defined()) {
        qr = rows("q", q, l, -1);
        Hq = q.size(1);
        if (!qo.defined()) qo = fresh(q.sizes(), l.type, l.device);
        qor = rows("q_out", qo, l, Hq);
    } else if (qo.defined()) {
        refuse("q_out without q");
    }
    done(bevpool_kv_append(l.code, c.code, kr.p, kr.ts, kr.hs, vr.p, vr.ts, vr.hs, qr.p, qr.ts, qr.hs, l.T, Hq, l.H, l.D, w0, w1,
                           eps, p.p, p.axes, p.sections, p.rotary_dim, p.inv_freq, p.interleaved, qor.p, qor.ts, qor.hs, c.k,
                           c.v, c.ps, c.ss, c.hs, c.n_pages, c.page, c.table, c.table_pages, c.kv_len, c.cu_q, c.n_seqs, ks,
                           vs, l.stream),
         "bevpool_kv_append");
    return THPVariable_Wrap(qo);
}

// A cache's scales of pages and heads.
float *scales_of(const char *name, const at::Tensor &t, const Cache &c, const Like &l) {
    if (c.code != BEVPOOL_E4M3) refuse("caches: E4M3 codes are wanted", BEVPOOL_ERR_UNSUPPORTED);
    if (t.dim() != 2 || t.size(0) != c.n_pages || t.size(1) != c.heads) refuse(std::string(name) + ": [n_pages, n_k_heads] is wanted");
    return static_cast<float *>(vector(name, t, static_cast<int64_t>(c.n_pages) * c.heads, at::kFloat, l.device));
}

// k, v, q, k_weight, q_weight, q_out, k_scales, v_scales, k_cache.. , eps, positions..
PyObject *kv_append_scaled(Args a) {
    const at::Tensor k = a.tensor("k"), v = a.tensor("v"), q = a.maybe("q"), kw = a.maybe("k_weight"), qw = a.maybe("q_weight");
    at::Tensor qo = a.maybe("q_out");
    const at::Tensor kt = a.tensor("k_scales"), vt = a.tensor("v_scales");
    const Like l = like("k", k);
    const Rows kr = rows("k", k, l, l.H), vr = rows("v", v, l, l.H);
    const Cache c = cache(a, l, l.H);
    const float eps = a.f32();
    const Positions p = positions(a, l);
    const float *w0 = weight("q_weight", qw, l), *w1 = weight("k_weight", kw, l);
    float *ks = scales_of("k_scales", kt, c, l), *vs = scales_of("v_scales", vt, c, l);
    Rows qr = {nullptr, 0, 0}, qor = {nullptr, 0, 0};
    int64_t Hq = 0;
    if (q.defined()) {
        qr = rows("q", q, l, -1);
        Hq = q.size(1);
        if (!qo.defined()) qo = fresh(q.sizes(), l.type, l.device);
        qor = rows("q_out", qo, l, Hq);
    } else if (qo.defined()) {
        refuse("q_out without q");
    }
    done(bevpool_kv_append_scaled(l.code, kr.p, kr.ts, kr.hs, vr.p, vr.ts, vr.hs, qr.p, qr.ts, qr.hs, l.T, Hq, l.H, l.D, w0, w1, eps,
                                  p.p, p.axes, p.sections, p.rotary_dim, p.inv_freq, p.interleaved, qor.p, qor.ts, qor.hs, c.k, c.v,
                                  c.ps, c.ss, c.hs, ks, vs, c.n_pages, c.page, c.table, c.table_pages, c.kv_len, c.cu_q, c.n_seqs,
                                  l.stream),
         "bevpool_kv_append_scaled");
    return THPVariable_Wrap(qo);
}

// q, workspace, (scaled: k_scales, v_scales,) k_cache.., max_q_len, max_kv_len, scale (None: head_dim ** -0.5), causal, window,
// (not scaled: k_scale, v_scale,) out, lse?
template <bool SCALED>
PyObject *attend(Args a) {
    const at::Tensor q = a.tensor("q");
    at::Tensor ws = a.maybe("workspace");
    workspace_ok(ws);
    at::Tensor kt, vt;
    if (SCALED) {
        kt = a.tensor("k_scales");
        vt = a.tensor("v_scales");
    }
    const Like l = like("q", q);
    const Rows qr = rows("q", q, l, l.H);
    const Cache c = cache(a, l, -1);
    const float *kp = nullptr, *vp = nullptr;
    if (SCALED) {
        kp = scales_of("k_scales", kt, c, l);
        vp = scales_of("v_scales", vt, c, l);
    }
    const int32_t max_q = a.i32("max_q_len"), max_kv = a.i32("max_kv_len");
    PyObject *so = a.next();
    float scale = 1.0f / std::sqrt(static_cast<float>(l.D));
    if (so != Py_None) {
        scale = static_cast<float>(PyFloat_AsDouble(so));
        if (PyErr_Occurred()) throw python_error();
    }
    const bool causal = a.flag();
    const int32_t window = a.i32("window");
    float ks = 1.0f, vs = 1.0f;
    if (!SCALED) {
        ks = a.f32();
        vs = a.f32();
    }
    at::Tensor out = a.maybe("out"), lse;
    const bool want_lse = a.flag();
    if (!out.defined()) out = fresh(q.sizes(), l.type, l.device);
    const Rows o = rows("out", out, l, l.H);
    if (want_lse) lse = fresh({l.T, l.H}, at::kFloat, l.device);
    if (!ws.defined()) {
        const auto size = SCALED ? bevpool_paged_attention_scaled_workspace_size : bevpool_paged_attention_workspace_size;
        const size_t n = size(c.n_seqs, l.T, l.H, c.heads, l.D, max_q, max_kv, window);
        if (n) ws = fresh({static_cast<int64_t>(n)}, at::kByte, l.device);
    }
    float *lp = want_lse ? static_cast<float *>(lse.data_ptr()) : nullptr;
    void *wp = ws.defined() ? ws.data_ptr() : nullptr;
    const size_t wn = ws.defined() ? ws.nbytes() : 0;
    if (SCALED)
        done(bevpool_paged_attention_scaled(l.code, qr.p, qr.ts, qr.hs, c.k, c.v, c.ps, c.ss, c.hs, kp, vp, c.n_pages, c.page, c.table,
                                            c.table_pages, c.kv_len, c.cu_q, c.n_seqs, l.T, l.H, c.heads, l.D, max_q, max_kv, scale,
                                            causal, window, o.p, o.ts, o.hs, lp, wp, wn, l.stream),
             "bevpool_paged_attention_scaled");
    else
        done(bevpool_paged_attention(l.code, c.code, qr.p, qr.ts, qr.hs, c.k, c.v, c.ps, c.ss, c.hs, c.n_pages, c.page, c.table,
                                     c.table_pages, c.kv_len, c.cu_q, c.n_seqs, l.T, l.H, c.heads, l.D, max_q, max_kv, scale, causal,
                                     window, ks, vs, o.p, o.ts, o.hs, lp, wp, wn, l.stream),
             "bevpool_paged_attention");
    if (!want_lse) return THPVariable_Wrap(out);
    return Py_BuildValue("NN", THPVariable_Wrap(out), THPVariable_Wrap(lse));
}

// Byte ranges of a call's tensors.
struct Span {
    const char *from, *to;
    Span(const at::Tensor &t) : from(static_cast<const char *>(t.data_ptr())), to(from + t.nbytes()) {}
    bool meets(const Span &o) const { return from < o.to && o.from < to; }
};

// A contiguous tensor on the bytes of `all` from `at` on.
at::Tensor part_of(const at::Tensor &all, int64_t at, at::IntArrayRef sizes, at::ScalarType type) {
    at::Tensor t = at::detail::make_tensor<c10::TensorImpl>(c10::Storage(all.storage()), all.key_set(), c10::scalarTypeToTypeMeta(type));
    t.unsafeGetTensorImpl()->set_sizes_contiguous(sizes);
    t.unsafeGetTensorImpl()->set_storage_offset(at / static_cast<int64_t>(c10::elementSize(type)));
    return t;
}

// q_len, kv_len, first, drop, block_table, free_pages, n_free, page_size, n_tokens, out (None or its nine tensors)
PyObject *plan_pages(Args a) {
    const at::Tensor q = a.tensor("q_len"), kv = a.tensor("kv_len"), first = a.tensor("first"), drop = a.maybe("drop"),
                     table = a.tensor("block_table"), pool = a.tensor("free_pages"), n_free = a.tensor("n_free");
    const int32_t page = a.i32("page_size"), n_tokens = a.i32("n_tokens");
    PyObject *given = a.next();
    if (table.dim() != 2) refuse("block_table: [n_seqs, pages] is wanted");
    if (!table.is_cuda() || table.device().index() != c10::cuda::current_device())
        refuse("block_table: tensors must be on the current CUDA device");
    if (n_tokens < 0) refuse("n_tokens: a count is wanted");
    const int64_t B = table.size(0), W = table.size(1), P = pool.numel();
    if (B > INT32_MAX || W > INT32_MAX || P > INT32_MAX) refuse("block_table, free_pages: too large");
    const c10::Device device = table.device();
    const auto ints = [&](const char *name, const at::Tensor &t, int64_t n) {
        return static_cast<const int32_t *>(vector(name, t, n, at::kInt, device));
    };
    const int32_t *in[] = {ints("q_len", q, B),           ints("kv_len", kv, B), ints("first", first, B), ints("drop", drop, B),
                           ints("block_table", table, B * W), ints("free_pages", pool, P), ints("n_free", n_free, 1)};
    // outputs, in the order of the result
    constexpr int N = 9, SLOTS = 2;
    static const char *const names[N] = {"cu_q", "positions", "slots", "kv_len", "first", "block_table", "free_pages", "n_free", "missing"};
    const int64_t sizes[N] = {B + 1, n_tokens, n_tokens, B, B, B * W, P, 1, 1};
    at::Tensor out[N];
    void *p[N];
    if (given == Py_None) {
        // One allocation for all of them: nine take longer than the plan of a small batch.
        int64_t at[N], bytes = 0;
        for (int i = 0; i < N; ++i) {
            at[i] = bytes;
            bytes += (sizes[i] * (i == SLOTS ? 8 : 4) + 255) / 256 * 256;
        }
        const at::Tensor all = fresh({bytes}, at::kByte, device);
        for (int i = 0; i < N; ++i) {
            out[i] = i == 5 ? part_of(all, at[i], {B, W}, at::kInt) : part_of(all, at[i], {sizes[i]}, i == SLOTS ? at::kLong : at::kInt);
            p[i] = static_cast<char *>(all.data_ptr()) + at[i];
        }
    } else {
        PyObject *seq = PySequence_Fast(given, "out: the tensors of a plan are wanted");
        if (!seq) throw python_error();
        const bool fits = PySequence_Fast_GET_SIZE(seq) == N;
        for (int i = 0; fits && i < N; ++i) {
            PyObject *o = PySequence_Fast_GET_ITEM(seq, i);
            if (THPVariable_Check(o)) out[i] = THPVariable_Unpack(o);
        }
        Py_DECREF(seq);
        for (int i = 0; i < N; ++i) {
            if (!out[i].defined()) refuse("out: the nine tensors of a plan are wanted");
            p[i] = vector(names[i], out[i], sizes[i], i == SLOTS ? at::kLong : at::kInt, device);
            const Span x(out[i]);
            for (int j = 0; j < i; ++j)
                if (x.meets(out[j])) refuse(std::string("out: ") + names[i] + " and " + names[j] + " overlap");
            for (const at::Tensor &t : {q, kv, first, drop, table, pool, n_free})
                if (t.defined() && x.meets(t)) refuse(std::string("out: ") + names[i] + " overlaps an input");
        }
        if (out[5].sizes() != table.sizes()) refuse("out: block_table has another shape");
    }
    const auto i32 = [&](int i) { return static_cast<int32_t *>(p[i]); };
    done(bevpool_plan_pages(in[0], in[1], in[2], in[3], in[4], in[5], in[6], static_cast<int32_t>(B), static_cast<int32_t>(W),
                            static_cast<int32_t>(P), n_tokens, page, i32(0), i32(1), static_cast<int64_t *>(p[2]), i32(3),
                            i32(4), i32(5), i32(6), i32(7), i32(8), c10::cuda::getCurrentCUDAStream(device.index()).stream()),
         "bevpool_plan_pages");
    PyObject *res = PyTuple_New(N);
    if (!res) throw python_error();
    for (int i = 0; i < N; ++i) PyTuple_SET_ITEM(res, i, THPVariable_Wrap(out[i]));
    return res;
}

// A method of the module: C++ exceptions become Python's.
template <PyObject *(*Fn)(Args), int N>
PyObject *method(PyObject *, PyObject *const *args, Py_ssize_t n) {
    HANDLE_TH_ERRORS
    try {
        return Fn(Args(args, n, N));
    } catch (const Refusal &r) {
        PyObject *e = PyObject_CallFunction(g_error, "is", r.status, r.what.c_str());
        if (e) {
            PyErr_SetObject(g_error, e);
            Py_DECREF(e);
        }
        return nullptr;
    }
    END_HANDLE_TH_ERRORS
}

PyObject *set_error(PyObject *, PyObject *cls) {
    Py_INCREF(cls);
    Py_XDECREF(g_error);
    g_error = cls;
    Py_RETURN_NONE;
}

template <PyObject *(*Fn)(Args), int N>
PyMethodDef entry(const char *name) {
    return {name, reinterpret_cast<PyCFunction>(reinterpret_cast<void *>(&method<Fn, N>)), METH_FASTCALL, nullptr};
}

PyMethodDef g_methods[] = {entry<qk_norm_rope, 11>("qk_norm_rope"),
                           entry<qk_norm_rope_backward, 14>("qk_norm_rope_backward"),
                           entry<kv_append, 18>("kv_append"),
                           entry<kv_append_scaled, 18>("kv_append_scaled"),
                           entry<attend<false>, 16>("paged_attention"),
                           entry<attend<true>, 16>("paged_attention_scaled"),
                           entry<plan_pages, 10>("plan_pages"),
                           {"set_error", set_error, METH_O, nullptr},
                           {nullptr, nullptr, 0, nullptr}};

PyModuleDef g_module = {PyModuleDef_HEAD_INIT, "_token_ops", nullptr, -1, g_methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__token_ops(void) { return PyModule_Create(&g_module); }
