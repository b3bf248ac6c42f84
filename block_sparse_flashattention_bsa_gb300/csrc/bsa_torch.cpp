// bsa_torch.cpp -- compiled marshalling of the projection and paged-cache
// calls (rope.py, paged.py): checks torch tensors, takes outputs and
// workspaces from torch's allocator, fills the C ABI's structs and calls
// libbsa.so on the tensors' device and its current stream.  The same steps in
// Python took longer than the kernels of a small call.  Calls in a row on the
// same tensors: appending one token 27 us (12 now, of which the views of a fused
// projection are 4.5; with new inputs from call to call 17), one decoding step
// 17 (9, the GPU's own time), gradients of 8K packed tokens 45 (29, the same).
// No arithmetic, no state.
//
// Every function takes its arguments by position and returns its result, or
// the bsa_status as an int where the library refused; what a check here
// refuses is a ValueError.

#define PY_SSIZE_T_CLEAN
#include <Python.h>

#include <ATen/ATen.h>
#include <ATen/cuda/EmptyTensor.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/autograd/python_variable.h>

#include <cmath>
#include <string>

#include "bsa.h"

namespace {

struct Refused : std::exception {
    std::string what_;
    explicit Refused(std::string s) : what_(std::move(s)) {}
    const char* what() const noexcept override { return what_.c_str(); }
};
struct PyFailed {};  // a Python exception is set

void want(bool ok, const char* message) {
    if (!ok) throw Refused(message);
}

// ------------------------------------------------------------ arguments
using T = const at::Tensor*;

T tensor_or_none(PyObject* o, const char* name) {
    if (o == Py_None) return nullptr;
    if (!THPVariable_Check(o)) throw Refused(std::string(name) + ": expected a tensor");
    return &THPVariable_Unpack(o);
}
T tensor(PyObject* o, const char* name) {
    T t = tensor_or_none(o, name);
    if (!t) throw Refused(std::string(name) + ": expected a tensor");
    return t;
}
int32_t int_arg(PyObject* o, const char* name) {
    const long long v = PyLong_AsLongLong(o);
    if (v == -1 && PyErr_Occurred()) throw PyFailed();
    if (v < INT32_MIN || v > INT32_MAX) throw Refused(std::string(name) + ": out of range");
    return (int32_t)v;
}
float float_arg(PyObject* o) {
    const double v = PyFloat_AsDouble(o);
    if (v == -1.0 && PyErr_Occurred()) throw PyFailed();
    return (float)v;
}
bool bool_arg(PyObject* o) {
    const int v = PyObject_IsTrue(o);
    if (v < 0) throw PyFailed();
    return v != 0;
}

// ------------------------------------------------------------ checks
int32_t size32(int64_t n) {
    want(n <= INT32_MAX, "a dimension is too large");
    return (int32_t)n;
}

// All given tensors on the first one's CUDA device.
c10::Device same_device(T first, std::initializer_list<T> rest) {
    want(first->is_cuda(), "expected CUDA tensors");
    for (T t : rest)
        if (t && t->device() != first->device())
            throw Refused("tensors on different devices: " + first->device().str() + " and " + t->device().str());
    return first->device();
}

bool shape_is(const at::Tensor& t, at::IntArrayRef s) { return t.sizes() == s; }

void ints(T t, at::IntArrayRef shape, const char* name, at::ScalarType type = at::kInt) {
    if (t->scalar_type() != type || !shape_is(*t, shape) || !t->is_contiguous())
        throw Refused(std::string(name) + ": contiguous " + (type == at::kInt ? "int32" : type == at::kLong ? "int64" : "float32") +
                      " of the documented shape");
}

template <typename P>
P* data(T t) {
    return t ? static_cast<P*>(t->data_ptr()) : nullptr;
}

// (batch, token, head) strides in elements of a token-major bf16 tensor
// ([tokens, heads, D]: batch 0).  An extent of one has no stride worth checking.
void row_strides(T t, int64_t* out, const char* name) {
    if (t->scalar_type() != at::kBFloat16) throw Refused(std::string(name) + ": expected bf16");
    const int nd = (int)t->dim();
    if (t->stride(nd - 1) != 1) throw Refused(std::string(name) + ": head rows must be contiguous");
    out[0] = 0;
    for (int i = 0; i < nd - 1; ++i) out[i + 4 - nd] = t->size(i) > 1 ? t->stride(i) : 0;
}

at::Tensor new_tensor(at::IntArrayRef shape, at::ScalarType type, c10::Device dev) {
    // past the dispatcher: a projection call with its three outputs 7.3 -> 5.1 us
    return at::Tensor(at::detail::empty_cuda(shape, type, dev, std::nullopt));
}

// The given output, checked, or a new one.
at::Tensor output(T given, at::IntArrayRef shape, c10::Device dev) {
    if (!given) return new_tensor(shape, at::kBFloat16, dev);
    want(given->scalar_type() == at::kBFloat16 && shape_is(*given, shape) && given->is_contiguous() &&
             given->device() == dev,
         "out: a contiguous bf16 tensor of the result's shape on the inputs' device");
    return *given;
}

bsa_stream_t current_stream(c10::Device dev) {
    return reinterpret_cast<bsa_stream_t>(c10::cuda::getCurrentCUDAStream(dev.index()).stream());
}

// ------------------------------------------------------------ results
PyObject* wrap(const at::Tensor& t) {
    if (!t.defined()) Py_RETURN_NONE;
    return THPVariable_Wrap(t);
}
PyObject* wrap_all(std::initializer_list<at::Tensor> ts) {
    PyObject* r = PyTuple_New((Py_ssize_t)ts.size());
    if (!r) throw PyFailed();
    Py_ssize_t i = 0;
    for (const at::Tensor& t : ts) {
        PyObject* o = wrap(t);
        if (!o) {
            Py_DECREF(r);
            throw PyFailed();
        }
        PyTuple_SET_ITEM(r, i++, o);
    }
    return r;
}
PyObject* status(int st) { return PyLong_FromLong(st); }

// Calls f with the argument count checked and C++ exceptions turned into Python's.
template <typename F>
PyObject* guarded(Py_ssize_t n, Py_ssize_t expected, F f) {
    if (n != expected) {
        PyErr_Format(PyExc_TypeError, "expected %zd arguments, got %zd", expected, n);
        return nullptr;
    }
    try {
        return f();
    } catch (const PyFailed&) {
    } catch (const Refused& e) {
        PyErr_SetString(PyExc_ValueError, e.what());
    } catch (const c10::OutOfMemoryError& e) {
        // what torch's own functions raise
        PyObject* torch = PyImport_ImportModule("torch");
        PyObject* cls = torch ? PyObject_GetAttrString(torch, "OutOfMemoryError") : nullptr;
        if (cls) PyErr_SetString(cls, e.what_without_backtrace());
        Py_XDECREF(cls);
        Py_XDECREF(torch);
    } catch (const c10::Error& e) {
        PyErr_SetString(PyExc_RuntimeError, e.what_without_backtrace());
    } catch (const std::exception& e) {
        PyErr_SetString(PyExc_RuntimeError, e.what());
    }
    return nullptr;
}

// ------------------------------------------------------------ projection
// q, k, v, inv_freq, positions, q_weight, k_weight, eps, gain, interleaved, kv_repeat
struct Side {
    bsa_norm_rope_args a{};
    c10::Device dev{c10::kCPU};
    T q, k, v;
    int64_t B, N, Hq, Hkv, D;
};

Side side(PyObject* const* o, bool batched) {
    Side s;
    s.q = tensor(o[0], "q");
    s.k = tensor(o[1], "k");
    s.v = tensor_or_none(o[2], "v");
    T inv = tensor_or_none(o[3], "inv_freq"), pos = tensor_or_none(o[4], "positions");
    T qw = tensor_or_none(o[5], "q_weight"), kw = tensor_or_none(o[6], "k_weight");
    const int nd = batched ? 4 : 3;
    bool ok = s.q->dim() == nd && s.k->dim() == nd && (!s.v || s.v->sizes() == s.k->sizes());
    for (int i = 0; ok && i < nd; ++i) ok = i == nd - 2 || s.q->size(i) == s.k->size(i);
    want(ok, "expected q, k, v with one shape up to their number of heads (k, v alike)");
    s.dev = same_device(s.q, {s.k, s.v, inv, pos, qw, kw});
    s.B = batched ? s.q->size(0) : 1;
    s.N = s.q->size(nd - 3);
    s.Hq = s.q->size(nd - 2);
    s.Hkv = s.k->size(nd - 2);
    s.D = s.q->size(nd - 1);
    bsa_norm_rope_args& a = s.a;
    a.B = size32(s.B);
    a.N = size32(s.N);
    a.Hq = size32(s.Hq);
    a.Hkv = size32(s.Hkv);
    a.D = size32(s.D);
    if (inv) {
        want(inv->scalar_type() == at::kDouble && inv->dim() == 1 && inv->is_contiguous(),
             "inv_freq: contiguous float64 [rotary_dim / 2] (rope_inv_freq)");
        a.rotary_dim = size32(2 * inv->numel());
        a.inv_freq = data<double>(inv);
    }
    if (pos) {
        const bool flat = pos->dim() == 1 && pos->size(0) == s.N;
        const bool two = batched && pos->dim() == 2 && pos->size(0) == s.B && pos->size(1) == s.N;
        want(pos->scalar_type() == at::kInt && (flat || two) && (s.N <= 1 || pos->stride(-1) == 1),
             "positions: int32 [N] or [B, N], one per token");
        a.positions = data<int32_t>(pos);
        a.position_stride = two && s.B > 1 ? pos->stride(0) : 0;
    }
    for (T w : {qw, kw})
        want(!w || (w->scalar_type() == at::kFloat && w->dim() == 1 && w->size(0) == s.D && w->is_contiguous()),
             "norm weights: contiguous float32 [D]");
    a.q_weight = data<float>(qw);
    a.k_weight = data<float>(kw);
    a.eps = float_arg(o[7]);
    a.gain = float_arg(o[8]);
    a.interleaved = bool_arg(o[9]);
    a.kv_repeat = int_arg(o[10], "kv_repeat");
    a.q = s.q->data_ptr();
    a.k = s.k->data_ptr();
    a.v = data<void>(s.v);
    row_strides(s.q, a.q_stride, "q");
    row_strides(s.k, a.k_stride, "k");
    if (s.v) row_strides(s.v, a.v_stride, "v");
    return s;
}

// side arguments (11), out q, out k, out v
PyObject* qk_norm_rope(PyObject*, PyObject* const* o, Py_ssize_t n) {
    return guarded(n, 14, [&]() -> PyObject* {
        Side s = side(o, true);
        want(s.v || o[13] == Py_None, "out: no v to write");
        const c10::cuda::CUDAGuard guard(s.dev);
        if (s.a.kv_repeat < 1) return status(BSA_ERR_INVALID_ARG);
        const int64_t hq[4] = {s.B, s.Hq, s.N, s.D}, hk[4] = {s.B, s.Hkv * s.a.kv_repeat, s.N, s.D};
        at::Tensor q = output(tensor_or_none(o[11], "out"), hq, s.dev), k = output(tensor_or_none(o[12], "out"), hk, s.dev), v;
        if (s.v) v = output(tensor_or_none(o[13], "out"), hk, s.dev);
        const int st = bsa_qk_norm_rope(&s.a, q.data_ptr(), k.data_ptr(), s.v ? v.data_ptr() : nullptr, current_stream(s.dev));
        return st ? status(st) : wrap_all({q, k, v});
    });
}

// side arguments (11, v None), dq, dk, dv, out or None, out q, out k, out v
PyObject* qk_norm_rope_backward(PyObject*, PyObject* const* o, Py_ssize_t n) {
    return guarded(n, 18, [&]() -> PyObject* {
        Side s = side(o, true);
        T dq = tensor(o[11], "dq"), dk = tensor(o[12], "dk"), dv = tensor_or_none(o[13], "dv");
        same_device(s.q, {dq, dk, dv});
        if (s.a.kv_repeat < 1) return status(BSA_ERR_INVALID_ARG);
        const int64_t hq[4] = {s.B, s.Hq, s.N, s.D}, hk[4] = {s.B, s.Hkv * s.a.kv_repeat, s.N, s.D};
        const T dz[3] = {dq, dk, dv};
        for (int i = 0; i < 3; ++i)
            want(!dz[i] || (shape_is(*dz[i], i ? hk : hq) && dz[i]->scalar_type() == at::kBFloat16 && dz[i]->is_contiguous()),
                 "dq, dk, dv: contiguous bf16 tensors of the forward's output shapes");
        const c10::cuda::CUDAGuard guard(s.dev);
        const int64_t tq[4] = {s.B, s.N, s.Hq, s.D}, tk[4] = {s.B, s.N, s.Hkv, s.D};
        at::Tensor g[3];
        bsa_norm_rope_grads b{};
        int64_t* st3[3] = {b.q_stride, b.k_stride, b.v_stride};
        for (int i = 0; i < 3; ++i) {
            if (i == 2 && !dv) {
                want(o[17] == Py_None, "out: no v gradient to write");
                continue;
            }
            const at::IntArrayRef shape = i ? tk : tq;
            if (o[14] == Py_None) {
                g[i] = new_tensor(shape, at::kBFloat16, s.dev);
            } else {
                g[i] = *tensor(o[15 + i], "out");
                want(g[i].device() == s.dev && shape_is(g[i], shape), "out: token-major tensors of the inputs' shapes");
            }
            row_strides(&g[i], st3[i], "out");
        }
        at::Tensor qw, kw, ws;
        if (s.a.q_weight) qw = new_tensor({s.D}, at::kFloat, s.dev);
        if (s.a.k_weight) kw = new_tensor({s.D}, at::kFloat, s.dev);
        const int64_t bytes = qw.defined() || kw.defined() ? bsa_qk_norm_rope_backward_workspace(s.a.D) : 0;
        if (bytes) ws = new_tensor({bytes}, at::kByte, s.dev);
        b.dq = dq->data_ptr();
        b.dk = dk->data_ptr();
        b.dv = data<void>(dv);
        b.q = g[0].data_ptr();
        b.k = g[1].data_ptr();
        b.v = dv ? g[2].data_ptr() : nullptr;
        b.q_weight = qw.defined() ? qw.data_ptr<float>() : nullptr;
        b.k_weight = kw.defined() ? kw.data_ptr<float>() : nullptr;
        const int st = bsa_qk_norm_rope_backward(&s.a, &b, bytes ? ws.data_ptr() : nullptr, bytes, current_stream(s.dev));
        return st ? status(st) : wrap_all({g[0], g[1], g[2], qw, kw});
    });
}

// ------------------------------------------------------------ paged cache
// The scales of 8-bit pools (`given` false: bf16 pools).
struct Scales {
    bsa_page_scales s{};
    bool given = false;
    const bsa_page_scales* ptr() const { return given ? &s : nullptr; }
};

bsa_page_cache pool(T kc, T vc, T table, bool layers, T ks, T vs, Scales* scales) {
    const int64_t nd = kc->dim();
    want(kc->sizes() == vc->sizes() && (nd == 4 || (layers && nd == 5)),
         layers ? "expected k_cache and v_cache of one shape [n_pages, Hkv, page, D] or [layers, n_pages, Hkv, page, D]"
                : "expected k_cache and v_cache of one shape [n_pages, Hkv, page, D]");
    want((ks != nullptr) == (vs != nullptr), "k_scale and v_scale come together");
    scales->given = ks != nullptr;
    if (scales->given) {
        auto codes = [](T t) { return t->scalar_type() == at::kFloat8_e4m3fn || t->scalar_type() == at::kByte; };
        auto exps = [&](T t) {
            return (t->scalar_type() == at::kFloat8_e8m0fnu || t->scalar_type() == at::kByte) && t->is_contiguous() &&
                   t->sizes() == kc->sizes().slice(0, nd - 1);
        };
        want(codes(kc) && codes(vc) && kc->is_contiguous() && vc->is_contiguous(),
             "caches with scales: contiguous float8_e4m3fn (or uint8 codes)");
        want(exps(ks) && exps(vs), "k_scale, v_scale: contiguous float8_e8m0fnu (or uint8) of the caches' shape without D");
        scales->s.k = ks->data_ptr();
        scales->s.v = vs->data_ptr();
    } else {
        want(kc->scalar_type() == at::kBFloat16 && vc->scalar_type() == at::kBFloat16 && kc->is_contiguous() &&
                 vc->is_contiguous(),
             "expected contiguous bf16 caches");
    }
    want(table->scalar_type() == at::kInt && table->dim() == 2 && table->is_contiguous(),
         "page_table: contiguous int32 [n_seqs, max_pages]");
    bsa_page_cache c{};
    c.k = kc->data_ptr();
    c.v = vc->data_ptr();
    c.layers = nd == 5 ? size32(kc->size(0)) : 1;
    c.n_pages = size32(kc->size(nd - 4));
    c.Hkv = size32(kc->size(nd - 3));
    c.page = size32(kc->size(nd - 2));
    c.D = size32(kc->size(nd - 1));
    c.page_table = data<int32_t>(table);
    c.n_seqs = size32(table->size(0));
    c.max_pages = size32(table->size(1));
    return c;
}

// side arguments (11), k_cache, v_cache, page_table, seq_ids, slots, out, k_scale, v_scale
PyObject* cache_append(PyObject*, PyObject* const* o, Py_ssize_t n) {
    return guarded(n, 19, [&]() -> PyObject* {
        Side s = side(o, false);
        T kc = tensor(o[11], "k_cache"), vc = tensor(o[12], "v_cache"), table = tensor(o[13], "page_table");
        T seq = tensor(o[14], "seq_ids"), slot = tensor(o[15], "slots");
        T ks = tensor_or_none(o[17], "k_scale"), vs = tensor_or_none(o[18], "v_scale");
        Scales sc;
        const bsa_page_cache c = pool(kc, vc, table, false, ks, vs, &sc);
        same_device(s.q, {kc, vc, table, seq, slot, ks, vs});
        want(s.v && c.Hkv == s.Hkv && c.D == s.D, "k and v need the cache's heads and head size");
        ints(seq, {s.N}, "seq_ids");
        ints(slot, {s.N}, "slots");
        const c10::cuda::CUDAGuard guard(s.dev);
        const int64_t shape[3] = {s.N, s.Hq, s.D};
        at::Tensor q = output(tensor_or_none(o[16], "out"), shape, s.dev);
        const bsa_stream_t on = current_stream(s.dev);
        const int st = sc.given ? bsa_cache_append_fp8(&s.a, &c, &sc.s, data<int32_t>(seq), data<int32_t>(slot), q.data_ptr(), on)
                                : bsa_cache_append(&s.a, &c, data<int32_t>(seq), data<int32_t>(slot), q.data_ptr(), on);
        return st ? status(st) : wrap(q);
    });
}

// q, k_cache, v_cache, page_table, context_len, draft_len, tree_mask, row_ptr, col_idx, scale or None, out, lse
PyObject* tree_attention(PyObject*, PyObject* const* o, Py_ssize_t n) {
    return guarded(n, 12, [&]() -> PyObject* {
        T q = tensor(o[0], "q"), kc = tensor(o[1], "k_cache"), vc = tensor(o[2], "v_cache"), table = tensor(o[3], "page_table");
        T ctx = tensor(o[4], "context_len"), dl = tensor_or_none(o[5], "draft_len"), mask = tensor_or_none(o[6], "tree_mask");
        T rp = tensor_or_none(o[7], "row_ptr"), ci = tensor_or_none(o[8], "col_idx");
        T out = tensor_or_none(o[10], "out"), lse = tensor_or_none(o[11], "lse");
        want(q->dim() == 4 && q->scalar_type() == at::kBFloat16 && q->is_contiguous(), "q: contiguous bf16 [B, T, Hq, D]");
        const int64_t B = q->size(0), Tn = q->size(1), Hq = q->size(2), D = q->size(3);
        Scales sc;
        const bsa_page_cache c = pool(kc, vc, table, false, nullptr, nullptr, &sc);
        const c10::Device dev = same_device(q, {kc, vc, table, ctx, dl, mask, rp, ci, out, lse});
        want(c.n_seqs == B && c.D == D, "page_table needs one row per sequence, the caches q's head size");
        ints(ctx, {B}, "context_len");
        if (dl) ints(dl, {B}, "draft_len");
        if (mask) ints(mask, {B, Tn}, "tree_mask", at::kLong);
        want((rp != nullptr) == (ci != nullptr), "row_ptr and col_idx come together");
        bsa_tree_args a{};
        a.B = size32(B);
        a.T = size32(Tn);
        a.Hq = size32(Hq);
        if (rp) {
            ints(rp, {B * c.Hkv + 1}, "row_ptr");
            ints(ci, {ci->numel()}, "col_idx");
            a.row_ptr = data<int32_t>(rp);
            // an empty list has no storage: any address does, nothing below its capacity of 0 is read
            a.col_idx = ci->numel() ? data<int32_t>(ci) : a.row_ptr;
            a.col_capacity = ci->numel();
        }
        a.scale = o[9] == Py_None ? (float)(1.0 / std::sqrt((double)std::max<int64_t>(D, 1))) : float_arg(o[9]);
        const c10::cuda::CUDAGuard guard(dev);
        at::Tensor r = output(out, q->sizes(), dev), l;
        if (lse) {
            ints(lse, {B, Tn, Hq}, "lse", at::kFloat);
            l = *lse;
        } else {
            l = new_tensor({B, Tn, Hq}, at::kFloat, dev);
        }
        const int64_t bytes = bsa_tree_attention_workspace(a.B, a.T, a.Hq, c.Hkv, a.B > 0 ? c.D : 0);
        at::Tensor ws = new_tensor({bytes}, at::kByte, dev);
        a.q = q->data_ptr();
        a.context_len = data<int32_t>(ctx);
        a.draft_len = data<int32_t>(dl);
        a.tree_mask = data<uint64_t>(mask);
        a.out = r.data_ptr();
        a.lse = l.data_ptr<float>();
        const int st = bsa_tree_attention(&a, &c, ws.data_ptr(), bytes, current_stream(dev));
        return st ? status(st) : wrap_all({r, l});
    });
}

// k_cache, v_cache, page_table, context_len, accepted, n_accepted, new_len, k_scale, v_scale
PyObject* cache_accept(PyObject*, PyObject* const* o, Py_ssize_t n) {
    return guarded(n, 9, [&]() -> PyObject* {
        T kc = tensor(o[0], "k_cache"), vc = tensor(o[1], "v_cache"), table = tensor(o[2], "page_table");
        T ctx = tensor(o[3], "context_len"), acc = tensor(o[4], "accepted"), na = tensor(o[5], "n_accepted");
        T given = tensor_or_none(o[6], "new_len"), ks = tensor_or_none(o[7], "k_scale"), vs = tensor_or_none(o[8], "v_scale");
        Scales sc;
        const bsa_page_cache c = pool(kc, vc, table, true, ks, vs, &sc);
        const c10::Device dev = same_device(kc, {vc, table, ctx, acc, na, given, ks, vs});
        want(acc->dim() == 2, "accepted: int32 [n_seqs, T]");
        const int64_t S = c.n_seqs, Tn = acc->size(1);
        ints(ctx, {S}, "context_len");
        ints(acc, {S, Tn}, "accepted");
        ints(na, {S}, "n_accepted");
        if (given) ints(given, {S}, "new_len");
        const c10::cuda::CUDAGuard guard(dev);
        at::Tensor r = given ? *given : new_tensor({S}, at::kInt, dev);
        const int32_t *x = data<int32_t>(ctx), *y = data<int32_t>(acc), *z = data<int32_t>(na), t = size32(Tn);
        const bsa_stream_t on = current_stream(dev);
        const int st = sc.given ? bsa_cache_accept_fp8(&c, &sc.s, x, y, z, t, r.data_ptr<int32_t>(), on)
                                : bsa_cache_accept(&c, x, y, z, t, r.data_ptr<int32_t>(), on);
        return st ? status(st) : wrap(r);
    });
}

// fork (True or False), page_table, page_ref, three request vectors (in the C call's order), k_cache, v_cache,
// k_scale, v_scale
PyObject* cache_request(PyObject*, PyObject* const* o, Py_ssize_t n) {
    return guarded(n, 10, [&]() -> PyObject* {
        const bool fork = bool_arg(o[0]);
        T table = tensor(o[1], "page_table"), ref = tensor(o[2], "page_ref"), kc = tensor(o[6], "k_cache"), vc = tensor(o[7], "v_cache");
        T r[3] = {tensor(o[3], "requests"), tensor(o[4], "requests"), tensor(o[5], "requests")};
        T ks = tensor_or_none(o[8], "k_scale"), vs = tensor_or_none(o[9], "v_scale");
        Scales sc;
        const bsa_page_cache c = pool(kc, vc, table, true, ks, vs, &sc);
        const c10::Device dev = same_device(kc, {vc, table, ref, r[0], r[1], r[2], ks, vs});
        ints(ref, {c.n_pages}, "page_ref");
        const int64_t N = r[0]->numel();
        for (T t : r) ints(t, {N}, "requests");
        const c10::cuda::CUDAGuard guard(dev);
        at::Tensor granted = new_tensor({N}, at::kInt, dev);
        if (N == 0) return wrap(granted);
        const int64_t bytes = bsa_cache_pages_workspace(size32(N), c.n_seqs, c.n_pages);
        at::Tensor ws = new_tensor({bytes}, at::kByte, dev);
        const int32_t *x = data<int32_t>(r[0]), *y = data<int32_t>(r[1]), *z = data<int32_t>(r[2]);
        int32_t *rc = data<int32_t>(ref), *got = granted.data_ptr<int32_t>();
        const bsa_stream_t on = current_stream(dev);
        const int st =
            sc.given ? (fork ? bsa_cache_fork_fp8 : bsa_cache_resize_fp8)(&c, &sc.s, rc, (int32_t)N, x, y, z, got,
                                                                          ws.data_ptr(), bytes, on)
                     : (fork ? bsa_cache_fork : bsa_cache_resize)(&c, rc, (int32_t)N, x, y, z, got, ws.data_ptr(), bytes, on);
        return st ? status(st) : wrap(granted);
    });
}

// page_table, page_ref, k_cache, v_cache, k_scale, v_scale
PyObject* cache_compact(PyObject*, PyObject* const* o, Py_ssize_t n) {
    return guarded(n, 6, [&]() -> PyObject* {
        T table = tensor(o[0], "page_table"), ref = tensor(o[1], "page_ref"), kc = tensor(o[2], "k_cache"), vc = tensor(o[3], "v_cache");
        T ks = tensor_or_none(o[4], "k_scale"), vs = tensor_or_none(o[5], "v_scale");
        Scales sc;
        const bsa_page_cache c = pool(kc, vc, table, true, ks, vs, &sc);
        const c10::Device dev = same_device(kc, {vc, table, ref, ks, vs});
        ints(ref, {c.n_pages}, "page_ref");
        const c10::cuda::CUDAGuard guard(dev);
        at::Tensor r = new_tensor({c.n_pages}, at::kInt, dev);
        const int64_t bytes = bsa_cache_pages_workspace(0, c.n_seqs, c.n_pages);
        at::Tensor ws = new_tensor({bytes}, at::kByte, dev);
        int32_t *rc = data<int32_t>(ref), *to = r.data_ptr<int32_t>();
        const bsa_stream_t on = current_stream(dev);
        const int st = sc.given ? bsa_cache_compact_fp8(&c, &sc.s, rc, to, ws.data_ptr(), bytes, on)
                                : bsa_cache_compact(&c, rc, to, ws.data_ptr(), bytes, on);
        return st ? status(st) : wrap(r);
    });
}

// k_cache, v_cache, page_table, seq_ids, lens or None, n, first or None, kv_repeat, k_scale, v_scale, out k, out v
PyObject* cache_read(PyObject*, PyObject* const* o, Py_ssize_t n) {
    return guarded(n, 12, [&]() -> PyObject* {
        T kc = tensor(o[0], "k_cache"), vc = tensor(o[1], "v_cache"), table = tensor(o[2], "page_table");
        T seq = tensor(o[3], "seq_ids"), len = tensor_or_none(o[4], "lens"), first = tensor_or_none(o[6], "first");
        T ks = tensor_or_none(o[8], "k_scale"), vs = tensor_or_none(o[9], "v_scale");
        T ok = tensor_or_none(o[10], "out"), ov = tensor_or_none(o[11], "out");
        Scales sc;
        const bsa_page_cache c = pool(kc, vc, table, false, ks, vs, &sc);
        const c10::Device dev = same_device(kc, {vc, table, seq, len, first, ks, vs, ok, ov});
        bsa_read_args a{};
        const int64_t R = seq->numel();
        a.R = size32(R);
        a.n = int_arg(o[5], "n");
        a.kv_repeat = int_arg(o[7], "kv_repeat");
        ints(seq, {R}, "seq_ids");
        if (len) ints(len, {R}, "lens");
        if (first) ints(first, {R}, "first");
        if (a.n < 0 || a.kv_repeat < 1) return status(BSA_ERR_INVALID_ARG);
        want((ok != nullptr) == (ov != nullptr), "out: both tensors or none");
        const c10::cuda::CUDAGuard guard(dev);
        const int64_t shape[4] = {R, (int64_t)c.Hkv * a.kv_repeat, a.n, c.D};
        at::Tensor k = output(ok, shape, dev), v = output(ov, shape, dev);
        a.seq_ids = data<int32_t>(seq);
        a.len = data<int32_t>(len);
        a.first = data<int32_t>(first);
        a.k = k.data_ptr();
        a.v = v.data_ptr();
        const int st = bsa_cache_read(&a, &c, sc.ptr(), current_stream(dev));
        return st ? status(st) : wrap_all({k, v});
    });
}

// q, k_cache, v_cache, page_table, context_len, q_ptr or None, window, sinks, k_scale, v_scale, scale or None, out, lse, max_context
PyObject* chunk_attention(PyObject*, PyObject* const* o, Py_ssize_t n) {
    return guarded(n, 14, [&]() -> PyObject* {
        T q = tensor(o[0], "q"), kc = tensor(o[1], "k_cache"), vc = tensor(o[2], "v_cache"), table = tensor(o[3], "page_table");
        T ctx = tensor(o[4], "context_len"), qp = tensor_or_none(o[5], "q_ptr");
        T ks = tensor_or_none(o[8], "k_scale"), vs = tensor_or_none(o[9], "v_scale");
        T out = tensor_or_none(o[11], "out"), lse = tensor_or_none(o[12], "lse");
        want(q->dim() == 3 && q->scalar_type() == at::kBFloat16 && q->is_contiguous(), "q: contiguous bf16 [tokens, Hq, D]");
        const int64_t N = q->size(0), Hq = q->size(1), D = q->size(2);
        Scales sc;
        const bsa_page_cache c = pool(kc, vc, table, false, ks, vs, &sc);
        const c10::Device dev = same_device(q, {kc, vc, table, ctx, qp, ks, vs, out, lse});
        want(c.D == D, "the caches need q's head size");
        const int64_t B = c.n_seqs;
        ints(ctx, {B}, "context_len");
        if (qp) ints(qp, {B + 1}, "q_ptr");
        want(qp || N == B, "q_ptr: needed where the sequences do not bring one token each");
        bsa_chunk_args a{};
        a.B = size32(B);
        a.tokens = size32(N);
        a.Hq = size32(Hq);
        a.window = int_arg(o[6], "window");
        a.sinks = int_arg(o[7], "sinks");
        a.max_context = int_arg(o[13], "max_context");
        a.scale = o[10] == Py_None ? (float)(1.0 / std::sqrt((double)std::max<int64_t>(D, 1))) : float_arg(o[10]);
        const c10::cuda::CUDAGuard guard(dev);
        at::Tensor r = output(out, q->sizes(), dev), l;
        if (lse) {
            ints(lse, {N, Hq}, "lse", at::kFloat);
            l = *lse;
        } else {
            l = new_tensor({N, Hq}, at::kFloat, dev);
        }
        const int64_t bytes = bsa_chunk_attention_workspace(a.B, a.tokens, a.Hq, c.Hkv, c.D);
        at::Tensor ws = new_tensor({bytes}, at::kByte, dev);
        a.q = q->data_ptr();
        a.q_ptr = data<int32_t>(qp);
        a.context_len = data<int32_t>(ctx);
        a.out = r.data_ptr();
        a.lse = l.data_ptr<float>();
        const int st = bsa_chunk_attention(&a, &c, sc.ptr(), ws.data_ptr(), bytes, current_stream(dev));
        return st ? status(st) : wrap_all({r, l});
    });
}

#define CALL(name) {#name, (PyCFunction)(void (*)(void))name, METH_FASTCALL, nullptr}
PyMethodDef kMethods[] = {CALL(qk_norm_rope),  CALL(qk_norm_rope_backward), CALL(cache_append),
                          CALL(tree_attention), CALL(cache_accept),         CALL(cache_request),
                          CALL(cache_compact),  CALL(cache_read),           CALL(chunk_attention),
                          {nullptr, nullptr, 0, nullptr}};
PyModuleDef kModule = {PyModuleDef_HEAD_INIT, "_bsa_torch", "Compiled marshalling (see rope.py and paged.py).", -1,
                       kMethods,              nullptr,       nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__bsa_torch(void) { return PyModule_Create(&kModule); }
