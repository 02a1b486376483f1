// Python binding of the norm + rotation, 4-bit cache, shared-page and bounded-cache calls:
// checks the tensors and passes their addresses to the library's entry point,
// whose address each call is given.  A decode step makes these calls once for
// every layer, and their kernels run for a few microseconds: the checks take
// about 1 us here, and 8 us as Python code.
//
// A refusal is a ValueError, raised before the library is called; otherwise a
// function returns the library's status code.
#include <Python.h>

#include <ATen/core/Tensor.h>
#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/autograd/python_variable.h>

#include <initializer_list>
#include <sstream>
#include <string>

#include "xs_paged.h"

namespace {

constexpr int kPage = 16;

struct Refusal {
    std::string what;
};
struct PythonError {};  // the Python error is set

[[noreturn]] void refuse(const std::string &what) { throw Refusal{what}; }

std::string shape_of(const at::Tensor &t) {
    std::ostringstream s;
    s << t.scalar_type() << " " << t.sizes();
    return s.str();
}

// The arguments of one call, taken in order.
struct Args {
    PyObject *const *at;
    PyObject *const *end;
    PyObject *next() {
        if (at == end) refuse("too few arguments");
        return *at++;
    }
    void *entry() {
        void *p = PyLong_AsVoidPtr(next());
        if (PyErr_Occurred()) throw PythonError{};
        return p;
    }
    const at::Tensor &tensor(const char *name) {
        PyObject *o = next();
        if (!THPVariable_Check(o)) refuse(std::string(name) + " must be a tensor");
        return THPVariable_Unpack(o);
    }
    const at::Tensor *maybe(const char *name) {
        if (at != end && *at == Py_None) return ++at, nullptr;
        return &tensor(name);
    }
    double number() {
        const double v = PyFloat_AsDouble(next());
        if (PyErr_Occurred()) throw PythonError{};
        return v;
    }
    int integer(const char *name) {
        const long long v = PyLong_AsLongLong(next());
        if (PyErr_Occurred()) throw PythonError{};
        if (v != static_cast<int>(v)) refuse(std::string(name) + " is out of range");
        return static_cast<int>(v);
    }
    bool truth() {
        const int v = PyObject_IsTrue(next());
        if (v < 0) throw PythonError{};
        return v != 0;
    }
};

void want(const at::Tensor &t, at::ScalarType type, std::initializer_list<int64_t> sizes,
          const char *name) {
    if (t.scalar_type() == type && t.sizes() == at::IntArrayRef(sizes)) return;
    std::ostringstream s;
    s << name << " must be " << type << " " << at::IntArrayRef(sizes) << ", got " << shape_of(t);
    refuse(s.str());
}
void want(const at::Tensor *t, at::ScalarType type, std::initializer_list<int64_t> sizes,
          const char *name) {
    if (t) want(*t, type, sizes, name);
}
int as_int(int64_t v, const char *name) {
    if (v != static_cast<int>(v)) refuse(std::string(name) + " is too large");
    return static_cast<int>(v);
}
int dtype_code(const at::Tensor &t) {
    if (t.scalar_type() == at::kBFloat16) return XS_BF16;
    if (t.scalar_type() == at::kFloat) return XS_F32;
    refuse("unsupported dtype " + shape_of(t));
}
void *whole(const at::Tensor &t, const char *name) {
    if (!t.is_contiguous()) refuse(std::string(name) + " must be contiguous");
    return t.data_ptr();
}
void *whole(const at::Tensor *t, const char *name) { return t ? whole(*t, name) : nullptr; }

// Token stride of rows [T, H, D] whose heads lie next to one another.
int64_t rows(const at::Tensor &t, const char *name) {
    const auto z = t.sizes(), s = t.strides();
    if (s[2] != 1 || (s[1] != z[2] && z[1] != 1))
        refuse(std::string(name) + ": the heads of a token must be contiguous");
    return z[0] > 1 ? s[0] : z[1] * z[2];
}
void dims(const at::Tensor &t, int64_t n, const char *name) {
    if (t.dim() != n) {
        std::ostringstream s;
        s << name << " must have " << n << " dimensions, got " << shape_of(t);
        refuse(s.str());
    }
}

// All tensors (null: not given) on the current CUDA device, where the launch
// goes.  Its current stream, unless the caller names one.
cudaStream_t stream_for(PyObject *stream, std::initializer_list<const at::Tensor *> tensors) {
    const c10::Device dev = (*tensors.begin())->device();
    if (!dev.is_cuda()) refuse("tensors must be on a CUDA device");
    for (const at::Tensor *t : tensors)
        if (t && t->device() != dev) refuse("tensors are on different devices");
    if (dev.index() != c10::cuda::current_device())
        refuse("tensors are on " + dev.str() + ", which is not the current device");
    if (stream == Py_None) return c10::cuda::getCurrentCUDAStream(dev.index()).stream();
    void *s = PyLong_AsVoidPtr(stream);
    if (PyErr_Occurred()) throw PythonError{};
    return static_cast<cudaStream_t>(s);
}

// The blocks of a pair of pools for rows of q's type, [blocks, Hkv, 16, D], or
// of a pair of 4-bit pools, uint8 [blocks, Hkv, 9 D].
int64_t pools(const at::Tensor &k, const at::Tensor &v, at::ScalarType type, int64_t Hkv, int64_t D,
              bool *kv4) {
    if (k.scalar_type() != v.scalar_type() || k.sizes() != v.sizes())
        refuse("k_cache and v_cache differ in type or shape");
    *kv4 = k.scalar_type() == at::kByte;
    const int64_t n = k.dim() ? k.size(0) : 0;
    if (*kv4)
        want(k, at::kByte, {n, Hkv, 9 * D}, "a 4-bit pool");
    else
        want(k, type, {n, Hkv, kPage, D}, "a pool");
    return n;
}
int64_t kv4_pools(const at::Tensor &k, const at::Tensor &v, int64_t Hkv, int64_t D) {
    bool kv4 = false;
    if (k.scalar_type() != at::kByte) refuse("k_cache and v_cache must be 4-bit (uint8) pools");
    return pools(k, v, at::kByte, Hkv, D, &kv4);
}
int table_width(const at::Tensor &tables, const at::Tensor &lens, int64_t B) {
    if (tables.scalar_type() != at::kInt || tables.dim() != 2 || tables.size(0) != B)
        refuse("block_tables must be int32 [" + std::to_string(B) + ", max_blocks]");
    want(lens, at::kInt, {B}, "context_lens");
    return as_int(tables.size(1), "block_tables");
}

template <typename F> PyObject *status(F &&call) {
    int code;
    Py_BEGIN_ALLOW_THREADS;
    code = call();
    Py_END_ALLOW_THREADS;
    return PyLong_FromLong(code);
}

// ------------------------------------------------------------------ norm + rotation + append

enum Form { kPlain, kSlots, kPaged };

PyObject *norm_rope(Args a, Form form) {
    void *entry = a.entry();
    const at::Tensor &q_out = a.tensor("q_out");
    const at::Tensor *k_out = form == kPlain ? &a.tensor("k_out") : nullptr;
    const at::Tensor &q = a.tensor("q"), &k = a.tensor("k");
    const at::Tensor *v = form == kPlain ? nullptr : &a.tensor("v");
    const at::Tensor *qw = a.maybe("q_weight"), *kw = a.maybe("k_weight");
    const float eps = static_cast<float>(a.number());
    const at::Tensor *cos_sin = a.maybe("cos_sin");
    const at::Tensor *positions = form == kPaged ? nullptr : a.maybe("positions");
    const at::Tensor *kc = nullptr, *vc = nullptr, *where = nullptr, *lens = nullptr;
    if (form != kPlain) {
        kc = &a.tensor("k_cache"), vc = &a.tensor("v_cache");
        where = &a.tensor(form == kPaged ? "block_tables" : "slot_mapping");
        if (form == kPaged) lens = &a.tensor("context_lens");
    }
    int flags = a.truth() ? XS_ROPE_INTERLEAVED : 0;
    const at::Tensor *err = a.maybe("err_flag");
    PyObject *stream = a.next();

    dims(q, 3, "q"), dims(k, 3, "k");
    const auto type = q.scalar_type();
    const int64_t T = q.size(0), Hq = q.size(1), D = q.size(2), Hkv = k.size(1);
    want(q_out, type, {T, Hq, D}, "q_out");
    want(k, type, {T, Hkv, D}, "k");
    want(k_out, type, {T, Hkv, D}, "k_out");
    want(v, type, {T, Hkv, D}, "v");
    want(qw, type, {D}, "q_weight");
    want(kw, type, {D}, "k_weight");
    want(positions, at::kInt, {T}, "positions");
    want(err, at::kInt, {1}, "err_flag");
    int max_pos = 0, rot = 0;
    if (cos_sin) {
        if (cos_sin->scalar_type() != at::kFloat || cos_sin->dim() != 2)
            refuse("cos_sin must be float32 [max_pos, rotary_dim]");
        max_pos = as_int(cos_sin->size(0), "cos_sin"), rot = as_int(cos_sin->size(1), "cos_sin");
    }
    const int64_t q_stride = rows(q, "q"), k_stride = rows(k, "k"), v_stride = v ? rows(*v, "v") : 0;
    int64_t blocks = 0;
    int width = 0;
    if (form != kPlain) {
        bool kv4 = false;
        blocks = pools(*kc, *vc, type, Hkv, D, &kv4);
        if (kv4) flags |= XS_CACHE_KV4;
        if (form == kPaged)
            width = table_width(*where, *lens, T);
        else
            want(where, at::kLong, {T}, "slot_mapping");
    }
    const int code = dtype_code(q), t = as_int(T, "q"), hq = as_int(Hq, "q"), hkv = as_int(Hkv, "k"),
              d = as_int(D, "q");
    const cudaStream_t s = stream_for(stream, {&q, &k, v, &q_out, k_out, qw, kw, cos_sin, positions,
                                               kc, vc, where, lens, err});
    void *qo = whole(q_out, "q_out"), *ko = whole(k_out, "k_out");
    const void *w0 = whole(qw, "q_weight"), *w1 = whole(kw, "k_weight");
    const float *cs = static_cast<float *>(whole(cos_sin, "cos_sin"));
    const int32_t *pos = static_cast<int32_t *>(whole(positions, "positions"));
    int *flag = static_cast<int *>(whole(err, "err_flag"));
    if (T == 0) return PyLong_FromLong(XS_OK);
    const void *qp = q.data_ptr(), *kp = k.data_ptr();
    if (form == kPlain)
        return status([&] {
            return reinterpret_cast<decltype(&xs_qk_norm_rope)>(entry)(
                qo, ko, qp, q_stride, kp, k_stride, w0, w1, eps, cs, max_pos, rot, pos, t, hq, hkv, d,
                flags, code, flag, s);
        });
    const void *vp = v->data_ptr();
    void *kcp = whole(*kc, "k_cache"), *vcp = whole(*vc, "v_cache");
    const void *wp = whole(where, form == kPaged ? "block_tables" : "slot_mapping");
    if (form == kSlots)
        return status([&] {
            return reinterpret_cast<decltype(&xs_qk_norm_rope_append)>(entry)(
                qo, qp, q_stride, kp, k_stride, vp, v_stride, w0, w1, eps, cs, max_pos, rot, pos, kcp,
                vcp, static_cast<const int64_t *>(wp), t, hq, hkv, d, kPage, blocks, flags, code, flag,
                s);
        });
    const int32_t *lp = static_cast<int32_t *>(whole(lens, "context_lens"));
    return status([&] {
        return reinterpret_cast<decltype(&xs_qk_norm_rope_append_paged)>(entry)(
            qo, qp, q_stride, kp, k_stride, vp, v_stride, w0, w1, eps, cs, max_pos, rot, kcp, vcp,
            static_cast<const int32_t *>(wp), width, lp, t, hq, hkv, d, kPage, blocks, flags, code,
            flag, s);
    });
}

// ------------------------------------------------------------------ 4-bit cache

PyObject *kv4_append(Args a, bool paged) {
    void *entry = a.entry();
    const at::Tensor &k = a.tensor("k_new"), &v = a.tensor("v_new");
    const at::Tensor &kc = a.tensor("k_cache"), &vc = a.tensor("v_cache");
    const at::Tensor &where = a.tensor(paged ? "block_tables" : "slot_mapping");
    const at::Tensor *lens = paged ? &a.tensor("context_lens") : nullptr;
    const at::Tensor *err = a.maybe("err_flag");
    PyObject *stream = a.next();
    dims(k, 3, "k_new");
    const int64_t T = k.size(0), Hkv = k.size(1), D = k.size(2);
    want(v, k.scalar_type(), {T, Hkv, D}, "v_new");
    const int64_t blocks = kv4_pools(kc, vc, Hkv, D);
    int width = 0;
    if (paged)
        width = table_width(where, *lens, T);
    else
        want(where, at::kLong, {T}, "slot_mapping");
    want(err, at::kInt, {1}, "err_flag");
    const int64_t k_stride = rows(k, "k_new"), v_stride = rows(v, "v_new");
    const int code = dtype_code(k), t = as_int(T, "k_new"), hkv = as_int(Hkv, "k_new"),
              d = as_int(D, "k_new");
    const cudaStream_t s = stream_for(stream, {&k, &v, &kc, &vc, &where, lens, err});
    void *kcp = whole(kc, "k_cache"), *vcp = whole(vc, "v_cache");
    const void *wp = whole(where, paged ? "block_tables" : "slot_mapping");
    const int32_t *lp = static_cast<int32_t *>(whole(lens, "context_lens"));
    int *flag = static_cast<int *>(whole(err, "err_flag"));
    if (T == 0) return PyLong_FromLong(XS_OK);
    const void *kp = k.data_ptr(), *vp = v.data_ptr();
    return status([&] {
        return paged ? reinterpret_cast<decltype(&xs_kv4_append_paged)>(entry)(
                           kp, k_stride, vp, v_stride, kcp, vcp, static_cast<const int32_t *>(wp), width,
                           lp, t, hkv, d, kPage, blocks, code, flag, s)
                     : reinterpret_cast<decltype(&xs_kv4_append)>(entry)(
                           kp, k_stride, vp, v_stride, kcp, vcp, static_cast<const int64_t *>(wp), t,
                           hkv, d, kPage, blocks, code, flag, s);
    });
}

PyObject *kv4_unpack(Args a) {
    void *entry = a.entry();
    const at::Tensor &ko = a.tensor("k_out"), &vo = a.tensor("v_out");
    const at::Tensor &kc = a.tensor("k_cache"), &vc = a.tensor("v_cache");
    const at::Tensor &ids = a.tensor("block_ids");
    const at::Tensor *err = a.maybe("err_flag");
    PyObject *stream = a.next();
    dims(ko, 4, "k_out");
    const int64_t n = ko.size(0), Hkv = ko.size(1), D = ko.size(3);
    want(ko, ko.scalar_type(), {n, Hkv, kPage, D}, "k_out");
    want(vo, ko.scalar_type(), {n, Hkv, kPage, D}, "v_out");
    want(ids, at::kInt, {n}, "block_ids");
    want(err, at::kInt, {1}, "err_flag");
    const int64_t blocks = kv4_pools(kc, vc, Hkv, D);
    const int code = dtype_code(ko), count = as_int(n, "k_out"), hkv = as_int(Hkv, "k_out"),
              d = as_int(D, "k_out");
    const cudaStream_t s = stream_for(stream, {&ko, &vo, &kc, &vc, &ids, err});
    void *kop = whole(ko, "k_out"), *vop = whole(vo, "v_out");
    const void *kcp = whole(kc, "k_cache"), *vcp = whole(vc, "v_cache");
    const int32_t *ip = static_cast<int32_t *>(whole(ids, "block_ids"));
    int *flag = static_cast<int *>(whole(err, "err_flag"));
    if (n == 0) return PyLong_FromLong(XS_OK);
    return status([&] {
        return reinterpret_cast<decltype(&xs_kv4_unpack)>(entry)(kop, vop, kcp, vcp, ip, count, hkv, d,
                                                                 kPage, blocks, code, flag, s);
    });
}

PyObject *kv4_decode(Args a) {
    void *entry = a.entry();
    const at::Tensor &out = a.tensor("out"), &q = a.tensor("q");
    const at::Tensor &kc = a.tensor("k_cache"), &vc = a.tensor("v_cache");
    const at::Tensor &tables = a.tensor("block_tables"), &lens = a.tensor("context_lens");
    const float scale = static_cast<float>(a.number());
    const at::Tensor &ws = a.tensor("workspace");
    const int ws_batch = a.integer("workspace"), ws_hq = a.integer("workspace"),
              ws_hkv = a.integer("workspace"), ws_d = a.integer("workspace");
    const at::Tensor *sinks = a.maybe("sinks");
    const int window = a.integer("window");
    const at::Tensor *err = a.maybe("err_flag");
    PyObject *stream = a.next();
    dims(q, 3, "q"), dims(kc, 3, "a 4-bit pool");
    const int64_t B = q.size(0), Hq = q.size(1), D = q.size(2), Hkv = kc.size(1);
    want(out, q.scalar_type(), {B, Hq, D}, "out");
    const int64_t blocks = kv4_pools(kc, vc, Hkv, D);
    const int width = table_width(tables, lens, B);
    want(sinks, q.scalar_type(), {Hq}, "sinks");
    want(err, at::kInt, {1}, "err_flag");
    if (ws_hq != Hq || ws_hkv != Hkv || ws_d != D || B > ws_batch)
        refuse("the workspace is for other heads or a smaller batch");
    const int code = dtype_code(q), b = as_int(B, "q"), hq = as_int(Hq, "q"),
              hkv = as_int(Hkv, "k_cache"), d = as_int(D, "q");
    const cudaStream_t s = stream_for(stream, {&q, &out, &kc, &vc, &tables, &lens, &ws, sinks, err});
    void *op = whole(out, "out"), *wp = whole(ws, "workspace");
    const void *qp = whole(q, "q"), *kcp = whole(kc, "k_cache"), *vcp = whole(vc, "v_cache");
    const int32_t *tp = static_cast<int32_t *>(whole(tables, "block_tables"));
    const int32_t *lp = static_cast<int32_t *>(whole(lens, "context_lens"));
    const void *zp = whole(sinks, "sinks");
    int *flag = static_cast<int *>(whole(err, "err_flag"));
    if (B == 0) return PyLong_FromLong(XS_OK);
    const size_t bytes = static_cast<size_t>(ws.numel()) * ws.element_size();
    return status([&] {
        return reinterpret_cast<decltype(&xs_kv4_decode)>(entry)(op, qp, kcp, vcp, tp, width, lp, zp,
                                                                 window, b, hq, hkv, d, kPage, blocks,
                                                                 scale, wp, bytes, code, flag, s);
    });
}

// ------------------------------------------------------------------ shared pages

// The pool's state: free stack, its top, and the counts of further owners.
struct Share {
    const at::Tensor &stack, &top, &extra;
    explicit Share(Args &a)
        : stack(a.tensor("free_stack")), top(a.tensor("free_top")), extra(a.tensor("extra_refs")) {
        if (stack.scalar_type() != at::kInt || top.scalar_type() != at::kInt ||
            extra.scalar_type() != at::kInt)
            refuse("free_stack, free_top and extra_refs must be int32");
        if (top.numel() != 1) refuse("free_top must be one int32");
    }
    int32_t *ptr(const at::Tensor &t, const char *name) const {
        return static_cast<int32_t *>(whole(t, name));
    }
};

PyObject *block_fork(Args a) {
    void *entry = a.entry();
    const at::Tensor &parents = a.tensor("parents"), &children = a.tensor("children");
    const at::Tensor &tables = a.tensor("block_tables"), &lens = a.tensor("context_lens");
    const Share sh(a);
    const at::Tensor &copies = a.tensor("copies");
    const int bs = a.integer("block_size");
    const at::Tensor *err = a.maybe("err_flag");
    PyObject *stream = a.next();
    const int64_t n = parents.numel(), B = lens.numel();
    want(parents, at::kInt, {n}, "parents");
    want(children, at::kInt, {n}, "children");
    want(copies, at::kLong, {n, 2}, "copies");
    want(err, at::kInt, {1}, "err_flag");
    const int width = table_width(tables, lens, B);
    const cudaStream_t s = stream_for(
        stream, {&parents, &children, &tables, &lens, &sh.stack, &sh.top, &sh.extra, &copies, err});
    const int32_t *pp = static_cast<int32_t *>(whole(parents, "parents"));
    const int32_t *cp = static_cast<int32_t *>(whole(children, "children"));
    int32_t *tp = static_cast<int32_t *>(whole(tables, "block_tables"));
    int32_t *lp = static_cast<int32_t *>(whole(lens, "context_lens"));
    const int32_t *sp = sh.ptr(sh.stack, "free_stack");
    int32_t *top = sh.ptr(sh.top, "free_top"), *ep = sh.ptr(sh.extra, "extra_refs");
    int64_t *op = static_cast<int64_t *>(whole(copies, "copies"));
    int *flag = static_cast<int *>(whole(err, "err_flag"));
    if (n == 0) return PyLong_FromLong(XS_OK);
    const int count = as_int(n, "parents"), b = as_int(B, "context_lens");
    return status([&] {
        return reinterpret_cast<decltype(&xs_block_fork)>(entry)(
            pp, cp, count, tp, width, lp, b, bs, sp, top, ep, sh.extra.numel(), op, flag, s);
    });
}

// cut: to new lengths (xs_block_truncate).
PyObject *block_release(Args a, bool cut) {
    void *entry = a.entry();
    const at::Tensor &ids = a.tensor("seq_ids");
    const at::Tensor *to = cut ? &a.tensor("new_lens") : nullptr;
    const at::Tensor &tables = a.tensor("block_tables"), &lens = a.tensor("context_lens");
    const Share sh(a);
    const int bs = a.integer("block_size");
    const at::Tensor *err = a.maybe("err_flag");
    PyObject *stream = a.next();
    const int64_t n = ids.numel(), B = lens.numel();
    want(ids, at::kInt, {n}, "seq_ids");
    want(to, at::kInt, {n}, "new_lens");
    want(err, at::kInt, {1}, "err_flag");
    const int width = table_width(tables, lens, B);
    const cudaStream_t s =
        stream_for(stream, {&ids, to, &tables, &lens, &sh.stack, &sh.top, &sh.extra, err});
    const int32_t *ip = static_cast<int32_t *>(whole(ids, "seq_ids"));
    const int32_t *np = static_cast<int32_t *>(whole(to, "new_lens"));
    int32_t *tp = static_cast<int32_t *>(whole(tables, "block_tables"));
    int32_t *lp = static_cast<int32_t *>(whole(lens, "context_lens"));
    int32_t *sp = sh.ptr(sh.stack, "free_stack"), *top = sh.ptr(sh.top, "free_top"),
            *ep = sh.ptr(sh.extra, "extra_refs");
    int *flag = static_cast<int *>(whole(err, "err_flag"));
    if (n == 0) return PyLong_FromLong(XS_OK);
    const int count = as_int(n, "seq_ids"), b = as_int(B, "context_lens");
    return status([&] {
        return cut ? reinterpret_cast<decltype(&xs_block_truncate)>(entry)(
                         ip, np, count, tp, width, lp, b, bs, sp, top, sh.stack.numel(), ep,
                         sh.extra.numel(), flag, s)
                   : reinterpret_cast<decltype(&xs_block_release)>(entry)(
                         ip, count, tp, width, lp, b, bs, sp, top, sh.stack.numel(), ep,
                         sh.extra.numel(), flag, s);
    });
}

PyObject *block_compact(Args a) {
    void *entry = a.entry();
    const at::Tensor &tables = a.tensor("block_tables"), &out = a.tensor("block_tables_out");
    const at::Tensor &lens = a.tensor("context_lens");
    const at::Tensor &extra = a.tensor("extra_refs"), &extra_out = a.tensor("extra_refs_out");
    const at::Tensor &stack = a.tensor("free_stack"), &top = a.tensor("free_top");
    const at::Tensor &remap = a.tensor("remap"), &moves = a.tensor("moves"),
                     &n_moves = a.tensor("n_moves");
    const int bs = a.integer("block_size");
    const at::Tensor *err = a.maybe("err_flag");
    PyObject *stream = a.next();
    const int64_t B = lens.numel(), nb = extra.numel();
    const int width = table_width(tables, lens, B);
    want(out, at::kInt, {B, width}, "block_tables_out");
    want(extra, at::kInt, {nb}, "extra_refs");
    want(extra_out, at::kInt, {nb}, "extra_refs_out");
    want(stack, at::kInt, {nb}, "free_stack");
    want(top, at::kInt, {1}, "free_top");
    want(remap, at::kInt, {nb}, "remap");
    want(moves, at::kLong, {nb / 2, 2}, "moves");
    want(n_moves, at::kInt, {1}, "n_moves");
    want(err, at::kInt, {1}, "err_flag");
    const cudaStream_t s = stream_for(stream, {&tables, &out, &lens, &extra, &extra_out, &stack, &top,
                                               &remap, &moves, &n_moves, err});
    auto i32 = [](const at::Tensor &t, const char *name) { return static_cast<int32_t *>(whole(t, name)); };
    const int32_t *tp = i32(tables, "block_tables"), *lp = i32(lens, "context_lens"),
                  *ep = i32(extra, "extra_refs");
    int32_t *to = i32(out, "block_tables_out"), *eo = i32(extra_out, "extra_refs_out"),
            *sp = i32(stack, "free_stack"), *tt = i32(top, "free_top"), *rp = i32(remap, "remap"),
            *np = i32(n_moves, "n_moves");
    int64_t *mp = static_cast<int64_t *>(whole(moves, "moves"));
    int *flag = static_cast<int *>(whole(err, "err_flag"));
    const int b = as_int(B, "context_lens");
    return status([&] {
        return reinterpret_cast<decltype(&xs_block_compact)>(entry)(tp, to, width, lp, b, bs, ep, eo, sp,
                                                                    tt, nb, rp, mp, np, flag, s);
    });
}

PyObject *block_copy(Args a) {
    void *entry = a.entry();
    const at::Tensor &k = a.tensor("k_pools"), &v = a.tensor("v_pools"), &pairs = a.tensor("pairs");
    const at::Tensor *count = a.maybe("count"), *err = a.maybe("err_flag");
    PyObject *stream = a.next();
    if (k.dim() < 3 || k.scalar_type() != v.scalar_type() || k.sizes() != v.sizes())
        refuse("k_pools and v_pools must be [layers, num_blocks, ...] of one type and shape");
    const int64_t n = pairs.dim() ? pairs.size(0) : 0;
    want(pairs, at::kLong, {n, 2}, "pairs");
    want(count, at::kInt, {1}, "count");
    want(err, at::kInt, {1}, "err_flag");
    const cudaStream_t s = stream_for(stream, {&k, &v, &pairs, count, err});
    void *kp = whole(k, "k_pools"), *vp = whole(v, "v_pools");
    const int64_t *pp = static_cast<int64_t *>(whole(pairs, "pairs"));
    const int32_t *cp = static_cast<int32_t *>(whole(count, "count"));
    int *flag = static_cast<int *>(whole(err, "err_flag"));
    if (k.numel() == 0 || n == 0) return PyLong_FromLong(XS_OK);
    const int layers = as_int(k.size(0), "k_pools");
    const int64_t nb = k.size(1), block = k.numel() / (layers * nb) * k.element_size();
    return status([&] {
        return reinterpret_cast<decltype(&xs_block_copy)>(entry)(kp, vp, layers, nb * block, pp, n, cp,
                                                                 block, nb, flag, s);
    });
}

// ------------------------------------------------------------------ bounded caches

PyObject *decode_bounded(Args a, bool weights) {
    void *entry = a.entry();
    const at::Tensor &out = a.tensor("out");
    const at::Tensor *scores = weights ? &a.tensor("scores") : nullptr;
    const at::Tensor &q = a.tensor("q");
    const at::Tensor &kc = a.tensor("k_cache"), &vc = a.tensor("v_cache");
    const at::Tensor &tables = a.tensor("block_tables"), &lens = a.tensor("context_lens");
    const float scale = static_cast<float>(a.number());
    const at::Tensor &ws = a.tensor("workspace");
    const int ws_hq = a.integer("workspace"), ws_hkv = a.integer("workspace"), ws_d = a.integer("workspace");
    const int first = weights ? 0 : a.integer("first"), window = weights ? 0 : a.integer("window");
    const at::Tensor *scored = weights ? a.maybe("scored_lens") : nullptr;
    const at::Tensor *sinks = a.maybe("sinks"), *err = a.maybe("err_flag");
    PyObject *stream = a.next();
    dims(q, 3, "q"), dims(kc, 4, "a pool");
    const int64_t B = q.size(0), Hq = q.size(1), D = q.size(2), Hkv = kc.size(1);
    want(out, q.scalar_type(), {B, Hq, D}, "out");
    bool kv4 = false;
    const int64_t blocks = pools(kc, vc, q.scalar_type(), Hkv, D, &kv4);
    if (kv4) refuse("a 4-bit pool is not supported here");
    const int width = table_width(tables, lens, B);
    want(scores, at::kFloat, {B, Hkv, static_cast<int64_t>(width) * kPage}, "scores");
    want(scored, at::kInt, {B}, "scored_lens");
    want(sinks, q.scalar_type(), {Hq}, "sinks");
    want(err, at::kInt, {1}, "err_flag");
    if (ws_hq != Hq || ws_hkv != Hkv || ws_d != D) refuse("the workspace is for other heads");
    const int code = dtype_code(q), b = as_int(B, "q"), hq = as_int(Hq, "q"),
              hkv = as_int(Hkv, "k_cache"), d = as_int(D, "q");
    const int64_t q_stride = rows(q, "q");
    const cudaStream_t s = stream_for(stream, {&q, &out, scores, &kc, &vc, &tables, &lens, &ws, scored, sinks, err});
    void *op = whole(out, "out"), *wp = whole(ws, "workspace");
    float *sp = static_cast<float *>(whole(scores, "scores"));
    const int32_t *np = static_cast<int32_t *>(whole(scored, "scored_lens"));
    const void *qp = q.data_ptr(), *kcp = whole(kc, "k_cache"), *vcp = whole(vc, "v_cache");
    const int32_t *tp = static_cast<int32_t *>(whole(tables, "block_tables"));
    const int32_t *lp = static_cast<int32_t *>(whole(lens, "context_lens"));
    const void *zp = whole(sinks, "sinks");
    int *flag = static_cast<int *>(whole(err, "err_flag"));
    if (B == 0) return PyLong_FromLong(XS_OK);
    const size_t bytes = static_cast<size_t>(ws.numel()) * ws.element_size();
    return status([&] {
        return weights ? reinterpret_cast<decltype(&xs_paged_decode_weights)>(entry)(
                             op, sp, np, qp, q_stride, kcp, vcp, tp, width, lp, zp, b, hq, hkv, d, kPage, blocks,
                             scale, wp, bytes, code, flag, s)
                       : reinterpret_cast<decltype(&xs_paged_decode_first)>(entry)(
                             op, qp, q_stride, kcp, vcp, tp, width, lp, zp, first, window, b, hq, hkv, d, kPage,
                             blocks, scale, wp, bytes, code, flag, s);
    });
}

PyObject *prefill_first(Args a) {
    void *entry = a.entry();
    const at::Tensor &out = a.tensor("out"), &q = a.tensor("q");
    const at::Tensor &kc = a.tensor("k_cache"), &vc = a.tensor("v_cache"), &ids = a.tensor("block_ids");
    const int start = a.integer("start_pos");
    const float scale = static_cast<float>(a.number());
    const int first = a.integer("first"), window = a.integer("window");
    const at::Tensor *err = a.maybe("err_flag");
    PyObject *stream = a.next();
    dims(q, 3, "q"), dims(kc, 4, "a pool");
    const int64_t T = q.size(0), Hq = q.size(1), D = q.size(2), Hkv = kc.size(1), n = ids.numel();
    want(out, q.scalar_type(), {T, Hq, D}, "out");
    bool kv4 = false;
    const int64_t blocks = pools(kc, vc, q.scalar_type(), Hkv, D, &kv4);
    if (kv4) refuse("a 4-bit pool is not supported here");
    want(ids, at::kInt, {n}, "block_ids");
    want(err, at::kInt, {1}, "err_flag");
    const int code = dtype_code(q), t = as_int(T, "q"), hq = as_int(Hq, "q"), hkv = as_int(Hkv, "k_cache"),
              d = as_int(D, "q"), count = as_int(n, "block_ids");
    const cudaStream_t s = stream_for(stream, {&q, &out, &kc, &vc, &ids, err});
    void *op = whole(out, "out");
    const void *qp = whole(q, "q"), *kcp = whole(kc, "k_cache"), *vcp = whole(vc, "v_cache");
    const int32_t *ip = static_cast<int32_t *>(whole(ids, "block_ids"));
    int *flag = static_cast<int *>(whole(err, "err_flag"));
    if (T == 0) return PyLong_FromLong(XS_OK);
    return status([&] {
        return reinterpret_cast<decltype(&xs_paged_prefill_first)>(entry)(
            op, qp, kcp, vcp, ip, count, t, start, first, window, hq, hkv, d, kPage, blocks, scale, code, flag, s);
    });
}

PyObject *kv_evict(Args a) {
    void *entry = a.entry();
    const at::Tensor &ids = a.tensor("seq_ids");
    const at::Tensor &k = a.tensor("k_pools"), &v = a.tensor("v_pools"), &scores = a.tensor("scores");
    const at::Tensor &tables = a.tensor("block_tables"), &lens = a.tensor("context_lens");
    const at::Tensor &kept = a.tensor("kept"), &new_lens = a.tensor("new_lens");
    const int first = a.integer("first"), recent = a.integer("recent"), limit = a.integer("limit");
    const at::Tensor *extra = a.maybe("extra_refs"), *err = a.maybe("err_flag");
    PyObject *stream = a.next();
    dims(k, 5, "k_pools");
    const int64_t n = ids.numel(), B = lens.numel(), L = k.size(0), nb = k.size(1), Hkv = k.size(2), D = k.size(4);
    want(k, k.scalar_type(), {L, nb, Hkv, kPage, D}, "k_pools");
    want(v, k.scalar_type(), {L, nb, Hkv, kPage, D}, "v_pools");
    const int width = table_width(tables, lens, B);
    want(scores, at::kFloat, {L, B, Hkv, static_cast<int64_t>(width) * kPage}, "scores");
    want(ids, at::kInt, {n}, "seq_ids");
    dims(kept, 4, "kept");
    const int64_t budget = kept.size(3);
    want(kept, at::kInt, {L, n, Hkv, budget}, "kept");
    want(new_lens, at::kInt, {n}, "new_lens");
    want(extra, at::kInt, {nb}, "extra_refs");
    want(err, at::kInt, {1}, "err_flag");
    const int code = dtype_code(k), count = as_int(n, "seq_ids"), layers = as_int(L, "k_pools"),
              b = as_int(B, "context_lens"), hkv = as_int(Hkv, "k_pools"), d = as_int(D, "k_pools"),
              keep = as_int(budget, "kept");
    const cudaStream_t s = stream_for(stream, {&ids, &k, &v, &scores, &tables, &lens, &kept, &new_lens, extra, err});
    const int32_t *ip = static_cast<int32_t *>(whole(ids, "seq_ids"));
    void *kp = whole(k, "k_pools"), *vp = whole(v, "v_pools");
    float *sp = static_cast<float *>(whole(scores, "scores"));
    const int32_t *tp = static_cast<int32_t *>(whole(tables, "block_tables"));
    const int32_t *lp = static_cast<int32_t *>(whole(lens, "context_lens"));
    const int32_t *ep = static_cast<int32_t *>(whole(extra, "extra_refs"));
    int32_t *at = static_cast<int32_t *>(whole(kept, "kept")), *np = static_cast<int32_t *>(whole(new_lens, "new_lens"));
    int *flag = static_cast<int *>(whole(err, "err_flag"));
    if (n == 0) return PyLong_FromLong(XS_OK);
    return status([&] {
        return reinterpret_cast<decltype(&xs_kv_evict)>(entry)(
            ip, count, kp, vp, layers, nb * hkv * kPage * d * k.element_size(), sp, tp, width, lp, b, ep, first,
            recent, keep, limit, hkv, d, kPage, nb, code, at, np, flag, s);
    });
}

// ------------------------------------------------------------------ the module

template <typename F> PyObject *guarded(PyObject *const *args, Py_ssize_t n, F &&f) {
    try {
        return f(Args{args, args + n});
    } catch (const Refusal &r) {
        PyErr_SetString(PyExc_ValueError, r.what.c_str());
    } catch (const PythonError &) {
    } catch (const std::exception &e) {
        PyErr_SetString(PyExc_RuntimeError, e.what());
    }
    return nullptr;
}

#define XS_BIND(name, expr)                                                       \
    PyObject *py_##name(PyObject *, PyObject *const *args, Py_ssize_t n) {        \
        return guarded(args, n, [](Args a) { return expr; });                     \
    }
XS_BIND(xs_qk_norm_rope, norm_rope(a, kPlain))
XS_BIND(xs_qk_norm_rope_append, norm_rope(a, kSlots))
XS_BIND(xs_qk_norm_rope_append_paged, norm_rope(a, kPaged))
XS_BIND(xs_kv4_append, kv4_append(a, false))
XS_BIND(xs_kv4_append_paged, kv4_append(a, true))
XS_BIND(xs_kv4_unpack, kv4_unpack(a))
XS_BIND(xs_kv4_decode, kv4_decode(a))
XS_BIND(xs_block_fork, block_fork(a))
XS_BIND(xs_block_release, block_release(a, false))
XS_BIND(xs_block_truncate, block_release(a, true))
XS_BIND(xs_kv_evict, kv_evict(a))
XS_BIND(xs_block_compact, block_compact(a))
XS_BIND(xs_block_copy, block_copy(a))
XS_BIND(xs_paged_decode_first, decode_bounded(a, false))
XS_BIND(xs_paged_decode_weights, decode_bounded(a, true))
XS_BIND(xs_paged_prefill_first, prefill_first(a))

#define XS_METHOD(name) \
    {#name, reinterpret_cast<PyCFunction>(reinterpret_cast<void *>(py_##name)), METH_FASTCALL, nullptr}
PyMethodDef methods[] = {XS_METHOD(xs_qk_norm_rope),
                         XS_METHOD(xs_qk_norm_rope_append),
                         XS_METHOD(xs_qk_norm_rope_append_paged),
                         XS_METHOD(xs_kv4_append),
                         XS_METHOD(xs_kv4_append_paged),
                         XS_METHOD(xs_kv4_unpack),
                         XS_METHOD(xs_kv4_decode),
                         XS_METHOD(xs_block_fork),
                         XS_METHOD(xs_block_release),
                         XS_METHOD(xs_block_truncate),
                         XS_METHOD(xs_kv_evict),
                         XS_METHOD(xs_block_compact),
                         XS_METHOD(xs_block_copy),
                         XS_METHOD(xs_paged_decode_first),
                         XS_METHOD(xs_paged_decode_weights),
                         XS_METHOD(xs_paged_prefill_first),
                         {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "xs_bind", nullptr, -1, methods,
                      nullptr,               nullptr,   nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit_xs_bind() { return PyModule_Create(&module); }
