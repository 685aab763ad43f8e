// fastcall.cpp -- the short calls' argument checks, outside the interpreter.
//
// The page calls, rope_kv_write, norm_rope_kv_write, chunk_attn and lora_proj run for
// 2 to 20 us on the GPU in a serving step, and checking a dozen tensors attribute by
// attribute in Python and converting them for ctypes took 8 to 10 us a call.
// The functions here check the same things on the tensors themselves (about 0.1
// us a tensor) and call the C ABI. They know only the good case: a call that
// is not all in order, or leaves an output to be allocated, returns None, and
// the Python binding goes through its own checks, which name the fault.
//
// The addresses of the C functions are handed over by bind(), so that this
// module and ctypes use the same loaded library.
#include <Python.h>

#include <ATen/core/Tensor.h>
#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/autograd/python_variable.h>

#include "specverify.h"

namespace {

decltype(&svf_page_reserve) g_reserve;
decltype(&svf_page_release) g_release;
decltype(&svf_rope_kv_write) g_rope;
decltype(&svf_lora_proj) g_lora;
decltype(&svf_page_release_shared) g_release_shared;
decltype(&svf_page_fork) g_fork;
decltype(&svf_page_copy) g_copy;
decltype(&svf_norm_rope_kv_write) g_norm_rope;
decltype(&svf_chunk_attn) g_chunk;

PyObject *k_free, *k_state, *k_slots, *k_positions, *k_row_offsets, *k_status, *k_n_released,
    *k_cuda_stream, *k_shares, *k_copy_src, *k_copy_dst, *k_copy_len;

const at::Tensor *tensor(PyObject *o) {
    return o && THPVariable_Check(o) ? &THPVariable_Unpack(o) : nullptr;
}
const at::Tensor *entry(PyObject *dict, PyObject *key) {
    return PyDict_Check(dict) ? tensor(PyDict_GetItemWithError(dict, key)) : nullptr;
}

// A call's device and the checks against it.
struct Args {
    int dev = -1;
    bool ok = true;

    bool device_of(const at::Tensor *t) {
        dev = t && t->is_cuda() ? (int)t->get_device() : -1;
        return ok = dev >= 0 && (int)c10::cuda::current_device() == dev;
    }
    // the address of a contiguous tensor of this type, on the call's device
    template <typename T = void>
    T *ptr(const at::Tensor *t, at::ScalarType type) {
        if (!t || t->scalar_type() != type || !t->is_cuda() || (int)t->get_device() != dev ||
            !t->is_contiguous()) {
            ok = false;
            return nullptr;
        }
        return static_cast<T *>(t->data_ptr());
    }
    template <typename T = void>
    T *ptr(const at::Tensor *t, at::ScalarType type, std::initializer_list<int64_t> shape) {
        if (!t || t->sizes() != c10::IntArrayRef(shape)) {
            ok = false;
            return nullptr;
        }
        return ptr<T>(t, type);
    }
    int32_t *i32(const at::Tensor *t, std::initializer_list<int64_t> shape) {
        return ptr<int32_t>(t, at::kInt, shape);
    }
    // elements between the rows of [T, heads, D] with dense heads
    int64_t rows(const at::Tensor *t, at::ScalarType type, int64_t T, int64_t heads, int64_t D) {
        if (!t || t->dim() != 3 || t->size(0) != T || t->size(1) != heads || t->size(2) != D ||
            t->scalar_type() != type || !t->is_cuda() || (int)t->get_device() != dev ||
            (t->stride(2) != 1 && D > 1) || (t->stride(1) != D && heads > 1)) {
            ok = false;
            return 0;
        }
        return T > 1 ? t->stride(0) : heads * D;
    }
    double real(PyObject *o) {
        const double v = PyFloat_CheckExact(o) ? PyFloat_AS_DOUBLE(o) : -1.0;
        if (!(v >= 0.0)) ok = false;
        return v;
    }
    int integer(PyObject *o) {
        const long v = PyLong_Check(o) ? PyLong_AsLong(o) : -1;
        if (v < 0 || v > INT_MAX) {
            PyErr_Clear();
            ok = false;
            return 0;
        }
        return (int)v;
    }
    svf_stream_t stream(PyObject *o) {
        if (o == Py_None)
            return reinterpret_cast<svf_stream_t>(
                c10::cuda::getCurrentCUDAStream((c10::DeviceIndex)dev).stream());
        PyObject *v = PyObject_GetAttr(o, k_cuda_stream);
        void *p = v ? PyLong_AsVoidPtr(v) : nullptr;
        Py_XDECREF(v);
        if (PyErr_Occurred()) {
            PyErr_Clear();
            ok = false;
        }
        return reinterpret_cast<svf_stream_t>(p);
    }
};

bool fits(int64_t v) { return v <= INT_MAX; }

// The C call, with the interpreter free: a launch waits where the stream is full.
template <typename F>
PyObject *call(F f) {
    int rc;
    Py_BEGIN_ALLOW_THREADS
    rc = f();
    Py_END_ALLOW_THREADS
    return PyLong_FromLong(rc);
}

// page_reserve(pool, page_table, seq_lens, new_lens, page_size, rows, depth, outputs, stream)
PyObject *page_reserve(PyObject *const *a, Py_ssize_t n) {
    if (n != 9 || !g_reserve) Py_RETURN_NONE;
    const at::Tensor *table = tensor(a[1]), *free = entry(a[0], k_free);
    Args c;
    if (!c.device_of(table) || table->dim() != 2 || !free || free->dim() != 1) Py_RETURN_NONE;
    const int64_t B = table->size(0), mp = table->size(1), pages = free->numel();
    const int ps = c.integer(a[4]), rows = c.integer(a[5]);
    if (B < 1) Py_RETURN_NONE;  // the binding fills the outputs
    const at::Tensor *depth = tensor(a[6]);
    if ((a[6] != Py_None && (!depth || depth->numel() != rows)) || !fits(B) || !fits(mp) ||
        !fits(pages))
        Py_RETURN_NONE;
    int32_t *d = depth ? c.ptr<int32_t>(depth, at::kInt) : nullptr;
    int32_t *t = c.ptr<int32_t>(table, at::kInt), *f = c.ptr<int32_t>(free, at::kInt);
    int32_t *st = c.i32(entry(a[0], k_state), {4}), *l = c.i32(tensor(a[2]), {B}),
            *w = c.i32(tensor(a[3]), {B}), *slots = c.i32(entry(a[7], k_slots), {rows}),
            *pos = c.i32(entry(a[7], k_positions), {rows}),
            *off = c.i32(entry(a[7], k_row_offsets), {B + 1}),
            *status = c.i32(entry(a[7], k_status), {B});
    if (!c.ok) Py_RETURN_NONE;
    const svf_stream_t s = c.stream(a[8]);
    if (!c.ok) Py_RETURN_NONE;
    return call([&] {
        return g_reserve(t, (int)mp, ps, f, st, (int)pages, l, w, (int)B, rows, d, slots, pos, off,
                         status, s);
    });
}

// page_release(pool, page_table, old_lens, keep_lens, page_size, outputs, stream)
PyObject *page_release(PyObject *const *a, Py_ssize_t n) {
    if (n != 7 || !g_release) Py_RETURN_NONE;
    const at::Tensor *table = tensor(a[1]), *free = entry(a[0], k_free);
    Args c;
    if (!c.device_of(table) || table->dim() != 2 || !free || free->dim() != 1) Py_RETURN_NONE;
    const int64_t B = table->size(0), mp = table->size(1), pages = free->numel();
    const int ps = c.integer(a[4]);
    if (!fits(B) || !fits(mp) || !fits(pages)) Py_RETURN_NONE;
    int32_t *t = c.ptr<int32_t>(table, at::kInt), *f = c.ptr<int32_t>(free, at::kInt);
    int32_t *st = c.i32(entry(a[0], k_state), {4}), *o = c.i32(tensor(a[2]), {B}),
            *k = c.i32(tensor(a[3]), {B}), *nr = c.i32(entry(a[5], k_n_released), {B}),
            *status = c.i32(entry(a[5], k_status), {B});
    if (!c.ok) Py_RETURN_NONE;
    const svf_stream_t s = c.stream(a[6]);
    if (!c.ok) Py_RETURN_NONE;
    return call([&] {
        return g_release(t, (int)mp, ps, f, st, (int)pages, o, k, (int)B, nr, status, s);
    });
}

// rope_kv_write(q, k, v, rope, positions, slots, k_cache, v_cache, q_out, interleaved, status,
//               stream)
PyObject *rope_kv_write(PyObject *const *a, Py_ssize_t n) {
    if (n != 12 || !g_rope) Py_RETURN_NONE;
    const at::Tensor *q = tensor(a[0]), *k = tensor(a[1]), *v = tensor(a[2]), *rope = tensor(a[3]),
                     *kc = tensor(a[6]), *vc = tensor(a[7]);
    Args c;
    if (!c.device_of(q) || q->dim() != 3 || !k || k->dim() != 3 || !v || !rope ||
        rope->dim() != 2 || !kc || kc->dim() != 4 || !vc || (a[9] != Py_True && a[9] != Py_False))
        Py_RETURN_NONE;
    const at::ScalarType type = q->scalar_type();
    if (type != at::kFloat && type != at::kBFloat16) Py_RETURN_NONE;
    const int64_t T = q->size(0), Hq = q->size(1), D = q->size(2), Hkv = k->size(1),
                  max_pos = rope->size(0), rot = rope->size(1), pages = kc->size(0),
                  ps = kc->size(1);
    if (!fits(T) || !fits(Hq) || !fits(D) || !fits(Hkv) || !fits(max_pos) || !fits(pages) ||
        !fits(ps) || !fits(pages * ps))
        Py_RETURN_NONE;
    const int64_t qs = c.rows(q, type, T, Hq, D), ks = c.rows(k, type, T, Hkv, D),
                  vs = c.rows(v, type, T, Hkv, D);
    const float *r = c.ptr<float>(rope, at::kFloat);
    int32_t *pos = c.i32(tensor(a[4]), {T}), *slots = c.i32(tensor(a[5]), {T}),
            *status = c.i32(tensor(a[10]), {T});
    void *kp = c.ptr(kc, type, {pages, ps, Hkv, D}), *vp = c.ptr(vc, type, {pages, ps, Hkv, D}),
         *out = c.ptr(tensor(a[8]), type, {T, Hq, D});
    if (!c.ok) Py_RETURN_NONE;
    const svf_stream_t s = c.stream(a[11]);
    if (!c.ok) Py_RETURN_NONE;
    const void *qp = q->data_ptr(), *kin = k->data_ptr(), *vin = v->data_ptr();
    return call([&] {
        return g_rope(qp, kin, vin, qs, ks, vs, (int)T, (int)Hq, (int)Hkv, (int)D,
                      type == at::kFloat ? SVF_F32 : SVF_BF16, r, (int)rot, (int)max_pos,
                      a[9] == Py_True, pos, slots, out, kp, vp, (int)(pages * ps), status, s);
    });
}

// lora_proj(x, weight, lora_a, lora_b, ids, scales, out, workspace, status, stream)
PyObject *lora_proj(PyObject *const *a, Py_ssize_t n) {
    if (n != 10 || !g_lora) Py_RETURN_NONE;
    const at::Tensor *x = tensor(a[0]), *w = tensor(a[1]), *la = tensor(a[2]), *lb = tensor(a[3]),
                     *ids = tensor(a[4]), *scales = tensor(a[5]), *out = tensor(a[6]),
                     *ws = tensor(a[7]);
    Args c;
    const at::ScalarType bf = at::kBFloat16;
    if (!c.device_of(x) || x->dim() < 1 || x->scalar_type() != bf || !w || w->dim() != 2 || !la ||
        la->dim() != 3 || !lb || !ids || ids->dim() != 1 || !out || !ws || ws->dim() < 1 ||
        (a[5] != Py_None && !scales))
        Py_RETURN_NONE;
    const int64_t O = w->size(0), H = w->size(1), A = la->size(0), rank = la->size(1),
                  G = ids->size(0);
    if (H < 1 || x->size(-1) != H || G < 1 || !fits(O) || !fits(H) || !fits(A) || !fits(rank))
        Py_RETURN_NONE;
    const int64_t R = x->numel() / H;
    if (R < 1 || R % G || !fits(R)) Py_RETURN_NONE;
    int64_t xs = H, os = O;
    if (!x->is_contiguous()) {
        if (x->dim() != 2 || x->stride(1) != 1) Py_RETURN_NONE;
        xs = x->stride(0);
    }
    if (out->dim() != x->dim() || out->size(-1) != O || out->numel() != R * O ||
        out->scalar_type() != bf || !out->is_cuda() || (int)out->get_device() != c.dev)
        Py_RETURN_NONE;
    for (int64_t d = 0; d + 1 < x->dim(); ++d)
        if (out->size(d) != x->size(d)) Py_RETURN_NONE;
    if (!out->is_contiguous()) {
        if (out->dim() != 2 || out->stride(1) != 1) Py_RETURN_NONE;
        os = out->stride(0);
    }
    void *wp = c.ptr(w, bf), *ap = c.ptr(la, bf, {A, rank, H}), *bp = c.ptr(lb, bf, {A, O, rank});
    float *sp = scales ? c.ptr<float>(scales, at::kFloat, {A}) : nullptr;
    int32_t *ip = c.ptr<int32_t>(ids, at::kInt), *status = c.i32(tensor(a[8]), {G});
    void *wsp = c.ptr(ws, ws->scalar_type());
    if (!c.ok) Py_RETURN_NONE;
    const svf_stream_t s = c.stream(a[9]);
    if (!c.ok) Py_RETURN_NONE;
    const void *xp = x->data_ptr();
    void *op = out->data_ptr();
    const size_t bytes = ws->nbytes();
    return call([&] {
        return g_lora(xp, xs, wp, ap, bp, sp, ip, (int)(R / G), (int)R, (int)H, (int)O, (int)A,
                      (int)rank, op, os, wsp, bytes, status, s);
    });
}

// page_release_shared(pool, page_table, old_lens, keep_lens, page_size, outputs, stream)
PyObject *page_release_shared(PyObject *const *a, Py_ssize_t n) {
    if (n != 7 || !g_release_shared) Py_RETURN_NONE;
    const at::Tensor *table = tensor(a[1]), *free = entry(a[0], k_free);
    Args c;
    if (!c.device_of(table) || table->dim() != 2 || !free || free->dim() != 1) Py_RETURN_NONE;
    const int64_t B = table->size(0), mp = table->size(1), pages = free->numel();
    const int ps = c.integer(a[4]);
    if (!fits(B) || !fits(mp) || !fits(pages)) Py_RETURN_NONE;
    int32_t *t = c.ptr<int32_t>(table, at::kInt), *f = c.ptr<int32_t>(free, at::kInt);
    int32_t *st = c.i32(entry(a[0], k_state), {4}), *sh = c.i32(entry(a[0], k_shares), {pages}),
            *o = c.i32(tensor(a[2]), {B}), *k = c.i32(tensor(a[3]), {B}),
            *nr = c.i32(entry(a[5], k_n_released), {B}), *status = c.i32(entry(a[5], k_status), {B});
    if (!c.ok) Py_RETURN_NONE;
    const svf_stream_t s = c.stream(a[6]);
    if (!c.ok) Py_RETURN_NONE;
    return call([&] {
        return g_release_shared(t, (int)mp, ps, f, st, (int)pages, sh, o, k, (int)B, nr, status, s);
    });
}

// page_fork(pool, page_table, seq_lens, src, dst, page_size, outputs, stream)
PyObject *page_fork(PyObject *const *a, Py_ssize_t n) {
    if (n != 8 || !g_fork) Py_RETURN_NONE;
    const at::Tensor *table = tensor(a[1]), *free = entry(a[0], k_free), *src = tensor(a[3]);
    Args c;
    if (!c.device_of(table) || table->dim() != 2 || !free || free->dim() != 1 || !src ||
        src->dim() != 1)
        Py_RETURN_NONE;
    const int64_t B = table->size(0), mp = table->size(1), pages = free->numel(), F = src->size(0);
    const int ps = c.integer(a[5]);
    if (!fits(B) || !fits(mp) || !fits(pages) || !fits(F)) Py_RETURN_NONE;
    int32_t *t = c.ptr<int32_t>(table, at::kInt), *f = c.ptr<int32_t>(free, at::kInt);
    int32_t *st = c.i32(entry(a[0], k_state), {4}), *sh = c.i32(entry(a[0], k_shares), {pages}),
            *l = c.i32(tensor(a[2]), {B}), *sp = c.i32(src, {F}), *dp = c.i32(tensor(a[4]), {F}),
            *cs = c.i32(entry(a[6], k_copy_src), {F}), *cd = c.i32(entry(a[6], k_copy_dst), {F}),
            *cl = c.i32(entry(a[6], k_copy_len), {F}), *status = c.i32(entry(a[6], k_status), {F});
    if (!c.ok) Py_RETURN_NONE;
    const svf_stream_t s = c.stream(a[7]);
    if (!c.ok) Py_RETURN_NONE;
    return call([&] {
        return g_fork(t, (int)mp, ps, f, st, (int)pages, sh, l, (int)B, sp, dp, (int)F, cs, cd, cl,
                      status, s);
    });
}

// page_copy(k_cache, v_cache, src, dst, lens, status, stream)
PyObject *page_copy(PyObject *const *a, Py_ssize_t n) {
    if (n != 7 || !g_copy) Py_RETURN_NONE;
    const at::Tensor *kc = tensor(a[0]), *vc = tensor(a[1]), *src = tensor(a[2]), *lens = tensor(a[4]);
    Args c;
    if (!c.device_of(kc) || (kc->dim() != 4 && kc->dim() != 5) || !vc || !src || src->dim() != 1 ||
        (a[4] != Py_None && !lens))
        Py_RETURN_NONE;
    const at::ScalarType type = kc->scalar_type();
    if (type != at::kFloat && type != at::kBFloat16) Py_RETURN_NONE;
    // whole caches only: layers a distance apart are left to the binding
    if (!kc->is_contiguous() || vc->sizes() != kc->sizes()) Py_RETURN_NONE;
    const int64_t at0 = kc->dim() - 4, layers = at0 ? kc->size(0) : 1, pages = kc->size(at0),
                  ps = kc->size(at0 + 1), Hkv = kc->size(at0 + 2), D = kc->size(at0 + 3),
                  m = src->size(0);
    if (!fits(layers) || !fits(pages) || !fits(ps) || !fits(Hkv) || !fits(D) || !fits(m))
        Py_RETURN_NONE;
    void *kp = c.ptr(kc, type), *vp = c.ptr(vc, type);
    int32_t *sp = c.i32(src, {m}), *dp = c.i32(tensor(a[3]), {m}),
            *lp = lens ? c.i32(lens, {m}) : nullptr, *status = c.i32(tensor(a[5]), {m});
    if (!c.ok) Py_RETURN_NONE;
    const svf_stream_t s = c.stream(a[6]);
    if (!c.ok) Py_RETURN_NONE;
    return call([&] {
        return g_copy(kp, vp, (int)layers, at0 ? (long long)(pages * ps * Hkv * D) : 0, (int)pages,
                      (int)ps, sp, dp, lp, (int)m, (int)Hkv, (int)D,
                      type == at::kFloat ? SVF_F32 : SVF_BF16, status, s);
    });
}

// norm_rope_kv_write(q, k, v, q_norm, k_norm, rope, positions, slots, k_cache, v_cache, eps,
//                    pair_axis, q_out, interleaved, status, stream)
PyObject *norm_rope_kv_write(PyObject *const *a, Py_ssize_t n) {
    if (n != 16 || !g_norm_rope) Py_RETURN_NONE;
    const at::Tensor *q = tensor(a[0]), *k = tensor(a[1]), *v = tensor(a[2]), *wq = tensor(a[3]),
                     *wk = tensor(a[4]), *rope = tensor(a[5]), *positions = tensor(a[6]),
                     *kc = tensor(a[8]), *vc = tensor(a[9]), *axis = tensor(a[11]);
    Args c;
    if (!c.device_of(q) || q->dim() != 3 || !k || k->dim() != 3 || !v || !rope ||
        rope->dim() != 2 || !kc || kc->dim() != 4 || !vc || !positions ||
        (positions->dim() != 1 && positions->dim() != 2) || (a[3] != Py_None && !wq) ||
        (a[4] != Py_None && !wk) || (a[11] != Py_None && !axis) ||
        (a[13] != Py_True && a[13] != Py_False))
        Py_RETURN_NONE;
    const at::ScalarType type = q->scalar_type();
    if (type != at::kFloat && type != at::kBFloat16) Py_RETURN_NONE;
    const int64_t T = q->size(0), Hq = q->size(1), D = q->size(2), Hkv = k->size(1),
                  max_pos = rope->size(0), rot = rope->size(1), pages = kc->size(0),
                  ps = kc->size(1), axes = positions->dim() == 2 ? positions->size(0) : 1;
    if (!fits(T) || !fits(Hq) || !fits(D) || !fits(Hkv) || !fits(max_pos) || !fits(pages) ||
        !fits(ps) || !fits(pages * ps) || !fits(rot) || axes < 1 || !fits(axes) || (axes > 1 && !axis))
        Py_RETURN_NONE;
    const int64_t qs = c.rows(q, type, T, Hq, D), ks = c.rows(k, type, T, Hkv, D),
                  vs = c.rows(v, type, T, Hkv, D);
    const float *r = c.ptr<float>(rope, at::kFloat);
    int32_t *pos = positions->dim() == 2 ? c.i32(positions, {axes, T}) : c.i32(positions, {T}),
            *ax = axis ? c.i32(axis, {rot / 2}) : nullptr, *slots = c.i32(tensor(a[7]), {T}),
            *status = c.i32(tensor(a[14]), {T});
    void *wqp = wq ? c.ptr(wq, type, {D}) : nullptr, *wkp = wk ? c.ptr(wk, type, {D}) : nullptr;
    void *kp = c.ptr(kc, type, {pages, ps, Hkv, D}), *vp = c.ptr(vc, type, {pages, ps, Hkv, D}),
         *out = c.ptr(tensor(a[12]), type, {T, Hq, D});
    const float eps = (float)c.real(a[10]);
    if (!c.ok) Py_RETURN_NONE;
    const svf_stream_t s = c.stream(a[15]);
    if (!c.ok) Py_RETURN_NONE;
    const void *qp = q->data_ptr(), *kin = k->data_ptr(), *vin = v->data_ptr();
    return call([&] {
        return g_norm_rope(qp, kin, vin, qs, ks, vs, (int)T, (int)Hq, (int)Hkv, (int)D,
                           type == at::kFloat ? SVF_F32 : SVF_BF16, wqp, wkp, eps, r, (int)rot,
                           (int)max_pos, a[13] == Py_True, pos, (int)axes, ax, slots, out, kp, vp,
                           (int)(pages * ps), status, s);
    });
}

// chunk_attn(q, k_cache, v_cache, page_table, seq_lens, row_offsets, sm_scale, out, lse, workspace,
//            status, stream): lse None writes none
PyObject *chunk_attn(PyObject *const *a, Py_ssize_t n) {
    if (n != 12 || !g_chunk) Py_RETURN_NONE;
    const at::Tensor *q = tensor(a[0]), *kc = tensor(a[1]), *vc = tensor(a[2]), *table = tensor(a[3]),
                     *lse = tensor(a[8]), *ws = tensor(a[9]);
    Args c;
    if (!c.device_of(q) || q->dim() != 3 || !kc || kc->dim() != 4 || !vc || !table ||
        table->dim() != 2 || !ws || (a[8] != Py_None && !lse))
        Py_RETURN_NONE;
    const at::ScalarType type = q->scalar_type();
    if (type != at::kFloat && type != at::kBFloat16) Py_RETURN_NONE;
    const int64_t rows = q->size(0), Hq = q->size(1), D = q->size(2), pages = kc->size(0),
                  ps = kc->size(1), Hkv = kc->size(2), B = table->size(0), mp = table->size(1);
    if (!fits(rows) || !fits(Hq) || !fits(D) || !fits(pages) || !fits(ps) || !fits(Hkv) || !fits(B) ||
        !fits(mp))
        Py_RETURN_NONE;
    void *qp = c.ptr(q, type, {rows, Hq, D}), *kp = c.ptr(kc, type, {pages, ps, Hkv, D}),
         *vp = c.ptr(vc, type, {pages, ps, Hkv, D}), *op = c.ptr(tensor(a[7]), type, {rows, Hq, D}),
         *wp = c.ptr(ws, ws->scalar_type());
    int32_t *t = c.ptr<int32_t>(table, at::kInt), *l = c.i32(tensor(a[4]), {B}),
            *off = c.i32(tensor(a[5]), {B + 1}), *status = c.i32(tensor(a[10]), {B});
    float *lp = lse ? c.ptr<float>(lse, at::kFloat, {rows, Hq}) : nullptr;
    const float scale = (float)c.real(a[6]);
    if (!c.ok) Py_RETURN_NONE;
    const svf_stream_t s = c.stream(a[11]);
    if (!c.ok) Py_RETURN_NONE;
    const size_t bytes = ws->nbytes();
    return call([&] {
        return g_chunk(qp, kp, vp, (int)pages, (int)ps, t, (int)mp, l, off, (int)B, (int)rows, (int)Hq,
                       (int)Hkv, (int)D, type == at::kFloat ? SVF_F32 : SVF_BF16, scale, op, lp, wp,
                       bytes, status, s);
    });
}

// No C++ exception leaves a function (a tensor without storage throws).
template <PyObject *(*F)(PyObject *const *, Py_ssize_t)>
PyObject *guarded(PyObject *, PyObject *const *a, Py_ssize_t n) {
    try {
        return F(a, n);
    } catch (...) {
        PyErr_Clear();
        Py_RETURN_NONE;
    }
}

// bind(page_reserve, page_release, rope_kv_write, lora_proj, page_release_shared, page_fork,
//      page_copy, norm_rope_kv_write, chunk_attn): the addresses
PyObject *bind(PyObject *, PyObject *const *a, Py_ssize_t n) {
    constexpr int kCalls = 9;
    if (n != kCalls) {
        PyErr_SetString(PyExc_TypeError, "bind takes nine addresses");
        return nullptr;
    }
    void *p[kCalls];
    for (int i = 0; i < kCalls; ++i) {
        p[i] = PyLong_AsVoidPtr(a[i]);
        if (PyErr_Occurred()) return nullptr;
    }
    g_reserve = reinterpret_cast<decltype(g_reserve)>(p[0]);
    g_release = reinterpret_cast<decltype(g_release)>(p[1]);
    g_rope = reinterpret_cast<decltype(g_rope)>(p[2]);
    g_lora = reinterpret_cast<decltype(g_lora)>(p[3]);
    g_release_shared = reinterpret_cast<decltype(g_release_shared)>(p[4]);
    g_fork = reinterpret_cast<decltype(g_fork)>(p[5]);
    g_copy = reinterpret_cast<decltype(g_copy)>(p[6]);
    g_norm_rope = reinterpret_cast<decltype(g_norm_rope)>(p[7]);
    g_chunk = reinterpret_cast<decltype(g_chunk)>(p[8]);
    Py_RETURN_NONE;
}

#define FAST(f) reinterpret_cast<PyCFunction>(reinterpret_cast<void *>(f))
PyMethodDef methods[] = {
    {"bind", FAST(bind), METH_FASTCALL, nullptr},
    {"page_reserve", FAST(guarded<page_reserve>), METH_FASTCALL, nullptr},
    {"page_release", FAST(guarded<page_release>), METH_FASTCALL, nullptr},
    {"rope_kv_write", FAST(guarded<rope_kv_write>), METH_FASTCALL, nullptr},
    {"lora_proj", FAST(guarded<lora_proj>), METH_FASTCALL, nullptr},
    {"page_release_shared", FAST(guarded<page_release_shared>), METH_FASTCALL, nullptr},
    {"page_fork", FAST(guarded<page_fork>), METH_FASTCALL, nullptr},
    {"page_copy", FAST(guarded<page_copy>), METH_FASTCALL, nullptr},
    {"norm_rope_kv_write", FAST(guarded<norm_rope_kv_write>), METH_FASTCALL, nullptr},
    {"chunk_attn", FAST(guarded<chunk_attn>), METH_FASTCALL, nullptr},
    {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_fastcall", nullptr, -1, methods,
                      nullptr,               nullptr,     nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__fastcall() {
    k_free = PyUnicode_InternFromString("free");
    k_state = PyUnicode_InternFromString("state");
    k_slots = PyUnicode_InternFromString("slots");
    k_positions = PyUnicode_InternFromString("positions");
    k_row_offsets = PyUnicode_InternFromString("row_offsets");
    k_status = PyUnicode_InternFromString("status");
    k_n_released = PyUnicode_InternFromString("n_released");
    k_cuda_stream = PyUnicode_InternFromString("cuda_stream");
    k_shares = PyUnicode_InternFromString("shares");
    k_copy_src = PyUnicode_InternFromString("copy_src");
    k_copy_dst = PyUnicode_InternFromString("copy_dst");
    k_copy_len = PyUnicode_InternFromString("copy_len");
    return PyModule_Create(&module);
}
