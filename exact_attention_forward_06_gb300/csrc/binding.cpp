// binding.cpp -- the quick way from Python into the operators around the paged
// cache: one function per operator that looks at the tensors, makes the outputs and
// calls the C ABI (attn.h).
//
// These operators run for 4 to 6 us on a decode step's few tokens, and ten tensors'
// attributes read one by one from Python, with thirty arguments through ctypes, took
// 13 us a call.  Anything that is not plainly in order (a wrong type, shape,
// device or layout, a length to be read from the device, a status that is not 0)
// returns None: the caller then goes the long way, which says what is wrong.  Nothing
// has been launched then, but where a launch failed: the first of a call's two may
// have run, and runs again (it writes outputs and workspace only).
#include <Python.h>

#include <algorithm>
#include <climits>
#include <cmath>

#include <ATen/core/Tensor.h>
#include <ATen/ops/empty.h>
#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include "attn.h"

namespace {

constexpr at::ScalarType BF16 = at::kBFloat16, I32 = at::kInt, I64 = at::kLong, U8 = at::kByte, F32 = at::kFloat;

// Reads arguments; `ok` turns false at the first that is out of order.
struct Reader {
    int dev = -1;
    bool ok = true;

    const at::Tensor *tensor(PyObject *o, at::ScalarType type) {
        if (!ok || !THPVariable_Check(o)) return fail();
        const at::Tensor &t = THPVariable_Unpack(o);
        if (t.scalar_type() != type || !t.is_cuda()) return fail();
        if (dev < 0) {
            dev = t.get_device();
            if (dev != c10::cuda::current_device()) return fail();
        } else if (t.get_device() != dev) {
            return fail();
        }
        return &t;
    }
    const at::Tensor *dense(PyObject *o, at::ScalarType type) {
        const at::Tensor *t = tensor(o, type);
        return t && t->is_contiguous() ? t : fail();
    }
    const at::Tensor *strided(PyObject *o) {
        const at::Tensor *t = tensor(o, BF16);
        return t && t->dim() >= 2 && t->stride(-1) == 1 ? t : fail();
    }
    // An int argument of the C ABI.
    int narrow(int64_t v) {
        ok = ok && v >= 0 && v <= INT_MAX;
        return (int)v;
    }
    int64_t integer(PyObject *o) {
        const int64_t v = PyLong_Check(o) ? PyLong_AsLongLong(o) : -1;
        if (v < 0) {
            PyErr_Clear();
            ok = false;
        }
        return v;
    }
    float real(PyObject *o) {
        const double v = PyFloat_AsDouble(o);
        if (v == -1.0 && PyErr_Occurred()) {
            PyErr_Clear();
            ok = false;
        }
        return (float)v;
    }
    bool truth(PyObject *o) {
        const int v = PyObject_IsTrue(o);
        if (v < 0) {
            PyErr_Clear();
            ok = false;
        }
        return v > 0;
    }
    const at::Tensor *fail() {
        ok = false;
        return nullptr;
    }
    void *stream() const { return c10::cuda::getCurrentCUDAStream((c10::DeviceIndex)dev).stream(); }
};

void *at_of(const at::Tensor *t) { return t ? t->data_ptr() : nullptr; }

// An output: the given tensor (when it has the sizes), or a new one.
struct Output {
    PyObject *given = nullptr;
    at::Tensor made;
    void *ptr = nullptr;

    void take(Reader &r, PyObject *o, at::ScalarType type, at::IntArrayRef sizes, const at::Tensor &like) {
        if (!r.ok) return;
        if (o != Py_None) {
            const at::Tensor *t = r.dense(o, type);
            if (!t) return;
            r.ok = t->sizes() == sizes;
            given = o;
            ptr = t->data_ptr();
        } else {
            made = at::empty(sizes, like.options().dtype(type));
            ptr = made.data_ptr();
        }
    }
    PyObject *object() {
        if (!ptr) Py_RETURN_NONE;
        if (!given) return THPVariable_Wrap(std::move(made));
        Py_INCREF(given);
        return given;
    }
};

PyObject *pair(Output &a, Output &b) {
    PyObject *x = a.object(), *y = x ? b.object() : nullptr;
    PyObject *t = y ? PyTuple_Pack(2, x, y) : nullptr;
    Py_XDECREF(x);
    Py_XDECREF(y);
    return t;
}

// The norm and rotation arguments: q_weight, k_weight, eps, positions, rope, interleaved.
struct Rotate {
    void *wq = nullptr, *wk = nullptr;
    float eps = 0.f;
    const int32_t *positions = nullptr;
    int n_axes = 1, rotary_dim = 0, interleaved = 0;
    const attn_rope_pair_t *rope = nullptr;

    void read(Reader &r, PyObject *const *a, at::IntArrayRef pos_sizes) {
        void **to[2] = {&wq, &wk};
        for (int i = 0; i < 2; ++i) {
            if (a[i] == Py_None) continue;
            const at::Tensor *w = r.dense(a[i], BF16);
            r.ok = r.ok && w->dim() == 1 && w->size(0) == 128;
            *to[i] = r.ok ? w->data_ptr() : nullptr;
        }
        eps = r.real(a[2]);
        if (a[3] != Py_None) {
            const at::Tensor *p = r.dense(a[3], I32);
            if (!p) return;
            if (p->sizes() != pos_sizes) {
                r.ok = p->dim() == (int64_t)pos_sizes.size() + 1 && p->sizes().slice(1) == pos_sizes;
                n_axes = r.ok ? r.narrow(p->size(0)) : 1;
            }
            positions = static_cast<const int32_t *>(p->data_ptr());
        }
        if (a[4] != Py_None) {
            const at::Tensor *t = r.dense(a[4], I64);
            if (!t || t->dim() != 2 || t->size(1) != 2) {
                r.ok = false;
                return;
            }
            rope = static_cast<const attn_rope_pair_t *>(t->data_ptr());
            rotary_dim = r.narrow(2 * t->size(0));
            if (!positions) n_axes = 4;  // the default position is the same on every axis
        }
        interleaved = r.truth(a[5]);
    }
};

// q, k, q_weight, k_weight, eps, positions, rope, interleaved, layout, q_out, k_out
PyObject *qk_norm_rope(PyObject *, PyObject *const *a, Py_ssize_t n) {
    HANDLE_TH_ERRORS
    Reader r;
    const at::Tensor *q = n == 11 ? r.strided(a[0]) : nullptr;
    const at::Tensor *k = q && a[1] != Py_None ? r.strided(a[1]) : nullptr;
    if (!q || !r.ok) Py_RETURN_NONE;
    const int64_t layout = r.integer(a[8]);
    const bool four = q->dim() == 4;
    if (!r.ok || !(four || (q->dim() == 3 && layout == ATTN_LAYOUT_BSHD))) Py_RETURN_NONE;
    const int s_dim = four ? (layout == ATTN_LAYOUT_BSHD ? 1 : 2) : 0;
    const int h_dim = four ? 3 - s_dim : 1;
    const int64_t B = four ? q->size(0) : 1, S = q->size(s_dim), Hq = q->size(h_dim), d = q->size(-1);
    if (k && (k->dim() != q->dim() || k->size(s_dim) != S || k->size(-1) != d || (four && k->size(0) != B)))
        Py_RETURN_NONE;
    const int64_t Hkv = k ? k->size(h_dim) : 0;
    const int64_t pos_sizes[2] = {four ? B : S, S};
    Rotate rot;
    rot.read(r, a + 2, at::IntArrayRef(pos_sizes, four ? 2 : 1));
    const int b = r.narrow(B), s = r.narrow(S), hq = r.narrow(Hq), hk = r.narrow(Hkv), dd = r.narrow(d);
    Output qo, ko;
    qo.take(r, a[9], BF16, q->sizes(), *q);
    if (k)
        ko.take(r, a[10], BF16, k->sizes(), *k);
    else if (a[10] != Py_None)
        Py_RETURN_NONE;
    if (!r.ok) Py_RETURN_NONE;
    // the stride of a dimension of length one is never used, whatever it says
    const bool many = four && B > 1, lng = S > 1;
    const auto stride = [](const at::Tensor *t, int dim, bool used) { return t && used ? (size_t)t->stride(dim) : 0; };
    if (attn_qk_norm_rope(q->data_ptr(), at_of(k), qo.ptr, ko.ptr, rot.wq, rot.wk, rot.eps, rot.positions, rot.n_axes,
                          rot.rope, rot.rotary_dim, rot.interleaved, b, s, hq, hk, dd, (int)layout, stride(q, 0, many),
                          stride(q, s_dim, lng), stride(q, h_dim, Hq > 1), stride(k, 0, many), stride(k, s_dim, lng),
                          stride(k, h_dim, Hkv > 1), r.stream()) != ATTN_OK)
        Py_RETURN_NONE;
    return pair(qo, ko);
    END_HANDLE_TH_ERRORS
}

// q, k, v, k_pages, v_pages (None: k_pages is a 4-bit cache), block_table, seqlens, cu_seqlens,
// q_weight, k_weight, eps, positions, rope, interleaved, q_out.  Returns (q_out,).
PyObject *append(PyObject *, PyObject *const *a, Py_ssize_t n) {
    HANDLE_TH_ERRORS
    Reader r;
    const at::Tensor *k = n == 15 ? r.strided(a[1]) : nullptr;
    if (!k) Py_RETURN_NONE;
    const at::Tensor *v = r.strided(a[2]), *q = a[0] != Py_None ? r.strided(a[0]) : nullptr;
    const bool q4 = a[4] == Py_None;
    const at::Tensor *pool = r.dense(a[3], q4 ? U8 : BF16), *pool_v = q4 ? nullptr : r.dense(a[4], BF16);
    const at::Tensor *table = r.dense(a[5], I32), *lens = r.dense(a[6], I32);
    const at::Tensor *cu = a[7] != Py_None ? r.dense(a[7], I32) : nullptr;
    if (!r.ok || k->dim() != 3 || v->sizes() != k->sizes() || table->dim() != 2) Py_RETURN_NONE;
    const int64_t total = k->size(0), Hkv = k->size(1), d = k->size(2), B = lens->numel();
    const int64_t Hq = q ? q->size(1) : 0;
    if (q && (q->dim() != 3 || q->size(0) != total || q->size(2) != d)) Py_RETURN_NONE;
    if ((Hq > 1 && q->stride(1) != d) || (Hkv > 1 && (k->stride(1) != d || v->stride(1) != d))) Py_RETURN_NONE;
    int64_t page_size = 16;
    if (q4) {
        if (pool->dim() != 3 || pool->size(1) != Hkv || pool->size(2) != ATTN_Q4_BLOCK_BYTES) Py_RETURN_NONE;
    } else {
        if (pool->dim() != 4 || pool_v->sizes() != pool->sizes() || pool->size(2) != Hkv || pool->size(3) != 128)
            Py_RETURN_NONE;
        page_size = pool->size(1);
    }
    if (table->size(0) != B || (cu ? cu->numel() != B + 1 : total != B) || (!q && a[14] != Py_None)) Py_RETURN_NONE;
    Rotate rot;
    rot.read(r, a + 8, at::IntArrayRef(&total, 1));
    const int b = r.narrow(B), t = r.narrow(total), hq = r.narrow(Hq), hk = r.narrow(Hkv), dd = r.narrow(d);
    const int ps = r.narrow(page_size), np = r.narrow(pool->size(0)), mb = r.narrow(table->size(1));
    Output out;
    if (q) out.take(r, a[14], BF16, q->sizes(), *q);
    if (!r.ok) Py_RETURN_NONE;
    const auto stride = [&](const at::Tensor *x, int64_t heads) {
        return !x ? (size_t)0 : total > 1 ? (size_t)x->stride(0) : (size_t)(heads * d);
    };
    const auto *tab = static_cast<const int32_t *>(table->data_ptr()), *len = static_cast<const int32_t *>(lens->data_ptr());
    const auto *off = static_cast<const int32_t *>(at_of(cu));
    const attn_status_t st =
        q4 ? attn_append_paged_q4(at_of(q), k->data_ptr(), v->data_ptr(), out.ptr, pool->data_ptr(), tab, len, off, rot.wq,
                                  rot.wk, rot.eps, rot.positions, rot.n_axes, rot.rope, rot.rotary_dim, rot.interleaved, b,
                                  t, hq, hk, dd, ps, np, mb, stride(q, Hq), stride(k, Hkv), stride(v, Hkv), r.stream())
           : attn_append_paged(at_of(q), k->data_ptr(), v->data_ptr(), out.ptr, pool->data_ptr(), pool_v->data_ptr(), tab,
                               len, off, rot.wq, rot.wk, rot.eps, rot.positions, rot.n_axes, rot.rope, rot.rotary_dim,
                               rot.interleaved, b, t, hq, hk, dd, ps, np, mb, stride(q, Hq), stride(k, Hkv),
                               stride(v, Hkv), r.stream());
    if (st != ATTN_OK) Py_RETURN_NONE;
    PyObject *o = out.object();
    PyObject *one = o ? PyTuple_Pack(1, o) : nullptr;
    Py_XDECREF(o);
    return one;
    END_HANDLE_TH_ERRORS
}

// The cache and table of an operator that reads: cache, block_table, seqlens.
struct Cache {
    const at::Tensor *cache, *table, *lens;
    int64_t B = 0, Hkv = 0;

    Cache(Reader &r, PyObject *const *a)
        : cache(r.dense(a[0], U8)), table(r.dense(a[1], I32)), lens(r.dense(a[2], I32)) {
        r.ok = r.ok && cache->dim() == 3 && cache->size(2) == ATTN_Q4_BLOCK_BYTES && table->dim() == 2 &&
               table->size(0) == lens->numel();
        if (!r.ok) return;
        B = lens->numel();
        Hkv = cache->size(1);
    }
    const int32_t *tab() const { return static_cast<const int32_t *>(table->data_ptr()); }
    const int32_t *len() const { return static_cast<const int32_t *>(lens->data_ptr()); }
};

// cache, block_table, seqlens, cu_seqlens_k, total_k, k_out, v_out
PyObject *gather(PyObject *, PyObject *const *a, Py_ssize_t n) {
    HANDLE_TH_ERRORS
    Reader r;
    if (n != 7 || a[4] == Py_None) Py_RETURN_NONE;
    const Cache c(r, a);
    const at::Tensor *cu = r.ok ? r.dense(a[3], I32) : nullptr;
    const int64_t total = r.integer(a[4]);
    if (!r.ok || cu->numel() != c.B + 1) Py_RETURN_NONE;
    const int64_t sizes[3] = {total, c.Hkv, 128};
    Output k, v;
    k.take(r, a[5], BF16, sizes, *c.cache);
    v.take(r, a[6], BF16, sizes, *c.cache);
    const int b = r.narrow(c.B), h = r.narrow(c.Hkv), t = r.narrow(total), np = r.narrow(c.cache->size(0));
    const int mb = r.narrow(c.table->size(1));
    if (!r.ok || attn_gather_paged_q4(c.cache->data_ptr(), c.tab(), c.len(), static_cast<const int32_t *>(cu->data_ptr()),
                                      k.ptr, v.ptr, b, h, t, 128, 16, np, mb, r.stream()) != ATTN_OK)
        Py_RETURN_NONE;
    return pair(k, v);
    END_HANDLE_TH_ERRORS
}

// The queries, outputs and scale of an attention: q, scale, out, lse (False: none).
struct Attention {
    const at::Tensor *q;
    Output out, lse;
    float scale = 0.f;

    Attention(Reader &r, PyObject *const *a) : q(r.dense(a[0], BF16)) {
        r.ok = r.ok && q->dim() == 3;
        if (!r.ok) return;
        scale = a[1] == Py_None ? (float)(1.0 / std::sqrt((double)q->size(2))) : r.real(a[1]);
        out.take(r, a[2], BF16, q->sizes(), *q);
    }
    void lse_sizes(Reader &r, PyObject *o, int64_t rows, int64_t cols) {
        const int64_t sizes[2] = {rows, cols};
        if (r.ok && o != Py_False) lse.take(r, o, F32, sizes, *q);
    }
};

// q, scale, out, lse, cache, block_table, seqlens, workspace
PyObject *decode(PyObject *, PyObject *const *a, Py_ssize_t n) {
    HANDLE_TH_ERRORS
    Reader r;
    if (n != 8) Py_RETURN_NONE;
    Attention x(r, a);
    if (!r.ok) Py_RETURN_NONE;
    const Cache c(r, a + 4);
    if (!r.ok || x.q->size(0) != c.B) Py_RETURN_NONE;
    const int64_t Hq = x.q->size(1);
    x.lse_sizes(r, a[3], c.B, Hq);
    const int b = r.narrow(c.B), hq = r.narrow(Hq), h = r.narrow(c.Hkv), d = r.narrow(x.q->size(2));
    const int np = r.narrow(c.cache->size(0)), mb = r.narrow(c.table->size(1));
    if (!r.ok) Py_RETURN_NONE;
    Output ws;
    int64_t bytes = a[7] == Py_None ? std::max<int64_t>(1, (int64_t)attn_decode_q4_workspace_bytes(b, hq, h, d, mb)) : 0;
    if (a[7] != Py_None) {
        const at::Tensor *w = r.dense(a[7], U8);
        bytes = w ? w->numel() : 0;
        ws.ptr = at_of(w);
    } else {
        ws.take(r, a[7], U8, bytes, *c.cache);
    }
    if (!r.ok || attn_decode_paged_q4(x.q->data_ptr(), c.cache->data_ptr(), c.tab(), c.len(), x.out.ptr,
                                      static_cast<float *>(x.lse.ptr), b, hq, h, d, 16, np, mb, x.scale, ws.ptr,
                                      (size_t)bytes, r.stream()) != ATTN_OK)
        Py_RETURN_NONE;
    return pair(x.out, x.lse);
    END_HANDLE_TH_ERRORS
}

// q, scale, out, lse, cache, block_table, seqlens_k, workspace, cu_seqlens_q, max_seqlen_q, max_total_k, causal, rounding
PyObject *fwd(PyObject *, PyObject *const *a, Py_ssize_t n) {
    HANDLE_TH_ERRORS
    Reader r;
    if (n != 13 || a[9] == Py_None || a[10] == Py_None) Py_RETURN_NONE;
    Attention x(r, a);
    if (!r.ok) Py_RETURN_NONE;
    const Cache c(r, a + 4);
    const at::Tensor *cu = r.ok ? r.dense(a[8], I32) : nullptr;
    if (!r.ok || cu->numel() != c.B + 1) Py_RETURN_NONE;
    const int64_t total = x.q->size(0), Hq = x.q->size(1);
    x.lse_sizes(r, a[3], Hq, total);
    const int b = r.narrow(c.B), hq = r.narrow(Hq), h = r.narrow(c.Hkv), t = r.narrow(total), d = r.narrow(x.q->size(2));
    const int np = r.narrow(c.cache->size(0)), mb = r.narrow(c.table->size(1));
    const int longest = r.narrow(r.integer(a[9])), keys = r.narrow(r.integer(a[10]));
    const bool causal = r.truth(a[11]);
    const int rounding = r.narrow(r.integer(a[12]));
    if (!r.ok) Py_RETURN_NONE;
    Output ws;
    int64_t bytes = a[7] == Py_None ? std::max<int64_t>(1, (int64_t)attn_fwd_paged_q4_workspace_bytes(b, h, d, keys)) : 0;
    if (a[7] != Py_None) {
        const at::Tensor *w = r.dense(a[7], U8);
        bytes = w ? w->numel() : 0;
        ws.ptr = at_of(w);
    } else {
        ws.take(r, a[7], U8, bytes, *c.cache);
    }
    if (!r.ok || attn_fwd_paged_q4(x.q->data_ptr(), c.cache->data_ptr(), c.tab(), c.len(),
                                   static_cast<const int32_t *>(cu->data_ptr()), x.out.ptr,
                                   static_cast<float *>(x.lse.ptr), b, hq, h, t, longest, d, 16, np, mb, keys, causal,
                                   x.scale, rounding, ws.ptr, (size_t)bytes, r.stream()) != ATTN_OK)
        Py_RETURN_NONE;
    return pair(x.out, x.lse);
    END_HANDLE_TH_ERRORS
}

#define METHOD(name) {#name, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(name)), METH_FASTCALL, nullptr}
PyMethodDef methods[] = {METHOD(qk_norm_rope), METHOD(append), METHOD(gather), METHOD(decode), METHOD(fwd),
                         {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_quick", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__quick() { return PyModule_Create(&module); }
