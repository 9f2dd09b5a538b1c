// The plain calls of the cache and of the operators around its attention, from Python to the C entry points.
//
// A single token's kernels are done in a few microseconds, and a call's checks and buffers, step by step in Python, take
// three times as long.  What is here does them for the usual call: exact torch tensors on the current device, of the
// stated types, shapes and layouts, on the current stream, with results that the call makes.  Whatever differs returns
// None and is left to the functions of binding.py, which tell what is wrong or do what is unusual.
#include <Python.h>

#include <ATen/core/Tensor.h>
#include <ATen/ops/empty.h>
#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/Dtype.h>
#include <torch/csrc/autograd/python_variable.h>

#include "../../include/kda.h"

namespace {

decltype(&kda_add_rmsnorm) add_rmsnorm_fn;
decltype(&kda_kv4_append_rope) append_rope_fn;
decltype(&kda_kv4_bounds) bounds_fn;
decltype(&kda_kv4_pick) pick_fn;
decltype(&kda_kv4_attention_picked) attention_picked_fn;
decltype(&kda_kv4_append) append_fn;
decltype(&kda_kv4_gather) gather_fn;
decltype(&kda_kv4_attention) attention_fn;

// What the arguments of one call were found to be; `good` goes false at the first that is not plain.
struct Call {
    bool good = true;
    int dev = -1;

    const at::Tensor *exact(PyObject *o) {
        if (!good || !THPVariable_CheckExact(o)) {
            good = false;
            return nullptr;
        }
        return &THPVariable_Unpack(o);
    }
    // the operand that sets the device
    const at::Tensor *first(PyObject *o, int dims) {
        const at::Tensor *t = exact(o);
        if (!t) return nullptr;
        good = t->is_cuda() && t->layout() == at::kStrided && t->dim() == dims;
        if (!good) return nullptr;
        dev = t->get_device();
        good = dev == (int)c10::cuda::current_device();
        return good ? t : nullptr;
    }
    const at::Tensor *like(PyObject *o, at::ScalarType type, at::IntArrayRef shape) {
        const at::Tensor *t = exact(o);
        if (!t) return nullptr;
        good = t->is_cuda() && t->layout() == at::kStrided && t->get_device() == dev && t->scalar_type() == type && t->sizes() == shape;
        return good ? t : nullptr;
    }
    // its address; dense
    void *at(PyObject *o, at::ScalarType type, at::IntArrayRef shape) {
        const at::Tensor *t = like(o, type, shape);
        if (!t) return nullptr;
        good = t->is_contiguous();
        return good ? t->data_ptr() : nullptr;
    }
    // rows of one or two dense dimensions behind a strided one: address and stride
    void *rows(const at::Tensor *t, long long &stride) {
        if (!t) return nullptr;
        const auto sizes = t->sizes(), strides = t->strides();
        const int n = (int)sizes.size();
        long long row = 1;
        for (int i = n - 1; i > 0; --i) {
            if (strides[i] != row && (i == n - 1 || sizes[i] > 1)) good = false;
            row *= sizes[i];
        }
        stride = sizes[0] <= 1 ? row : strides[0];
        void *p = t->data_ptr();
        if (stride < row || stride * (long long)t->element_size() % 16 != 0 || (uintptr_t)p % 16 != 0) good = false;
        return p;
    }
    int integer(PyObject *o) {
        int overflow = 0;
        const long long x = PyLong_Check(o) ? PyLong_AsLongLongAndOverflow(o, &overflow) : 0;
        if (!PyLong_Check(o) || overflow || x < INT_MIN || x > INT_MAX) good = false;
        return (int)x;
    }
    double number(PyObject *o) {
        const double x = PyFloat_Check(o) ? PyFloat_AS_DOUBLE(o) : PyLong_Check(o) ? PyLong_AsDouble(o) : 0.0;
        if (PyErr_Occurred()) PyErr_Clear(), good = false;
        if (!PyFloat_Check(o) && !PyLong_Check(o)) good = false;
        return x;
    }
    int32_t *error(PyObject *o) {
        if (o == Py_None) return nullptr;
        const at::Tensor *t = exact(o);
        if (!t) return nullptr;
        good = t->is_cuda() && t->get_device() == dev && t->scalar_type() == at::kInt && t->is_contiguous() && t->numel() >= 1;
        return good ? t->data_ptr<int32_t>() : nullptr;
    }
    at::Tensor make(at::IntArrayRef shape, at::ScalarType type) const {
        return at::empty(shape, at::TensorOptions().dtype(type).device(at::kCUDA, dev));
    }
    void *stream() const { return (void *)c10::cuda::getCurrentCUDAStream((c10::DeviceIndex)dev).stream(); }
};

int kv_type(at::ScalarType t) { return t == at::kBFloat16 ? KDA_DTYPE_BF16 : t == at::kHalf ? KDA_DTYPE_FP16 : -1; }

// pool uint8 [pages][H][P / 16][18 D]
struct Pool {
    void *p = nullptr;
    int pages = 0, heads = 0, page_size = 0;
};
Pool pool_of(Call &c, PyObject *o, int64_t D) {
    Pool r;
    const at::Tensor *t = c.exact(o);
    if (!t) return r;
    c.good = t->is_cuda() && t->get_device() == c.dev && t->scalar_type() == at::kByte && t->dim() == 4 && t->size(3) == 18 * D &&
             t->is_contiguous();
    if (!c.good) return r;
    r.p = t->data_ptr(), r.pages = (int)t->size(0), r.heads = (int)t->size(1), r.page_size = (int)t->size(2) * 16;
    return r;
}
// page table int32 [B][M]
struct Table {
    int32_t *p = nullptr;
    int64_t B = 0, M = 0;
};
Table table_of(Call &c, PyObject *o) {
    Table r;
    const at::Tensor *t = c.exact(o);
    if (!t) return r;
    c.good = t->is_cuda() && t->get_device() == c.dev && t->scalar_type() == at::kInt && t->dim() == 2 && t->is_contiguous() &&
             t->size(0) <= INT_MAX && t->size(1) <= INT_MAX;
    if (c.good) r.p = t->data_ptr<int32_t>(), r.B = t->size(0), r.M = t->size(1);
    return r;
}

PyObject *none() { Py_RETURN_NONE; }
// Results are made and the library is called without the interpreter's lock, as a launch may wait for room in its stream's
// queue, and what makes room may wait for the lock.  No Python object is touched meanwhile.
struct Unlocked {
    PyThreadState *const state = PyEval_SaveThread();
    ~Unlocked() { PyEval_RestoreThread(state); }
};
// None instead of an exception: the functions of binding.py take over
template <typename F>
PyObject *plain(const F &f) {
    try {
        return f();
    } catch (...) {
        return none();
    }
}

// (x, residual or None, weight, eps, mode, residual_out or None)
PyObject *add_rmsnorm(PyObject *, PyObject *const *a, Py_ssize_t n) {
    if (n != 6) return none();
    return plain([&]() -> PyObject * {
        Call c;
        const at::Tensor *x = c.first(a[0], 2);
        if (!x) return none();
        const auto type = x->scalar_type();
        const int dt = type == at::kFloat ? KDA_DTYPE_FP32 : kv_type(type), mode = c.integer(a[4]);
        const int64_t T = x->size(0), C = x->size(1);
        if (dt < 0 || C < 1 || T > INT_MAX || C > INT_MAX || mode < KDA_NORM_TYPE || mode > KDA_NORM_E4M3_BLOCK) return none();
        long long xs, rs = 0, hs = 0;
        void *xp = c.rows(x, xs), *wp = c.at(a[2], type, {C}), *rp = nullptr, *hp = nullptr;
        const double eps = c.number(a[3]);
        const bool adds = a[1] != Py_None;
        if (adds) rp = c.rows(c.like(a[1], type, {T, C}), rs);
        const at::Tensor *given = nullptr;
        if (a[5] != Py_None) given = c.like(a[5], type, {T, C}), hp = c.rows(given, hs);
        if (!c.good || (given && !adds)) return none();
        at::Tensor h, out, scales;
        int status;
        {
            const Unlocked u;
            if (adds && !given) h = c.make({T, C}, type), hp = h.data_ptr(), hs = C;
            out = c.make({T, C}, mode == KDA_NORM_TYPE ? type : at::kFloat8_e4m3fn);
            if (mode == KDA_NORM_E4M3_ROW) scales = c.make({T}, at::kFloat);
            if (mode == KDA_NORM_E4M3_BLOCK) scales = c.make({T, (C + 127) / 128}, at::kFloat);
            status = add_rmsnorm_fn((kda_dtype)dt, (int)T, (int)C, xp, xs, rp, rs, wp, (float)eps, (kda_norm_out)mode, hp, hs, out.data_ptr(),
                                    scales.defined() ? scales.data_ptr<float>() : nullptr, c.stream());
        }
        if (status != KDA_OK) return none();
        PyObject *s = scales.defined() ? THPVariable_Wrap(scales) : Py_NewRef(Py_None);
        PyObject *kept = given ? Py_NewRef(a[5]) : adds ? THPVariable_Wrap(h) : Py_NewRef(a[0]);
        return Py_BuildValue("NNN", THPVariable_Wrap(out), s, kept);
    });
}

// (q, k, v, rope, cu_seqlens, start, page_table, pool, pairs, k_scale, v_scale, q_out or None, dev_err or None)
PyObject *append_rope(PyObject *, PyObject *const *a, Py_ssize_t n) {
    if (n != 13) return none();
    return plain([&]() -> PyObject * {
        Call c;
        const at::Tensor *q = c.first(a[0], 3);
        if (!q) return none();
        const auto type = q->scalar_type();
        const int64_t T = q->size(0), Hq = q->size(1), D = q->size(2);
        const Pool pool = pool_of(c, a[7], D);
        const Table table = table_of(c, a[6]);
        const at::Tensor *rope = c.exact(a[3]);
        if (!c.good || kv_type(type) < 0 || rope->dim() != 2) return none();
        const int64_t H = pool.heads, positions = rope->size(0), R = rope->size(1);
        long long qs, ks, vs, os = Hq * D;
        void *qp = c.rows(q, qs), *kp = c.rows(c.like(a[1], type, {T, H, D}), ks), *vp = c.rows(c.like(a[2], type, {T, H, D}), vs);
        void *rp = c.at(a[3], at::kFloat, {positions, R}), *cp = c.at(a[4], at::kInt, {table.B + 1}), *sp = c.at(a[5], at::kInt, {table.B});
        const at::Tensor *given = nullptr;
        void *op = nullptr;
        if (a[11] != Py_None) given = c.like(a[11], type, {T, Hq, D}), op = c.rows(given, os);
        const double k_scale = c.number(a[9]), v_scale = c.number(a[10]);
        int32_t *err = c.error(a[12]);
        const int pairs = PyObject_IsTrue(a[8]);
        if (!c.good || pairs < 0 || T > INT_MAX || positions > INT_MAX || R > INT_MAX) {
            PyErr_Clear();
            return none();
        }
        at::Tensor out;
        int status;
        {
            const Unlocked u;
            if (!given) out = c.make({T, Hq, D}, type), op = out.data_ptr();
            status = append_rope_fn((kda_dtype)kv_type(type), (int)table.B, (int)T, (int)Hq, (int)H, (int)D, (int)R, pairs, qp, qs, kp, ks, vp,
                                    vs, (const float *)rp, (int)positions, (const int32_t *)cp, (const int32_t *)sp, table.p, (int)table.M,
                                    pool.page_size, pool.p, pool.pages, (float)k_scale, (float)v_scale, op, os, err, c.stream());
        }
        if (status != KDA_OK) return none();
        return given ? Py_NewRef(a[11]) : THPVariable_Wrap(out);
    });
}

// (cu_seqlens, start, total_tokens, page_table, pool, bounds, dev_err or None); True where it was done
PyObject *bounds(PyObject *, PyObject *const *a, Py_ssize_t n) {
    if (n != 7) return none();
    return plain([&]() -> PyObject * {
        Call c;
        const at::Tensor *p = c.first(a[4], 4);
        if (!p) return none();
        const int64_t D = p->size(3) / 18;
        const Pool pool = pool_of(c, a[4], D);
        const Table table = table_of(c, a[3]);
        const int T = c.integer(a[2]);
        if (!c.good) return none();
        void *bp = c.at(a[5], at::kChar, {pool.pages, pool.heads, 2 * D + 16}), *cp = c.at(a[0], at::kInt, {table.B + 1});
        void *sp = c.at(a[1], at::kInt, {table.B});
        int32_t *err = c.error(a[6]);
        if (!c.good) return none();
        int status;
        {
            const Unlocked u;
            status = bounds_fn((int)table.B, T, pool.heads, (int)D, (const int32_t *)cp, (const int32_t *)sp, table.p, (int)table.M,
                               pool.page_size, pool.p, pool.pages, (int8_t *)bp, err, c.stream());
        }
        if (status != KDA_OK) return none();
        Py_RETURN_TRUE;
    });
}

// (q, cu_seqlens, max_q, kv_lens, page_table, bounds, page_size, count, first, recent, workspace, dev_err or None)
PyObject *pick(PyObject *, PyObject *const *a, Py_ssize_t n) {
    if (n != 12) return none();
    return plain([&]() -> PyObject * {
        Call c;
        const at::Tensor *q = c.first(a[0], 3);
        if (!q) return none();
        const auto type = q->scalar_type();
        const int64_t T = q->size(0), Hq = q->size(1), D = q->size(2);
        const Table table = table_of(c, a[4]);
        const at::Tensor *b = c.exact(a[5]), *w = c.exact(a[10]);
        if (!c.good || kv_type(type) < 0 || b->dim() != 3 || w->dim() != 1) return none();
        const int64_t pages = b->size(0), H = b->size(1), wb = w->size(0);
        long long qs;
        void *qp = c.rows(q, qs), *bp = c.at(a[5], at::kChar, {pages, H, 2 * D + 16}), *wp = c.at(a[10], at::kByte, {wb});
        void *cp = c.at(a[1], at::kInt, {table.B + 1}), *lp = c.at(a[3], at::kInt, {table.B});
        const int max_q = c.integer(a[2]), page = c.integer(a[6]), count = c.integer(a[7]), first = c.integer(a[8]), recent = c.integer(a[9]);
        int32_t *err = c.error(a[11]);
        if (!c.good || count < 1 || T > INT_MAX) return none();
        at::Tensor out;
        int status;
        {
            const Unlocked u;
            out = c.make({T, H, count}, at::kInt);
            status = pick_fn((kda_dtype)kv_type(type), (int)table.B, (int)T, max_q, (int)Hq, (int)H, (int)D, qp, qs, (const int32_t *)cp,
                             (const int32_t *)lp, table.p, (int)table.M, page, (const int8_t *)bp, (int)pages, count, first, recent,
                             out.data_ptr<int32_t>(), wp, (size_t)wb, err, c.stream());
        }
        if (status != KDA_OK) return none();
        return THPVariable_Wrap(out);
    });
}

// (q, cu_seqlens, max_q, kv_lens, page_table, picked, pool, scale or None, k_scale, v_scale, workspace, dev_err or None)
PyObject *attention_picked(PyObject *, PyObject *const *a, Py_ssize_t n) {
    if (n != 12) return none();
    return plain([&]() -> PyObject * {
        Call c;
        const at::Tensor *q = c.first(a[0], 3);
        if (!q) return none();
        const auto type = q->scalar_type();
        const int64_t T = q->size(0), Hq = q->size(1), D = q->size(2);
        const Pool pool = pool_of(c, a[6], D);
        const Table table = table_of(c, a[4]);
        const at::Tensor *p = c.exact(a[5]), *w = c.exact(a[10]);
        if (!c.good || kv_type(type) < 0 || p->dim() != 3 || w->dim() != 1) return none();
        const int64_t count = p->size(2), wb = w->size(0);
        long long qs;
        void *qp = c.rows(q, qs), *pp = c.at(a[5], at::kInt, {T, pool.heads, count}), *wp = c.at(a[10], at::kByte, {wb});
        void *cp = c.at(a[1], at::kInt, {table.B + 1}), *lp = c.at(a[3], at::kInt, {table.B});
        const int max_q = c.integer(a[2]);
        const double scale = a[7] == Py_None ? 1.0 / std::sqrt((double)D) : c.number(a[7]), k_scale = c.number(a[8]), v_scale = c.number(a[9]);
        int32_t *err = c.error(a[11]);
        if (!c.good || T > INT_MAX || count > INT_MAX) return none();
        at::Tensor o, lse;
        int status;
        {
            const Unlocked u;
            o = c.make({T, Hq, D}, type), lse = c.make({T, Hq}, at::kFloat);
            status = attention_picked_fn((kda_dtype)kv_type(type), (int)table.B, (int)T, max_q, (int)Hq, pool.heads, (int)D, qp, qs,
                                         (const int32_t *)cp, (const int32_t *)lp, table.p, (int)table.M, pool.page_size, (const int32_t *)pp,
                                         (int)count, pool.p, pool.pages, (float)scale, (float)k_scale, (float)v_scale, o.data_ptr(),
                                         lse.data_ptr<float>(), wp, (size_t)wb, err, c.stream());
        }
        if (status != KDA_OK) return none();
        return Py_BuildValue("NN", THPVariable_Wrap(o), THPVariable_Wrap(lse));
    });
}

// (k, v, cu_seqlens, start, page_table, pool, k_scale, v_scale, dev_err or None); True where it was done
PyObject *append(PyObject *, PyObject *const *a, Py_ssize_t n) {
    if (n != 9) return none();
    return plain([&]() -> PyObject * {
        Call c;
        const at::Tensor *k = c.first(a[0], 3);
        if (!k) return none();
        const auto type = k->scalar_type();
        const int64_t T = k->size(0), H = k->size(1), D = k->size(2);
        const Pool pool = pool_of(c, a[5], D);
        const Table table = table_of(c, a[4]);
        if (!c.good || kv_type(type) < 0 || pool.heads != H || T > INT_MAX) return none();
        long long ks, vs;
        void *kp = c.rows(k, ks), *vp = c.rows(c.like(a[1], type, {T, H, D}), vs);
        void *cp = c.at(a[2], at::kInt, {table.B + 1}), *sp = c.at(a[3], at::kInt, {table.B});
        const double k_scale = c.number(a[6]), v_scale = c.number(a[7]);
        int32_t *err = c.error(a[8]);
        if (!c.good) return none();
        int status;
        {
            const Unlocked u;
            status = append_fn((kda_dtype)kv_type(type), (int)table.B, (int)T, (int)H, (int)D, kp, ks, vp, vs, (const int32_t *)cp,
                               (const int32_t *)sp, table.p, (int)table.M, pool.page_size, pool.p, pool.pages, (float)k_scale, (float)v_scale,
                               err, c.stream());
        }
        if (status != KDA_OK) return none();
        Py_RETURN_TRUE;
    });
}

// (cu_seqlens, start, total_tokens, page_table, pool, dtype, k_scale, v_scale, dev_err or None)
PyObject *gather(PyObject *, PyObject *const *a, Py_ssize_t n) {
    if (n != 9) return none();
    return plain([&]() -> PyObject * {
        Call c;
        const at::Tensor *p = c.first(a[4], 4);
        if (!p || !THPDtype_Check(a[5])) return none();
        const auto type = ((THPDtype *)a[5])->scalar_type;
        const int64_t D = p->size(3) / 18;
        const Pool pool = pool_of(c, a[4], D);
        const Table table = table_of(c, a[3]);
        const int T = c.integer(a[2]);
        void *cp = c.at(a[0], at::kInt, {table.B + 1}), *sp = c.at(a[1], at::kInt, {table.B});
        const double k_scale = c.number(a[6]), v_scale = c.number(a[7]);
        int32_t *err = c.error(a[8]);
        if (!c.good || kv_type(type) < 0 || T < 0) return none();
        at::Tensor k, v;
        int status;
        {
            const Unlocked u;
            k = c.make({T, pool.heads, D}, type), v = c.make({T, pool.heads, D}, type);
            status = gather_fn((kda_dtype)kv_type(type), (int)table.B, T, pool.heads, (int)D, k.data_ptr(), v.data_ptr(), (const int32_t *)cp,
                               (const int32_t *)sp, table.p, (int)table.M, pool.page_size, pool.p, pool.pages, (float)k_scale, (float)v_scale,
                               err, c.stream());
        }
        if (status != KDA_OK) return none();
        return Py_BuildValue("NN", THPVariable_Wrap(k), THPVariable_Wrap(v));
    });
}

// (q, cu_seqlens, max_q, kv_lens, page_table, pool, scale or None, window, k_scale, v_scale, workspace, dev_err or None)
PyObject *attention(PyObject *, PyObject *const *a, Py_ssize_t n) {
    if (n != 12) return none();
    return plain([&]() -> PyObject * {
        Call c;
        const at::Tensor *q = c.first(a[0], 3);
        if (!q) return none();
        const auto type = q->scalar_type();
        const int64_t T = q->size(0), Hq = q->size(1), D = q->size(2);
        const Pool pool = pool_of(c, a[5], D);
        const Table table = table_of(c, a[4]);
        const at::Tensor *w = c.exact(a[10]);
        if (!c.good || kv_type(type) < 0 || w->dim() != 1) return none();
        const int64_t wb = w->size(0);
        long long qs;
        void *qp = c.rows(q, qs), *wp = c.at(a[10], at::kByte, {wb});
        void *cp = c.at(a[1], at::kInt, {table.B + 1}), *lp = c.at(a[3], at::kInt, {table.B});
        const int max_q = c.integer(a[2]), window = c.integer(a[7]);
        const double scale = a[6] == Py_None ? 1.0 / std::sqrt((double)D) : c.number(a[6]), k_scale = c.number(a[8]), v_scale = c.number(a[9]);
        int32_t *err = c.error(a[11]);
        if (!c.good || T > INT_MAX) return none();
        at::Tensor o, lse;
        int status;
        {
            const Unlocked u;
            o = c.make({T, Hq, D}, type), lse = c.make({T, Hq}, at::kFloat);
            status = attention_fn((kda_dtype)kv_type(type), (int)table.B, (int)T, max_q, (int)Hq, pool.heads, (int)D, qp, qs,
                                  (const int32_t *)cp, (const int32_t *)lp, table.p, (int)table.M, pool.page_size, pool.p, pool.pages, window,
                                  (float)scale, (float)k_scale, (float)v_scale, o.data_ptr(), lse.data_ptr<float>(), wp, (size_t)wb, err,
                                  c.stream());
        }
        if (status != KDA_OK) return none();
        return Py_BuildValue("NN", THPVariable_Wrap(o), THPVariable_Wrap(lse));
    });
}

// bind(addresses of the eight entry points, in this order)
PyObject *bind(PyObject *, PyObject *const *a, Py_ssize_t n) {
    if (n != 8) {
        PyErr_SetString(PyExc_TypeError, "eight addresses");
        return nullptr;
    }
    void *p[8];
    for (int i = 0; i < 8; ++i) {
        p[i] = PyLong_AsVoidPtr(a[i]);
        if (!p[i]) {
            if (!PyErr_Occurred()) PyErr_SetString(PyExc_ValueError, "no address");
            return nullptr;
        }
    }
    add_rmsnorm_fn = (decltype(add_rmsnorm_fn))p[0];
    append_rope_fn = (decltype(append_rope_fn))p[1];
    bounds_fn = (decltype(bounds_fn))p[2];
    pick_fn = (decltype(pick_fn))p[3];
    attention_picked_fn = (decltype(attention_picked_fn))p[4];
    append_fn = (decltype(append_fn))p[5];
    gather_fn = (decltype(gather_fn))p[6];
    attention_fn = (decltype(attention_fn))p[7];
    Py_RETURN_NONE;
}

#define FAST(name) {#name, (PyCFunction)(void (*)(void))name, METH_FASTCALL, nullptr}
PyMethodDef methods[] = {FAST(add_rmsnorm), FAST(append_rope), FAST(bounds), FAST(pick), FAST(attention_picked), FAST(append),
                         FAST(gather), FAST(attention), FAST(bind),
                         {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_quick", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__quick(void) { return PyModule_Create(&module); }
