// The short way from Python to nine calls of libpkv: a CPython module that checks
// the torch tensors of a call and passes their pointers on, as the ctypes functions
// of the binding do, in a tenth of the time (a decode step of a few rows runs for 6 us
// on the GPU; its checks take 4 us in Python and 0.4 us here).
//
// Every function returns the C entry's code, or None when anything about its
// arguments is not as it should be; the binding then takes its own way, which says what is
// wrong.  Nothing is computed here, and the module knows libpkv by the addresses that
// the binding gives it (bind), so the library itself does not depend on torch.
#define PY_SSIZE_T_CLEAN
#include <Python.h>

#include <ATen/core/Tensor.h>
#include <torch/csrc/autograd/python_variable.h>

#include <stdint.h>

namespace {

using Decode = int (*)(void*, const void*, const void*, const void*, const void*, const void*, const int32_t*,
                       const int32_t*, int, int, void*, void*, size_t, void*);
using Append = int (*)(void*, const void*, const void*, const void*, const int32_t*, const int32_t*, const int32_t*,
                       int, int, int, void*);
using Read = int (*)(void*, const int32_t*, const int32_t*, const int32_t*, int, int, int, void*, void*, int64_t, int64_t,
                     void*);
using NormRope = int (*)(void*, const void*, const void*, const void*, const void*, const int32_t*, int, int, int,
                         int64_t, int64_t, void*, void*, int64_t, int64_t, void*);
using Quantize = int (*)(void*, const void*, int64_t, int, int, int, void*, void*, void*);
using MxRead = int (*)(void*, int, const void*, const void*, int, int, void*, int64_t, void*);
using AddNorm = int (*)(void*, const void*, int64_t, const void*, void*, const void*, int, int, int, void*, void*, void*);
using MxLinear = int (*)(void*, int, const void*, const void*, const void*, const void*, void*, int, int, int, void*);
using MxQkv = int (*)(void*, int, const void*, const void*, const void*, const void*, int, int, void*, void*, void*, void*);
Decode g_decode;
Append g_append;
Read g_read;
NormRope g_norm_rope;
Quantize g_quantize;
MxRead g_mx_read;
AddNorm g_add_norm;
MxLinear g_mx_linear;
MxQkv g_mx_qkv;

struct Bad {};  // an argument that the binding's own checks shall see

void need(bool ok)
{
    if (!ok) throw Bad();
}

long long number(PyObject* o)
{
    need(PyLong_Check(o));
    const long long v = PyLong_AsLongLong(o);
    if (v == -1 && PyErr_Occurred()) throw Bad();
    return v;
}

void* address(PyObject* o)
{
    need(PyLong_Check(o));
    void* p = PyLong_AsVoidPtr(o);
    if (!p && PyErr_Occurred()) throw Bad();
    return p;
}

// What a pool's calls have in common: its handle and (device, heads, kv_heads, head_dim).
struct Pool {
    void* handle;
    int device;
    int64_t heads, kv_heads, dim;
    Pool(PyObject* h, PyObject* spec) : handle(address(h))
    {
        need(PyTuple_Check(spec) && PyTuple_GET_SIZE(spec) == 4);
        device = (int)number(PyTuple_GET_ITEM(spec, 0));
        heads = number(PyTuple_GET_ITEM(spec, 1));
        kv_heads = number(PyTuple_GET_ITEM(spec, 2));
        dim = number(PyTuple_GET_ITEM(spec, 3));
    }
    const at::Tensor& tensor(PyObject* o, at::ScalarType type) const
    {
        need(THPVariable_Check(o));
        const at::Tensor& t = THPVariable_Unpack(o);
        need(t.scalar_type() == type && t.is_cuda() && t.get_device() == device);
        return t;
    }
    // [n] int32, contiguous; n < 0: any
    const int32_t* ints(PyObject* o, int64_t n, int64_t* size = nullptr) const
    {
        const at::Tensor& t = tensor(o, at::kInt);
        need(t.dim() == 1 && t.is_contiguous() && (n < 0 || t.size(0) == n));
        if (size) *size = t.size(0);
        return static_cast<const int32_t*>(t.data_ptr());
    }
    // [tokens][h][dim], contiguous
    void* heads_of(PyObject* o, int64_t tokens, int64_t h) const
    {
        const at::Tensor& t = tensor(o, at::kBFloat16);
        need(t.dim() == 3 && t.size(0) == tokens && t.size(1) == h && t.size(2) == dim && t.is_contiguous());
        return t.data_ptr();
    }
    // the same with any token stride
    void* strided(PyObject* o, at::ScalarType type, int64_t tokens, int64_t h, int64_t* stride) const
    {
        const at::Tensor& t = tensor(o, type);
        need(t.dim() == 3 && t.size(0) == tokens && t.size(1) == h && t.size(2) == dim && t.stride(2) == 1 &&
             (h == 1 || t.stride(1) == dim));
        *stride = tokens > 1 ? t.stride(0) : h * dim;
        return t.data_ptr();
    }
    // [rows][cols] bf16, contiguous rows, any row stride (stride null: contiguous)
    void* matrix(PyObject* o, int64_t rows, int64_t cols, int64_t* stride) const
    {
        const at::Tensor& t = tensor(o, at::kBFloat16);
        need(t.dim() == 2 && t.size(0) == rows && t.size(1) == cols && (stride ? t.stride(1) == 1 : t.is_contiguous()));
        if (stride) *stride = rows > 1 ? t.stride(0) : cols;
        return t.data_ptr();
    }
    const void* weight(PyObject* o) const
    {
        const at::Tensor& t = tensor(o, at::kBFloat16);
        need(t.numel() == dim && t.is_contiguous());
        return t.data_ptr();
    }
    // a page table [rows][pages], or None with the two numbers
    const int32_t* table(PyObject* o, PyObject* rows_given, PyObject* pages_given, int64_t* rows, int64_t* pages) const
    {
        if (o == Py_None) {
            *rows = number(rows_given);
            *pages = number(pages_given);
            need(*rows > 0 && *rows <= INT32_MAX && *pages > 0 && *pages <= INT32_MAX);
            return nullptr;
        }
        const at::Tensor& t = tensor(o, at::kInt);
        need(t.dim() == 2 && t.is_contiguous());
        *rows = t.size(0);
        *pages = t.size(1);
        return static_cast<const int32_t*>(t.data_ptr());
    }
};

// Runs a call's checks and the call; None for whatever the checks do not like.
template <class F>
PyObject* checked(F f)
{
    int rc;
    try {
        rc = f();
    } catch (...) {
        PyErr_Clear();
        Py_RETURN_NONE;
    }
    return PyLong_FromLong(rc);
}

template <class F>
int without_gil(F f)
{
    int rc;
    Py_BEGIN_ALLOW_THREADS;
    rc = f();
    Py_END_ALLOW_THREADS;
    return rc;
}

// decode(handle, spec, q, k, v, q_norm_w, k_norm_w, positions, table, pages, out, workspace, bytes, stream)
PyObject* decode(PyObject*, PyObject* const* a, Py_ssize_t n)
{
    return checked([&] {
        need(n == 14 && g_decode);
        const Pool p(a[0], a[1]);
        int64_t rows, table_rows, pages;
        const int32_t* positions = p.ints(a[7], -1, &rows);
        void *q = p.heads_of(a[2], rows, p.heads), *k = p.heads_of(a[3], rows, p.kv_heads),
             *v = p.heads_of(a[4], rows, p.kv_heads), *out = p.heads_of(a[10], rows, p.heads);
        const void *qw = p.weight(a[5]), *kw = p.weight(a[6]);
        const int32_t* table = nullptr;
        if (a[8] == Py_None) {
            pages = number(a[9]);
            need(pages > 0 && pages <= INT32_MAX);
        } else {
            table = p.table(a[8], nullptr, nullptr, &table_rows, &pages);
            need(table_rows == rows);
        }
        need(rows <= INT32_MAX);
        void *ws = address(a[11]), *stream = address(a[13]);
        const size_t bytes = (size_t)number(a[12]);
        return without_gil([&] {
            return g_decode(p.handle, q, k, v, qw, kw, positions, table, (int)rows, (int)pages, out, ws, bytes, stream);
        });
    });
}

// append(handle, spec, k, v, k_norm_w, positions, prow, table, rows, pages, stream)
PyObject* append(PyObject*, PyObject* const* a, Py_ssize_t n)
{
    return checked([&] {
        need(n == 11 && g_append);
        const Pool p(a[0], a[1]);
        int64_t tokens, rows, pages;
        const int32_t* positions = p.ints(a[5], -1, &tokens);
        void *k = p.heads_of(a[2], tokens, p.kv_heads), *v = p.heads_of(a[3], tokens, p.kv_heads);
        const void* kw = p.weight(a[4]);
        const int32_t* prow = a[6] == Py_None ? nullptr : p.ints(a[6], tokens);
        const int32_t* table = p.table(a[7], a[8], a[9], &rows, &pages);
        need(tokens <= INT32_MAX);
        void* stream = address(a[10]);
        return without_gil([&] {
            return g_append(p.handle, k, v, kw, positions, prow, table, (int)tokens, (int)rows, (int)pages, stream);
        });
    });
}

// read(handle, spec, positions, prow, table, k, v, rows, pages, stream)
PyObject* read(PyObject*, PyObject* const* a, Py_ssize_t n)
{
    return checked([&] {
        need(n == 10 && g_read);
        const Pool p(a[0], a[1]);
        int64_t tokens, rows, pages;
        const int32_t* positions = p.ints(a[2], -1, &tokens);
        const int32_t* prow = a[3] == Py_None ? nullptr : p.ints(a[3], tokens);
        const int32_t* table = p.table(a[4], a[7], a[8], &rows, &pages);
        void* to[2];
        int64_t token_stride = 0, head_stride = 0;
        for (int i = 0; i < 2; ++i) {
            const at::Tensor& t = p.tensor(a[5 + i], at::kBFloat16);
            need(t.dim() == 3 && t.size(0) == tokens && t.size(1) == p.kv_heads && t.size(2) == p.dim && t.stride(2) == 1);
            need(i == 0 || (t.stride(0) == token_stride && t.stride(1) == head_stride));
            token_stride = t.stride(0);
            head_stride = t.stride(1);
            to[i] = t.data_ptr();
        }
        need(tokens <= INT32_MAX);
        void* stream = address(a[9]);
        return without_gil([&] {
            return g_read(p.handle, positions, prow, table, (int)tokens, (int)rows, (int)pages, to[0], to[1], token_stride,
                          head_stride, stream);
        });
    });
}

// norm_rope(handle, spec, q, k, q_norm_w, k_norm_w, positions, layout, q_out, k_out, stream)
PyObject* norm_rope(PyObject*, PyObject* const* a, Py_ssize_t n)
{
    return checked([&] {
        need(n == 11 && g_norm_rope);
        const Pool p(a[0], a[1]);
        int64_t tokens;
        const int32_t* positions = p.ints(a[6], -1, &tokens);
        PyObject* first_out = a[8] == Py_None ? a[9] : a[8];
        need(THPVariable_Check(first_out));
        const at::ScalarType kind = THPVariable_Unpack(first_out).scalar_type();
        need(kind == at::kBFloat16 || kind == at::kFloat);
        void *x[2] = {}, *y[2] = {};
        const void* w[2] = {};
        int64_t xs[2] = {}, ys[2] = {};
        for (int i = 0; i < 2; ++i) {
            const int64_t h = i ? p.kv_heads : p.heads;
            need((a[2 + i] == Py_None) == (a[8 + i] == Py_None));
            if (a[4 + i] != Py_None) w[i] = p.weight(a[4 + i]);
            if (a[2 + i] == Py_None) continue;
            x[i] = p.strided(a[2 + i], at::kBFloat16, tokens, h, &xs[i]);
            y[i] = p.strided(a[8 + i], kind, tokens, h, &ys[i]);
        }
        const int layout = (int)number(a[7]);
        need(tokens <= INT32_MAX);
        void* stream = address(a[10]);
        return without_gil([&] {
            return g_norm_rope(p.handle, x[0], x[1], w[0], w[1], positions, (int)tokens, layout, kind == at::kFloat, xs[0],
                               xs[1], y[0], y[1], ys[0], ys[1], stream);
        });
    });
}

// A microscaled tensor: (kind, rows, cols), its codes and its scales.
struct Mx {
    int kind;
    int64_t rows, cols;
    void *codes, *scales;
    Mx(const Pool& p, PyObject* spec, PyObject* c, PyObject* s)
    {
        need(PyTuple_Check(spec) && PyTuple_GET_SIZE(spec) == 3);
        kind = (int)number(PyTuple_GET_ITEM(spec, 0));
        rows = number(PyTuple_GET_ITEM(spec, 1));
        cols = number(PyTuple_GET_ITEM(spec, 2));
        need((kind == 2 || kind == 3) && rows > 0 && rows <= INT32_MAX && cols > 0 && cols <= INT32_MAX && cols % 128 == 0);
        codes = bytes(p, c, kind == 2 ? rows * cols : rows * (cols / 2));
        scales = bytes(p, s, (rows + 127) / 128 * (cols / 128) * 512);
    }
    static void* bytes(const Pool& p, PyObject* o, int64_t n)
    {
        const at::Tensor& t = p.tensor(o, at::kByte);
        need(t.numel() == n && t.is_contiguous());
        return t.data_ptr();
    }
};

// mx_quantize(handle, spec, x, mx, codes, scales, stream)
PyObject* mx_quantize(PyObject*, PyObject* const* a, Py_ssize_t n)
{
    return checked([&] {
        need(n == 7 && g_quantize);
        const Pool p(a[0], a[1]);
        const Mx m(p, a[3], a[4], a[5]);
        int64_t stride;
        void *x = p.matrix(a[2], m.rows, m.cols, &stride), *stream = address(a[6]);
        return without_gil([&] {
            return g_quantize(p.handle, x, stride, (int)m.rows, (int)m.cols, m.kind, m.codes, m.scales, stream);
        });
    });
}

// mx_read(handle, spec, mx, codes, scales, y, stream)
PyObject* mx_read(PyObject*, PyObject* const* a, Py_ssize_t n)
{
    return checked([&] {
        need(n == 7 && g_mx_read);
        const Pool p(a[0], a[1]);
        const Mx m(p, a[2], a[3], a[4]);
        int64_t stride;
        void *y = p.matrix(a[5], m.rows, m.cols, &stride), *stream = address(a[6]);
        return without_gil([&] {
            return g_mx_read(p.handle, m.kind, m.codes, m.scales, (int)m.rows, (int)m.cols, y, stride, stream);
        });
    });
}

// add_norm(handle, spec, x, residual, w, mx, out, scales, residual_out, stream); mx None: out is bf16
PyObject* add_norm(PyObject*, PyObject* const* a, Py_ssize_t n)
{
    return checked([&] {
        need(n == 10 && g_add_norm);
        const Pool p(a[0], a[1]);
        const at::Tensor& t = p.tensor(a[2], at::kBFloat16);
        need(t.dim() == 2 && t.size(0) <= INT32_MAX && t.size(1) <= INT32_MAX);
        const int64_t tokens = t.size(0), hidden = t.size(1);
        int64_t stride;
        const void* x = p.matrix(a[2], tokens, hidden, &stride);
        need((a[3] == Py_None) == (a[8] == Py_None));
        const void* residual = a[3] == Py_None ? nullptr : p.matrix(a[3], tokens, hidden, nullptr);
        void* residual_out = a[8] == Py_None ? nullptr : p.matrix(a[8], tokens, hidden, nullptr);
        const at::Tensor& w = p.tensor(a[4], at::kBFloat16);
        need(w.numel() == hidden && w.is_contiguous());
        int kind = 0;
        void *out, *scales = nullptr;
        if (a[5] == Py_None) {
            out = p.matrix(a[6], tokens, hidden, nullptr);
        } else {
            const Mx m(p, a[5], a[6], a[7]);
            need(m.rows == tokens && m.cols == hidden);
            kind = m.kind, out = m.codes, scales = m.scales;
        }
        const void* wp = w.data_ptr();
        void* stream = address(a[9]);
        return without_gil([&] {
            return g_add_norm(p.handle, x, stride, residual, residual_out, wp, (int)tokens, (int)hidden, kind, out, scales,
                              stream);
        });
    });
}

// mx_linear(handle, spec, x's mx, codes, scales, w's mx, codes, scales, y, stream)
PyObject* mx_linear(PyObject*, PyObject* const* a, Py_ssize_t n)
{
    return checked([&] {
        need(n == 10 && g_mx_linear);
        const Pool p(a[0], a[1]);
        const Mx x(p, a[2], a[3], a[4]), w(p, a[5], a[6], a[7]);
        need(x.kind == w.kind && x.cols == w.cols);
        void *y = p.matrix(a[8], x.rows, w.rows, nullptr), *stream = address(a[9]);
        return without_gil([&] {
            return g_mx_linear(p.handle, x.kind, x.codes, x.scales, w.codes, w.scales, y, (int)x.rows, (int)x.cols,
                               (int)w.rows, stream);
        });
    });
}

// mx_qkv_proj(handle, spec, x's mx, codes, scales, w's mx, codes, scales, q, k, v, stream)
PyObject* mx_qkv_proj(PyObject*, PyObject* const* a, Py_ssize_t n)
{
    return checked([&] {
        need(n == 12 && g_mx_qkv);
        const Pool p(a[0], a[1]);
        const Mx x(p, a[2], a[3], a[4]), w(p, a[5], a[6], a[7]);
        need(x.kind == w.kind && x.cols == w.cols && w.rows == (p.heads + 2 * p.kv_heads) * p.dim);
        void *q = p.heads_of(a[8], x.rows, p.heads), *k = p.heads_of(a[9], x.rows, p.kv_heads),
             *v = p.heads_of(a[10], x.rows, p.kv_heads), *stream = address(a[11]);
        return without_gil([&] {
            return g_mx_qkv(p.handle, x.kind, x.codes, x.scales, w.codes, w.scales, (int)x.rows, (int)x.cols, q, k, v, stream);
        });
    });
}

// bind(decode, append, read, norm_rope, mx_quantize, mx_read, add_norm, mx_linear, mx_qkv_proj): the addresses of
// libpkv's entries
PyObject* bind(PyObject*, PyObject* const* a, Py_ssize_t n)
{
    try {
        need(n == 9);
        g_decode = reinterpret_cast<Decode>(address(a[0]));
        g_append = reinterpret_cast<Append>(address(a[1]));
        g_read = reinterpret_cast<Read>(address(a[2]));
        g_norm_rope = reinterpret_cast<NormRope>(address(a[3]));
        g_quantize = reinterpret_cast<Quantize>(address(a[4]));
        g_mx_read = reinterpret_cast<MxRead>(address(a[5]));
        g_add_norm = reinterpret_cast<AddNorm>(address(a[6]));
        g_mx_linear = reinterpret_cast<MxLinear>(address(a[7]));
        g_mx_qkv = reinterpret_cast<MxQkv>(address(a[8]));
    } catch (const Bad&) {
        PyErr_Clear();
        PyErr_SetString(PyExc_TypeError, "bind takes nine addresses");
        return nullptr;
    }
    Py_RETURN_NONE;
}

template <PyObject* (*F)(PyObject*, PyObject* const*, Py_ssize_t)>
PyMethodDef method(const char* name)
{
    return {name, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(F)), METH_FASTCALL, nullptr};
}

PyMethodDef g_methods[] = {method<decode>("decode"), method<append>("append"),       method<read>("read"),
                           method<norm_rope>("norm_rope"), method<mx_quantize>("mx_quantize"), method<mx_read>("mx_read"),
                           method<add_norm>("add_norm"), method<mx_linear>("mx_linear"), method<mx_qkv_proj>("mx_qkv_proj"),
                           method<bind>("bind"), {nullptr, nullptr, 0, nullptr}};
PyModuleDef g_module = {PyModuleDef_HEAD_INIT, "_pkv_torch", nullptr, -1, g_methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__pkv_torch()
{
    PyObject* m = PyModule_Create(&g_module);
    if (m && PyModule_AddStringConstant(m, "torch_version", PKV_TORCH_VERSION) != 0) {
        Py_DECREF(m);
        return nullptr;
    }
    return m;
}
