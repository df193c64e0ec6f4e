// The short way from torch tensors to the C ABI for the calls of a decoding step
// (cp_rope without a plan, cp_kv4_write, cp_kv4_read, cp_attn_kv4).
//
// A step of a few tokens takes microseconds on the GPU, and marshalling its arguments
// in Python took 30 us a call.  Each function here takes the ordinary call (every
// tensor on the current device, nothing empty, its stream the current one), makes the
// same checks, allocates the outputs and launches: 5 to 8 us.  Whatever it
// does not take (another device, empty tensors, an argument to be refused) returns
// None before anything is launched, and the binding goes its own way, with its own errors.
#include <Python.h>

#include <cstdint>

#include <ATen/ATen.h>
#include <ATen/cuda/EmptyTensor.h>
#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/autograd/python_variable.h>

#include "cp_attn.h"

namespace {

decltype(&cp_rope) g_rope = nullptr;
decltype(&cp_kv4_write) g_write = nullptr;
decltype(&cp_kv4_read) g_read = nullptr;
decltype(&cp_attn_kv4) g_attn = nullptr;

using at::Tensor;

const Tensor* tensor(PyObject* o) { return THPVariable_Check(o) ? &THPVariable_Unpack(o) : nullptr; }

struct Where {
    int dev = -1;
    void* stream = nullptr;
    bool set(const Tensor& t)
    {
        if (!t.is_cuda()) return false;
        dev = c10::cuda::current_device();
        if (t.get_device() != dev) return false;
        stream = c10::cuda::getCurrentCUDAStream(static_cast<c10::DeviceIndex>(dev)).stream();
        return true;
    }
    bool here(const Tensor& t) const { return t.is_cuda() && t.get_device() == dev; }
    Tensor empty(at::IntArrayRef shape, at::ScalarType type) const
    {
        return at::detail::empty_cuda(shape, type, c10::Device(c10::kCUDA, static_cast<c10::DeviceIndex>(dev)),
                                      std::nullopt);
    }
};

// A bf16 [B, H, N, D] tensor whose rows are contiguous and start on 16 bytes, and its strides (0 for
// dimensions of one).
bool strided(const Tensor& t, const Where& w, int64_t* s)
{
    if (t.layout() != at::kStrided || t.dim() != 4 || t.scalar_type() != at::kBFloat16 || !w.here(t) || t.numel() == 0)
        return false;
    if (t.stride(3) != 1 && t.size(3) > 1) return false;
    for (int i = 0; i < 3; ++i) {
        s[i] = t.size(i) > 1 ? t.stride(i) : 0;
        if (s[i] % 8 != 0) return false;
    }
    return reinterpret_cast<uintptr_t>(t.data_ptr()) % 16 == 0;
}

bool exactly(const Tensor* t, at::ScalarType type, const Where& w, at::IntArrayRef shape)
{
    return t && t->layout() == at::kStrided && t->scalar_type() == type && w.here(*t) && t->sizes() == shape &&
           t->is_contiguous();
}

// None counts as given: *out = nullptr.
bool optional(PyObject* o, at::ScalarType type, const Where& w, at::IntArrayRef shape, const int32_t** out)
{
    *out = nullptr;
    if (o == Py_None) return true;
    const Tensor* t = tensor(o);
    if (!exactly(t, type, w, shape)) return false;
    *out = static_cast<const int32_t*>(t->data_ptr());
    return true;
}

bool integer(PyObject* o, int64_t* out)
{
    if (!PyLong_CheckExact(o)) return false;
    int over = 0;
    *out = PyLong_AsLongLongAndOverflow(o, &over);
    return over == 0 && *out >= -(int64_t(1) << 31) && *out < (int64_t(1) << 31);
}

bool cache(PyObject* pages, PyObject* table, int64_t head_dim, int64_t batch, Where& w, cp_kv4_cache_t* c)
{
    const Tensor *p = tensor(pages), *t = tensor(table);
    if (!p || !t || p->dim() != 3 || t->dim() != 2 || !w.set(*p)) return false;
    if (!exactly(p, at::kByte, w, p->sizes()) || p->numel() == 0) return false;
    if (!exactly(t, at::kInt, w, {batch, t->size(1)}) || t->numel() == 0) return false;
    if (head_dim != 64 && head_dim != 128 && head_dim != 256) return false;
    const int64_t block = 18 * head_dim, blocks = p->size(2) / block;
    if (p->size(2) % block != 0 || blocks < 1 || blocks > 4096) return false;
    if (p->size(0) > 0x7fffffff || p->size(1) > 0x7fffffff || t->size(1) > 0x7fffffff || batch > 0x7fffffff) return false;
    c->batch = static_cast<int32_t>(batch);
    c->num_kv_heads = static_cast<int32_t>(p->size(1));
    c->head_dim = static_cast<int32_t>(head_dim);
    c->page_size = static_cast<int32_t>(16 * blocks);
    c->num_pages = static_cast<int32_t>(p->size(0));
    c->table_width = static_cast<int32_t>(t->size(1));
    c->pages = p->data_ptr();
    c->block_table = static_cast<const int32_t*>(t->data_ptr());
    return reinterpret_cast<uintptr_t>(c->pages) % 16 == 0;
}

template <class F>
cp_status_t without_gil(F&& f)
{
    PyThreadState* s = PyEval_SaveThread();
    const cp_status_t st = f();
    PyEval_RestoreThread(s);
    return st;
}

// rope(tensors, inv_freq, positions, sections, adjacent, inverse, outs)
PyObject* rope(PyObject* const* a)
{
    if (!PyList_Check(a[0])) return nullptr;
    const Py_ssize_t n = PyList_GET_SIZE(a[0]);
    if (n < 1 || n > CP_ROPE_MAX_BUFS) return nullptr;
    const Tensor* x[CP_ROPE_MAX_BUFS];
    for (Py_ssize_t i = 0; i < n; ++i)
        if (!(x[i] = tensor(PyList_GET_ITEM(a[0], i)))) return nullptr;
    Where w;
    if (x[0]->dim() != 4 || !w.set(*x[0])) return nullptr;
    const int64_t B = x[0]->size(0), N = x[0]->size(2), D = x[0]->size(3);
    if (B > 0x7fffffff || N > 0x7fffffff || D > 256) return nullptr;
    int64_t strides[3 * CP_ROPE_MAX_BUFS];
    int32_t heads[CP_ROPE_MAX_BUFS];
    const void* in[CP_ROPE_MAX_BUFS];
    void* out[CP_ROPE_MAX_BUFS];
    for (Py_ssize_t i = 0; i < n; ++i) {
        if (!strided(*x[i], w, strides + 3 * i)) return nullptr;
        if (x[i]->size(0) != B || x[i]->size(2) != N || x[i]->size(3) != D || x[i]->size(1) > 0x7fffffff) return nullptr;
        heads[i] = static_cast<int32_t>(x[i]->size(1));
        in[i] = x[i]->data_ptr();
    }
    const Tensor* f = tensor(a[1]);
    if (!f || f->dim() != 1 || !exactly(f, at::kDouble, w, f->sizes())) return nullptr;
    const int64_t pairs = f->size(0);
    if (pairs < 8 || pairs % 8 != 0 || 2 * pairs > D) return nullptr;
    cp_rope_t r{};
    r.batch = static_cast<int32_t>(B);
    r.rows = static_cast<int32_t>(N);
    r.head_dim = static_cast<int32_t>(D);
    r.rotary_dim = static_cast<int32_t>(2 * pairs);
    r.layout = a[4] == Py_True ? CP_ROPE_ADJACENT : CP_ROPE_HALF;
    r.order = CP_ROPE_ROWS;
    r.inverse = a[5] == Py_True;
    r.inv_freq = static_cast<const double*>(f->data_ptr());
    r.n_axes = 1;
    if (a[2] != Py_None) {
        const Tensor* p = tensor(a[2]);
        if (!p || p->layout() != at::kStrided || p->scalar_type() != at::kInt || !w.here(*p)) return nullptr;
        const int64_t d = p->dim();
        if ((d != 2 && d != 3) || p->size(d - 1) != N || (d == 3 && p->size(0) != B) || p->numel() == 0) return nullptr;
        if ((p->stride(d - 1) != 1 && N > 1) || p->size(d - 2) > CP_ROPE_MAX_AXES) return nullptr;
        r.n_axes = static_cast<int32_t>(p->size(d - 2));
        r.pos_len = static_cast<int32_t>(N);
        r.pos_axis = p->stride(d - 2);
        r.pos_batch = d == 3 ? p->stride(0) : 0;
        r.positions = static_cast<const int32_t*>(p->data_ptr());
    }
    if (a[3] == Py_None) {
        if (r.n_axes != 1) return nullptr;
        r.sections[0] = static_cast<int32_t>(pairs);
    } else {
        const bool list = PyList_Check(a[3]);
        if (!list && !PyTuple_Check(a[3])) return nullptr;
        const Py_ssize_t k = list ? PyList_GET_SIZE(a[3]) : PyTuple_GET_SIZE(a[3]);
        if (k != r.n_axes) return nullptr;
        int64_t sum = 0;
        for (Py_ssize_t i = 0; i < k; ++i) {
            int64_t v;
            if (!integer(list ? PyList_GET_ITEM(a[3], i) : PyTuple_GET_ITEM(a[3], i), &v) || v < 0) return nullptr;
            sum += v;
            r.sections[i] = static_cast<int32_t>(v);
        }
        if (sum != pairs) return nullptr;
    }
    Tensor made[CP_ROPE_MAX_BUFS];
    if (a[6] == Py_None) {
        for (Py_ssize_t i = 0; i < n; ++i) {
            made[i] = w.empty(x[i]->sizes(), at::kBFloat16);
            out[i] = made[i].data_ptr();
        }
    } else {
        if (!PyList_Check(a[6]) || PyList_GET_SIZE(a[6]) != n) return nullptr;
        for (Py_ssize_t i = 0; i < n; ++i) {
            const Tensor* o = tensor(PyList_GET_ITEM(a[6], i));
            if (!exactly(o, at::kBFloat16, w, x[i]->sizes())) return nullptr;
            out[i] = o->data_ptr();
        }
    }
    if (without_gil([&] { return g_rope(&r, nullptr, nullptr, static_cast<int32_t>(n), in, out, heads, strides, w.stream); }) !=
        CP_OK)
        return nullptr;
    if (a[6] != Py_None) return Py_NewRef(a[6]);
    PyObject* list = PyList_New(n);
    if (!list) return nullptr;
    for (Py_ssize_t i = 0; i < n; ++i) PyList_SET_ITEM(list, i, THPVariable_Wrap(std::move(made[i])));
    return list;
}

// kv4_write(pages, block_table, start, k, v, counts, rows)
PyObject* kv4_write(PyObject* const* a)
{
    const Tensor *k = tensor(a[3]), *v = tensor(a[4]);
    if (!k || !v || k->dim() != 4 || k->sizes() != v->sizes()) return nullptr;
    Where w;
    cp_kv4_cache_t c;
    const int64_t B = k->size(0), N = k->size(2);
    if (!cache(a[0], a[1], k->size(3), B, w, &c) || k->size(1) != c.num_kv_heads || N > 0x7fffffff) return nullptr;
    int64_t ks[3], vs[3];
    const int32_t *start, *counts, *rows;
    if (!strided(*k, w, ks) || !strided(*v, w, vs)) return nullptr;
    int64_t T = N;
    if (a[6] != Py_None) {
        const Tensor* r = tensor(a[6]);
        if (!r || r->dim() != 1 || r->numel() == 0 || r->numel() > 0x7fffffff) return nullptr;
        T = r->size(0);
    }
    if (a[2] == Py_None || !optional(a[2], at::kInt, w, {B}, &start) || !optional(a[5], at::kInt, w, {B}, &counts) ||
        !optional(a[6], at::kInt, w, {T}, &rows))
        return nullptr;
    if (without_gil([&] {
            return g_write(&c, static_cast<int32_t>(T), start, counts, rows, static_cast<int32_t>(N), k->data_ptr(), ks,
                           v->data_ptr(), vs, w.stream);
        }) != CP_OK)
        return nullptr;
    return Py_NewRef(Py_True);
}

// kv4_read(pages, block_table, start, tokens, head_dim, counts, rows, k, v)
PyObject* kv4_read(PyObject* const* a)
{
    const Tensor* table = tensor(a[1]);
    int64_t T, D;
    if (!table || table->dim() != 2 || !integer(a[3], &T) || !integer(a[4], &D) || T < 1) return nullptr;
    Where w;
    cp_kv4_cache_t c;
    const int64_t B = table->size(0);
    if (!cache(a[0], a[1], D, B, w, &c)) return nullptr;
    const int32_t *start, *counts, *rows;
    if (a[2] == Py_None || !optional(a[2], at::kInt, w, {B}, &start) || !optional(a[5], at::kInt, w, {B}, &counts) ||
        !optional(a[6], at::kInt, w, {T}, &rows))
        return nullptr;
    int64_t N = T;
    Tensor made[2];
    void* out[2];
    const bool given = a[7] != Py_None;
    if (given != (a[8] != Py_None)) return nullptr;
    if (given) {
        const Tensor *k = tensor(a[7]), *v = tensor(a[8]);
        if (!k || k->dim() != 4) return nullptr;
        N = k->size(2);
        if (N > 0x7fffffff || (!rows && N < T)) return nullptr;
        const int64_t shape[4] = {B, c.num_kv_heads, N, D};
        if (!exactly(k, at::kBFloat16, w, shape) || !exactly(v, at::kBFloat16, w, shape)) return nullptr;
        out[0] = k->data_ptr();
        out[1] = v->data_ptr();
    } else {
        if (counts || rows) return nullptr;   // new tensors that have to be cleared
        for (int i = 0; i < 2; ++i) {
            made[i] = w.empty({B, c.num_kv_heads, N, D}, at::kBFloat16);
            out[i] = made[i].data_ptr();
        }
    }
    if (without_gil([&] {
            return g_read(&c, static_cast<int32_t>(T), start, counts, rows, static_cast<int32_t>(N), out[0], out[1],
                          w.stream);
        }) != CP_OK)
        return nullptr;
    if (given) return PyTuple_Pack(2, a[7], a[8]);
    PyObject* t = PyTuple_New(2);
    if (!t) return nullptr;
    for (int i = 0; i < 2; ++i) PyTuple_SET_ITEM(t, i, THPVariable_Wrap(std::move(made[i])));
    return t;
}

// attn_kv4(q, pages, block_table, seq_lens, causal, window, softmax_scale, partial, o, lse)
PyObject* attn_kv4(PyObject* const* a)
{
    const Tensor* q = tensor(a[0]);
    if (!q || q->dim() != 4) return nullptr;
    Where w;
    cp_kv4_cache_t c;
    const int64_t B = q->size(0), H = q->size(1), T = q->size(2), D = q->size(3);
    if (!cache(a[1], a[2], D, B, w, &c)) return nullptr;
    int64_t qs[3], window;
    const int32_t* lens;
    if (!strided(*q, w, qs) || H % c.num_kv_heads != 0 || H > 0x7fffffff || T > 0x7fffffff) return nullptr;
    if (a[3] == Py_None || !optional(a[3], at::kInt, w, {B}, &lens)) return nullptr;
    if (!PyBool_Check(a[4]) || !PyBool_Check(a[7]) || !integer(a[5], &window) || !PyFloat_CheckExact(a[6])) return nullptr;
    const bool causal = a[4] == Py_True, partial = a[7] == Py_True;
    if (window < 0 || (window > 0 && !causal)) return nullptr;
    const float scale = static_cast<float>(PyFloat_AS_DOUBLE(a[6]));
    const at::ScalarType type = partial ? at::kFloat : at::kBFloat16;
    Tensor o, lse;
    if (a[8] == Py_None)
        o = w.empty(q->sizes(), type);
    else if (exactly(tensor(a[8]), type, w, q->sizes()))
        o = *tensor(a[8]);
    else
        return nullptr;
    if (a[9] == Py_None)
        lse = w.empty({B, H, T}, at::kFloat);
    else if (exactly(tensor(a[9]), at::kFloat, w, {B, H, T}))
        lse = *tensor(a[9]);
    else
        return nullptr;
    auto call = [&](void* ws, size_t* n) {
        return g_attn(&c, static_cast<int32_t>(H), static_cast<int32_t>(T), causal, static_cast<int32_t>(window), scale,
                      lens, q->data_ptr(), qs, o.data_ptr(), partial, static_cast<float*>(lse.data_ptr()), ws, n,
                      w.stream);
    };
    size_t n = 0;
    if (call(nullptr, &n) != CP_OK) return nullptr;
    Tensor ws;
    if (n > 0) ws = w.empty({static_cast<int64_t>(n)}, at::kByte);
    if (without_gil([&] { return n > 0 ? call(ws.data_ptr(), &n) : call(nullptr, nullptr); }) != CP_OK) return nullptr;
    PyObject* t = PyTuple_New(2);
    if (!t) return nullptr;
    PyTuple_SET_ITEM(t, 0, THPVariable_Wrap(std::move(o)));
    PyTuple_SET_ITEM(t, 1, THPVariable_Wrap(std::move(lse)));
    return t;
}

// None where the function gives nothing; no C++ exception reaches Python's frames.
template <PyObject* (*F)(PyObject* const*), Py_ssize_t N>
PyObject* entry(PyObject*, PyObject* const* args, Py_ssize_t n)
{
    PyObject* r = nullptr;
    if (n == N && g_rope) {
        try {
            r = F(args);
        } catch (...) {
            r = nullptr;
        }
    }
    if (r) return r;
    PyErr_Clear();
    return Py_NewRef(Py_None);
}

// bind(rope, kv4_write, kv4_read, attn_kv4): the addresses of the library's functions
PyObject* bind(PyObject*, PyObject* args)
{
    unsigned long long p[4];
    if (!PyArg_ParseTuple(args, "KKKK", p, p + 1, p + 2, p + 3)) return nullptr;
    g_write = reinterpret_cast<decltype(g_write)>(p[1]);
    g_read = reinterpret_cast<decltype(g_read)>(p[2]);
    g_attn = reinterpret_cast<decltype(g_attn)>(p[3]);
    g_rope = reinterpret_cast<decltype(g_rope)>(p[0]);
    return Py_NewRef(Py_None);
}

template <PyObject* (*F)(PyObject* const*), Py_ssize_t N>
PyMethodDef method(const char* name)
{
    return {name, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(&entry<F, N>)), METH_FASTCALL, nullptr};
}

PyMethodDef g_methods[] = {
    method<rope, 7>("rope"),
    method<kv4_write, 7>("kv4_write"),
    method<kv4_read, 9>("kv4_read"),
    method<attn_kv4, 10>("attn_kv4"),
    {"bind", bind, METH_VARARGS, nullptr},
    {nullptr, nullptr, 0, nullptr},
};

// The doc string names the torch that this was built for; the binding compares it.
PyModuleDef g_module = {PyModuleDef_HEAD_INIT, "_calls", CALLS_MARK, -1, g_methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__calls() { return PyModule_Create(&g_module); }
