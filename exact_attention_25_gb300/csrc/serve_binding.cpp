// Native binding of the serving calls (rotary positions, the paged cache, the decodes over it and
// over shared prefixes).  They are made once per token and layer, where a kernel takes a few
// microseconds, so their host side is compiled: argument checks, output allocation by torch's
// allocator and the C call of include/fa.h take about a third of what the same steps cost in Python.
// Nothing is computed here.  A call without rows, or whose longest sequence has none, returns without
// launching anything (the C entry points take sizes from 1 on).  Every function takes the address of its C entry point first (the caller
// chooses the library) and returns the outputs, or the int code of a refused call.
#include <Python.h>

#include <ATen/ATen.h>
#include <ATen/cuda/EmptyTensor.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/autograd/python_variable.h>

#include "../../include/fa.h"

namespace {

struct Refused {};  // a Python exception is set

[[noreturn]] void value_error(const char* what)
{
    PyErr_SetString(PyExc_ValueError, what);
    throw Refused{};
}
[[noreturn]] void type_error(const char* what)
{
    PyErr_SetString(PyExc_TypeError, what);
    throw Refused{};
}

// Arguments of a call, read in order.
struct Args {
    PyObject* const* a;
    Py_ssize_t n, i = 0;
    PyObject* next()
    {
        if (i >= n) type_error("too few arguments");
        return a[i++];
    }
    const at::Tensor& tensor()
    {
        PyObject* o = next();
        if (!THPVariable_Check(o)) type_error("expected a tensor");
        return THPVariable_Unpack(o);
    }
    const at::Tensor* optional()  // null for None
    {
        PyObject* o = next();
        if (o == Py_None) return nullptr;
        if (!THPVariable_Check(o)) type_error("expected a tensor or None");
        return &THPVariable_Unpack(o);
    }
    long long integer()
    {
        const long long v = PyLong_AsLongLong(next());
        if (v == -1 && PyErr_Occurred()) throw Refused{};
        return v;
    }
    int int32()
    {
        const long long v = integer();
        if (v < INT_MIN || v > INT_MAX) value_error("a size does not fit in 32 bits");
        return static_cast<int>(v);
    }
    double real()
    {
        const double v = PyFloat_AsDouble(next());
        if (v == -1.0 && PyErr_Occurred()) throw Refused{};
        return v;
    }
    int truth()
    {
        const int v = PyObject_IsTrue(next());
        if (v < 0) throw Refused{};
        return v;
    }
    // an entry point or a host array, by its address
    template <class P>
    P address()
    {
        void* p = PyLong_AsVoidPtr(next());
        if (!p) {
            if (!PyErr_Occurred()) PyErr_SetString(PyExc_TypeError, "an address is null");
            throw Refused{};
        }
        return reinterpret_cast<P>(p);
    }
};

int size32(int64_t v)
{
    if (v > INT_MAX) value_error("a size does not fit in 32 bits");
    return static_cast<int>(v);
}

// The tensors of a call lie on one CUDA device.
struct Device {
    c10::Device d;
    explicit Device(const at::Tensor& t) : d(t.device()) {}
    const c10::Device& cuda() const
    {
        if (!d.is_cuda()) value_error("tensors must be CUDA tensors");
        return d;
    }
    void same(const at::Tensor& t) const
    {
        if (t.device() != d) value_error("tensors must lie on one device");
    }
};

// A new contiguous tensor from torch's allocator, on the current stream (no dispatch: this is most of
// a small call's time).
at::Tensor empty(at::IntArrayRef sizes, at::ScalarType type, const Device& dev)
{
    return at::detail::empty_cuda(sizes, type, dev.d, std::nullopt);
}

int dtype_of(const at::Tensor& t)
{
    if (t.scalar_type() == at::kBFloat16) return FA_BF16;
    if (t.scalar_type() == at::kFloat) return FA_F32;
    type_error("unsupported dtype; use bfloat16 or float32");
}

void int32s(const at::Tensor& t, const char* what, int64_t n)
{
    if (t.scalar_type() != at::kInt || t.dim() != 1 || t.size(0) != n || !t.is_contiguous()) {
        if (t.scalar_type() != at::kInt) {
            PyErr_Format(PyExc_TypeError, "%s must be int32", what);
            throw Refused{};
        }
        PyErr_Format(PyExc_ValueError, "%s must be contiguous, of %lld entries", what, static_cast<long long>(n));
        throw Refused{};
    }
}

bool is_rows(const at::Tensor& t, int64_t rows, int64_t heads, int64_t d)
{
    return t.dim() == 3 && t.size(0) == rows && t.size(1) == heads && t.size(2) == d;
}

// (row, head) element strides of [rows, heads, d] views; used says whether any is not contiguous.
struct Strides {
    long long v[8];
    int n = 0;
    bool used = false;
    void add(const at::Tensor* t)
    {
        if (!t) {
            v[n++] = v[n++] = 0;
            return;
        }
        if (!t->is_contiguous()) {
            used = true;
            if (t->stride(2) != 1) value_error("packed views need contiguous head dimensions (stride 1 in d)");
        }
        // a dimension of one row or head is never stepped over: any valid step will do
        const long long hs = t->size(1) > 1 ? t->stride(1) : t->size(2);
        v[n++] = t->size(0) > 1 ? t->stride(0) : t->size(1) * hs;
        v[n++] = hs;
    }
    const long long* get() const { return used ? v : nullptr; }
};

struct Cache {
    const at::Tensor *k, *v, *ke, *ve, *table;
    int pages, Hkv, page, d, B, max_pages;
    void read(Args& a)
    {
        k = &a.tensor();
        v = &a.tensor();
        ke = &a.tensor();
        ve = &a.tensor();
    }
    void check(const at::Tensor& page_table, const Device& dev)
    {
        table = &page_table;
        if (k->dim() != 4 || v->sizes() != k->sizes())
            value_error("the cache's codes must be [num_pages, Hkv, page_size, d]");
        if (ke->sizes() != k->sizes().slice(0, 3) || ve->sizes() != ke->sizes())
            value_error("the cache's exponents must be [num_pages, Hkv, page_size]");
        for (const at::Tensor* t : {k, v, ke, ve}) {
            if (t->element_size() != 1 || !t->is_contiguous())
                value_error("the cache's tensors must be contiguous, of 1-byte elements");
            dev.same(*t);
        }
        if (table->scalar_type() != at::kInt) type_error("page_table must be int32");
        if (table->dim() != 2 || !table->is_contiguous())
            value_error("page_table must be contiguous, [B, max_pages]");
        dev.same(*table);
        pages = size32(k->size(0));
        Hkv = size32(k->size(1));
        page = size32(k->size(2));
        d = size32(k->size(3));
        B = size32(table->size(0));
        max_pages = size32(table->size(1));
    }
};

void check_q(const at::Tensor& q, int64_t d)
{
    if (q.dim() != 3 || q.size(2) != d) value_error("q must be [total_q, H, d]");
    if (q.scalar_type() != at::kBFloat16) type_error("q must be bfloat16");
    if (!q.is_contiguous()) value_error("q must be contiguous");
}
void check_o(const at::Tensor& o, const at::Tensor* lse, const at::Tensor& q)
{
    if (o.sizes() != q.sizes() || o.scalar_type() != at::kBFloat16 || !o.is_contiguous())
        value_error("o must be contiguous bfloat16 of q's shape");
    if (lse && (lse->scalar_type() != at::kFloat || !lse->is_contiguous() || lse->dim() != 2 ||
                lse->size(0) != q.size(1) || lse->size(1) != q.size(0)))
        value_error("lse must be contiguous fp32 [H, total_q]");
}

void* at_(const at::Tensor* t) { return t ? t->data_ptr() : nullptr; }
void* raw_stream(const Device& dev) { return c10::cuda::getCurrentCUDAStream(dev.d.index()).stream(); }

PyObject* none()
{
    Py_INCREF(Py_None);
    return Py_None;
}

PyObject* two(const at::Tensor& a, const at::Tensor* b)
{
    PyObject* t = PyTuple_New(2);
    if (!t) throw Refused{};
    PyTuple_SET_ITEM(t, 0, THPVariable_Wrap(a));
    PyTuple_SET_ITEM(t, 1, b ? THPVariable_Wrap(*b) : none());
    return t;
}

// rope(fn, q, k|None, q_out|None, k_out|None, positions, inv_freq (address), axis (address), table
// axes, d, pairs, interleaved, inverse) -> (q_out, k_out); outputs that are None are allocated
PyObject* rope(Args a)
{
    auto fn = a.address<decltype(&fa_rope)>();
    const at::Tensor& q = a.tensor();
    const at::Tensor* k = a.optional();
    const at::Tensor* qo = a.optional();
    const at::Tensor* ko = a.optional();
    const at::Tensor& pos = a.tensor();
    const auto* freq = a.address<const double*>();
    const auto* axis = a.address<const int*>();
    const int axes = a.int32();
    const int d = a.int32();
    const int pairs = a.int32(), interleaved = a.truth(), inverse = a.truth();
    if (q.dim() != 3) value_error("q must be [total, heads, d]");
    const int64_t total = q.size(0);
    if (q.size(2) != d) value_error("the table is made for another d");
    if (k && (!is_rows(*k, total, k->dim() == 3 ? k->size(1) : 0, d) || k->scalar_type() != q.scalar_type()))
        value_error("q and k must be [total, heads, d] of one dtype");
    if (pos.scalar_type() != at::kInt) type_error("positions must be int32");
    if (pos.dim() != 2 || pos.size(0) < axes || pos.size(1) != total || !pos.is_contiguous())
        value_error("positions must be contiguous, [axes, total], with the table's axes at least");
    const int dt = dtype_of(q);
    const Device dev(q);
    dev.same(pos);
    if (k) dev.same(*k);
    const c10::cuda::CUDAGuard guard(dev.cuda());
    at::Tensor q_new, k_new;
    if (!qo) {
        q_new = empty(q.sizes(), q.scalar_type(), dev);
        qo = &q_new;
    }
    if (!ko && k) {
        k_new = empty(k->sizes(), k->scalar_type(), dev);
        ko = &k_new;
    }
    if ((k == nullptr) != (ko == nullptr)) value_error("k and k_out come together");
    if (qo->sizes() != q.sizes() || qo->scalar_type() != q.scalar_type() ||
        (k && (ko->sizes() != k->sizes() || ko->scalar_type() != q.scalar_type())))
        value_error("outputs must have their inputs' shape and dtype");
    dev.same(*qo);
    if (ko) dev.same(*ko);
    if (total == 0) return two(*qo, ko);
    Strides st;
    for (const at::Tensor* t : {&q, k, qo, ko}) st.add(t);
    const int rc = fn(q.data_ptr(), at_(k), qo->data_ptr(), at_(ko), pos.data_ptr<int>(), freq, axis,
                      st.get(), size32(total), size32(q.size(1)), k ? size32(k->size(1)) : 0, d,
                      size32(pos.size(0)), pairs, interleaved, inverse, dt, raw_stream(dev));
    if (rc) return PyLong_FromLong(rc);
    return two(*qo, ko);
}

void check_kv(const at::Tensor& k, const at::Tensor& v, int64_t Hkv, int64_t d)
{
    if (k.dim() != 3 || k.size(1) != Hkv || k.size(2) != d || v.sizes() != k.sizes() ||
        v.scalar_type() != k.scalar_type())
        value_error("k and v must be [rows, Hkv, d] of one dtype");
}

// cache_append(fn, k_cache, v_cache, k_exp, v_exp, k, v, cu_seqlens_new, seqlens_k, page_table,
// max_seqlen_new) -> None
PyObject* cache_append(Args a)
{
    auto fn = a.address<decltype(&fa_cache_append)>();
    Cache c;
    c.read(a);
    const at::Tensor &k = a.tensor(), &v = a.tensor(), &cu = a.tensor(), &n = a.tensor(), &table = a.tensor();
    const int most = a.int32();
    const Device dev(k);
    c.check(table, dev);
    check_kv(k, v, c.Hkv, c.d);
    int32s(cu, "cu_seqlens_new", static_cast<int64_t>(c.B) + 1);
    int32s(n, "seqlens_k", c.B);
    for (const at::Tensor* t : {&v, &cu, &n}) dev.same(*t);
    const int dt = dtype_of(k);
    Strides st;
    st.add(&k);
    st.add(&v);
    const c10::cuda::CUDAGuard guard(dev.cuda());
    if (k.size(0) == 0 || most == 0) return none();
    const int rc = fn(k.data_ptr(), v.data_ptr(), st.get(), c.k->data_ptr(), c.v->data_ptr(), c.ke->data_ptr(),
                      c.ve->data_ptr(), cu.data_ptr<int>(), n.data_ptr<int>(), table.data_ptr<int>(), c.B,
                      most, size32(k.size(0)), c.max_pages, c.pages, c.page, c.Hkv, c.d, dt, raw_stream(dev));
    return rc ? PyLong_FromLong(rc) : none();
}

// cache_read(fn, k_cache, v_cache, k_exp, v_exp, k|None, v|None, cu_seqlens_k, page_table,
// max_seqlen_k, total_k, fp32) -> (k, v); allocated where None
PyObject* cache_read(Args a)
{
    auto fn = a.address<decltype(&fa_cache_read)>();
    Cache c;
    c.read(a);
    const at::Tensor* k = a.optional();
    const at::Tensor* v = a.optional();
    const at::Tensor &cu = a.tensor(), &table = a.tensor();
    const int most = a.int32();
    const long long total = a.integer();
    const int fp32 = a.truth();
    const Device dev(*c.k);
    c.check(table, dev);
    int32s(cu, "cu_seqlens_k", static_cast<int64_t>(c.B) + 1);
    dev.same(cu);
    const c10::cuda::CUDAGuard guard(dev.cuda());
    at::Tensor k_new, v_new;
    if (!k || !v) {
        if (k || v) value_error("k and v come together");
        if (total < 0) value_error("total_k must not be negative");
        const auto type = fp32 ? at::kFloat : at::kBFloat16;
        k_new = empty({total, c.Hkv, c.d}, type, dev);
        v_new = empty({total, c.Hkv, c.d}, type, dev);
        k = &k_new;
        v = &v_new;
    }
    check_kv(*k, *v, c.Hkv, c.d);
    dev.same(*k);
    dev.same(*v);
    const int dt = dtype_of(*k);
    if (k->size(0) == 0 || most == 0) return two(*k, v);
    Strides st;
    st.add(k);
    st.add(v);
    const int rc = fn(c.k->data_ptr(), c.v->data_ptr(), c.ke->data_ptr(), c.ve->data_ptr(), k->data_ptr(),
                      v->data_ptr(), st.get(), cu.data_ptr<int>(), table.data_ptr<int>(), c.B, most,
                      size32(k->size(0)), c.max_pages, c.pages, c.page, c.Hkv, c.d, dt, raw_stream(dev));
    if (rc) return PyLong_FromLong(rc);
    return two(*k, v);
}

// A decode's outputs and workspace: those given, or new ones.
struct DecodeOut {
    const at::Tensor *o, *lse, *ws;
    at::Tensor o_new, lse_new, ws_new;
    void read(Args& a)
    {
        o = a.optional();
        lse = a.optional();
        ws = a.optional();
        if (ws && !ws->is_contiguous()) value_error("the workspace must be contiguous");
    }
    // without o everything is allocated, `bytes` of workspace
    void make(const at::Tensor& q, const Device& dev, size_t bytes)
    {
        if (!o) {
            o_new = empty(q.sizes(), q.scalar_type(), dev);
            lse_new = empty({q.size(1), q.size(0)}, at::kFloat, dev);
            o = &o_new;
            lse = &lse_new;
            if (bytes) {
                ws_new = empty({static_cast<int64_t>(bytes)}, at::kByte, dev);
                ws = &ws_new;
            }
        }
        check_o(*o, lse, q);
        dev.same(*o);
        if (lse) dev.same(*lse);
        if (ws) dev.same(*ws);
    }
    size_t ws_bytes() const { return ws ? ws->nbytes() : 0; }
    // the result of a call without queries
    PyObject* nothing(const at::Tensor& q, const Device& dev)
    {
        make(q, dev, 0);
        return two(*o, lse);
    }
};

// decode_cache(fn, ctas_fn, bytes_fn, q, k_cache, v_cache, k_exp, v_exp, o|None, lse|None, ws|None,
// cu_seqlens_q, seqlens_k, page_table, max_seqlen_q, max_seqlen_k, scale, causal, num_ctas or 0)
// -> (o, lse)
PyObject* decode_cache(Args a)
{
    auto fn = a.address<decltype(&fa_fwd_decode_cache)>();
    auto ctas_fn = a.address<decltype(&fa_decode_cache_num_ctas)>();
    auto bytes_fn = a.address<decltype(&fa_decode_cache_workspace_bytes)>();
    const at::Tensor& q = a.tensor();
    Cache c;
    c.read(a);
    DecodeOut out;
    out.read(a);
    const at::Tensor &cu = a.tensor(), &n = a.tensor(), &table = a.tensor();
    const int mq = a.int32(), mk = a.int32();
    const float scale = static_cast<float>(a.real());
    const int causal = a.truth();
    int ctas = a.int32();
    const Device dev(q);
    c.check(table, dev);
    check_q(q, c.d);
    int32s(cu, "cu_seqlens_q", static_cast<int64_t>(c.B) + 1);
    int32s(n, "seqlens_k", c.B);
    dev.same(cu);
    dev.same(n);
    const int H = size32(q.size(1));
    const c10::cuda::CUDAGuard guard(dev.cuda());
    if (q.size(0) == 0 || mq == 0) return out.nothing(q, dev);
    if (ctas == 0) ctas = ctas_fn(c.B, H, c.Hkv, mq, mk);
    if (ctas < 0) return PyLong_FromLong(ctas);
    out.make(q, dev, out.o ? 0 : bytes_fn(H, c.Hkv, c.d, mq, ctas));
    const int rc = fn(q.data_ptr(), c.k->data_ptr(), c.v->data_ptr(), c.ke->data_ptr(), c.ve->data_ptr(),
                      out.o->data_ptr(), static_cast<float*>(at_(out.lse)), cu.data_ptr<int>(),
                      n.data_ptr<int>(), table.data_ptr<int>(), c.B, mq, mk, size32(q.size(0)), c.max_pages,
                      c.pages, c.page, H, c.Hkv, c.d, scale, causal, ctas, at_(out.ws), out.ws_bytes(),
                      raw_stream(dev));
    if (rc) return PyLong_FromLong(rc);
    return two(*out.o, out.lse);
}

// decode_shared(fn, ctas_fn, bytes_fn, q, k_prefix, v_prefix, k, v, o|None, lse|None, ws|None,
// cu_seqlens_q, cu_seqlens_k, cu_groups, cu_seqlens_p, max_seqlen_q, max_seqlen_k, max_group_q,
// max_seqlen_p, scale, causal, num_ctas or 0) -> (o, lse)
PyObject* decode_shared(Args a)
{
    auto fn = a.address<decltype(&fa_fwd_decode_shared)>();
    auto ctas_fn = a.address<decltype(&fa_decode_shared_num_ctas)>();
    auto bytes_fn = a.address<decltype(&fa_decode_shared_workspace_bytes)>();
    const at::Tensor &q = a.tensor(), &kp = a.tensor(), &vp = a.tensor(), &k = a.tensor(), &v = a.tensor();
    DecodeOut out;
    out.read(a);
    const at::Tensor &cq = a.tensor(), &ck = a.tensor(), &cg = a.tensor(), &cp = a.tensor();
    const int mq = a.int32();
    int mk = a.int32();
    const int mg = a.int32();
    int mp = a.int32();
    const float scale = static_cast<float>(a.real());
    const int causal = a.truth();
    int ctas = a.int32();
    const Device dev(q);
    if (q.dim() != 3) value_error("q must be [total_q, H, d]");
    const int64_t d = q.size(2);
    check_q(q, d);
    const int64_t Hkv = k.dim() == 3 ? k.size(1) : 0;
    check_kv(k, v, Hkv, d);
    check_kv(kp, vp, Hkv, d);
    for (const at::Tensor* t : {&k, &v, &kp, &vp}) {
        if (t->scalar_type() != at::kBFloat16 || !t->is_contiguous())
            value_error("keys and values must be contiguous bfloat16");
        dev.same(*t);
    }
    if (cq.dim() != 1 || cg.dim() != 1) value_error("cu_seqlens_q and cu_groups must have one dimension");
    int32s(cq, "cu_seqlens_q", cq.size(0));
    int32s(ck, "cu_seqlens_k", cq.size(0));
    int32s(cg, "cu_groups", cg.size(0));
    int32s(cp, "cu_seqlens_p", cg.size(0));
    for (const at::Tensor* t : {&cq, &ck, &cg, &cp}) dev.same(*t);
    const int H = size32(q.size(1)), total_q = size32(q.size(0));
    // no rows, or none that count: the call takes both numbers as 0
    int total_k = size32(k.size(0)), total_p = size32(kp.size(0));
    if (total_k == 0 || mk == 0) total_k = mk = 0;
    if (total_p == 0 || mp == 0) total_p = mp = 0;
    const c10::cuda::CUDAGuard guard(dev.cuda());
    if (total_q == 0 || mq == 0) return out.nothing(q, dev);
    if (ctas == 0) ctas = ctas_fn();
    if (ctas < 0) return PyLong_FromLong(ctas);
    out.make(q, dev, out.o ? 0 : bytes_fn(total_q, H, size32(d), ctas));
    const int rc = fn(q.data_ptr(), kp.data_ptr(), vp.data_ptr(), k.data_ptr(), v.data_ptr(), out.o->data_ptr(),
                      static_cast<float*>(at_(out.lse)), cq.data_ptr<int>(), ck.data_ptr<int>(),
                      cg.data_ptr<int>(), cp.data_ptr<int>(), size32(cq.size(0)) - 1, size32(cg.size(0)) - 1, mq,
                      mk, mg, mp, total_q, total_k, total_p, H, size32(Hkv), size32(d), scale, causal, ctas,
                      at_(out.ws), out.ws_bytes(), raw_stream(dev));
    if (rc) return PyLong_FromLong(rc);
    return two(*out.o, out.lse);
}

// No C++ exception leaves the module.
template <PyObject* (*F)(Args)>
PyObject* guarded(PyObject*, PyObject* const* args, Py_ssize_t n)
{
    try {
        return F(Args{args, n});
    } catch (const Refused&) {
    } catch (const std::exception& e) {
        PyErr_SetString(PyExc_RuntimeError, e.what());
    } catch (...) {
        PyErr_SetString(PyExc_RuntimeError, "unknown C++ exception");
    }
    return nullptr;
}

template <PyObject* (*F)(Args)>
PyMethodDef method(const char* name)
{
    return {name, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(&guarded<F>)), METH_FASTCALL, nullptr};
}

PyMethodDef g_methods[] = {method<rope>("rope"),
                           method<cache_append>("cache_append"),
                           method<cache_read>("cache_read"),
                           method<decode_cache>("decode_cache"),
                           method<decode_shared>("decode_shared"),
                           {nullptr, nullptr, 0, nullptr}};

PyModuleDef g_module = {PyModuleDef_HEAD_INIT, "_serve", nullptr, -1, g_methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__serve(void) { return PyModule_Create(&g_module); }
