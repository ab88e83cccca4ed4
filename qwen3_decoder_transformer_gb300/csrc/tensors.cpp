// The binding's checks of a call's tensors and its argument block (the args structs of qwen3.h), as an extension module: through
// Python attributes checks and block take 4.5 us of an append and 3.3 of a read, as much as the launch; here 0.7 and
// 0.8, the binding's own call included (1 token appended and read: 14-15 us in calls, 7.2). Each function takes the tensors
// of the binding's call, and returns the block as bytes (empty: there are no rows), or None if anything is wrong, which
// the binding then words.
#include <torch/csrc/autograd/python_variable.h>

#include <algorithm>
#include <initializer_list>
#include <limits>

#include "qwen3.h"

namespace {

// Tensors of one device; ok becomes false at the first that is not as wanted.
struct Call {
    int64_t device;
    bool ok = true;

    const at::Tensor* tensor(PyObject* o, int64_t dims) {
        if (ok && THPVariable_Check(o)) {
            const at::Tensor& t = THPVariable_Unpack(o);
            if (t.layout() == at::kStrided && t.dim() == dims && t.get_device() == device) return &t;
        }
        ok = false;
        return nullptr;
    }
    // The address of a contiguous tensor of this type and shape.
    void* dense(PyObject* o, at::ScalarType type, std::initializer_list<int64_t> shape) {
        const at::Tensor* t = tensor(o, (int64_t)shape.size());
        if (t && t->scalar_type() == type && t->sizes() == at::IntArrayRef(shape) && t->is_contiguous()) return t->data_ptr();
        ok = false;
        return nullptr;
    }
    void* dense_or_none(PyObject* o, at::ScalarType type, std::initializer_list<int64_t> shape) {
        return o == Py_None ? nullptr : dense(o, type, shape);
    }
    // The address of contiguous scratch of any type and shape.
    void* scratch(PyObject* o, size_t& bytes) {
        if (ok && THPVariable_Check(o)) {
            const at::Tensor& t = THPVariable_Unpack(o);
            if (t.layout() == at::kStrided && t.get_device() == device && t.is_contiguous()) {
                bytes = t.nbytes();
                return t.data_ptr();
            }
        }
        ok = false;
        return nullptr;
    }
    int32_t i32(int64_t v) {
        if (v < 0 || v > std::numeric_limits<int32_t>::max()) ok = false;
        return (int32_t)v;
    }
};

// k_pages, v_pages [n_pages, Hkv, page bytes] uint8 and page_table [sequences, max_pages] int32
struct Pages {
    void *k = nullptr, *v = nullptr, *table = nullptr;
    int32_t n_pages = 0, page_size = 0, max_pages = 0;
    int64_t Hkv = 0, sequences = 0;

    Pages(Call& c, PyObject* k_pages, PyObject* v_pages, PyObject* page_table, int64_t dh) {
        const at::Tensor *kt = c.tensor(k_pages, 3), *tt = c.tensor(page_table, 2);
        if (!c.ok) return;
        const int64_t n = kt->size(0), size = kt->size(2), max = tt->size(1);
        Hkv = kt->size(1);
        sequences = tt->size(0);
        k = c.dense(k_pages, at::kByte, {n, Hkv, size});
        v = c.dense(v_pages, at::kByte, {n, Hkv, size});
        table = c.dense(page_table, at::kInt, {sequences, max});
        for (int32_t p = 16; p <= 256; p *= 2)
            if ((dh == 64 || dh == 128) && p * (dh / 2 + dh / 64 * 4) == size) page_size = p;
        n_pages = c.i32(n);
        max_pages = c.i32(max);
        c.i32(sequences);
        c.ok = c.ok && page_size && n >= 1 && Hkv >= 1 && max >= 1;
    }
};

int64_t device_of(PyObject* o) { return THPVariable_Check(o) ? THPVariable_Unpack(o).get_device() : -2; }

template <typename Args>
PyObject* block(const Call& c, bool rows, const Args& a) {
    if (!c.ok) Py_RETURN_NONE;
    return PyBytes_FromStringAndSize(reinterpret_cast<const char*>(&a), rows ? sizeof(a) : 0);
}

// qkv, cu, start, cos_sin, k_pages, v_pages, page_table, q_out, k_out, q_gamma, k_gamma, eps, err
PyObject* append_paged4(PyObject* const* o) {
    Call c{device_of(o[0])};
    qwen3_append_paged4_args a{};
    a.eps = (float)PyFloat_AsDouble(o[11]);
    if (PyErr_Occurred()) return nullptr;
    const at::Tensor *qkv = c.tensor(o[0], 2), *q = c.tensor(o[7], 3), *angles = c.tensor(o[3], 2);
    if (!c.ok) Py_RETURN_NONE;
    const int64_t N = q->size(0), Hq = q->size(1), dh = q->size(2);
    const Pages p(c, o[4], o[5], o[6], dh);
    if (!c.ok) Py_RETURN_NONE;
    const int64_t width = (Hq + 2 * p.Hkv) * dh;
    c.ok = Hq >= 1 && Hq % p.Hkv == 0 && qkv->scalar_type() == at::kBFloat16 && qkv->size(0) == N && qkv->size(1) == width &&
           qkv->stride(1) == 1;
    a.d_qkv = qkv->data_ptr();
    a.ld = N == 1 ? width : qkv->stride(0);  // (the stride of a single row says nothing)
    a.N = c.i32(N);
    a.d_cu = (const int*)c.dense(o[1], at::kInt, {p.sequences + 1});
    a.d_start = (const int*)c.dense(o[2], at::kInt, {p.sequences});
    a.S = (int32_t)p.sequences;
    a.Hq = c.i32(Hq);
    a.Hkv = c.i32(p.Hkv);
    a.dh = (int32_t)dh;
    a.d_q_gamma = c.dense_or_none(o[9], at::kBFloat16, {dh});
    a.d_k_gamma = c.dense_or_none(o[10], at::kBFloat16, {dh});
    a.d_cos_sin = c.dense(o[3], at::kBFloat16, {angles->size(0), dh});
    a.n_pos = c.i32(angles->size(0));
    a.d_q_out = c.dense(o[7], at::kBFloat16, {N, Hq, dh});
    a.d_k_out = c.dense_or_none(o[8], at::kBFloat16, {N, p.Hkv, dh});
    a.d_k_pages = p.k;
    a.d_v_pages = p.v;
    a.n_pages = p.n_pages;
    a.page_size = p.page_size;
    a.d_page_table = (const int*)p.table;
    a.max_pages = p.max_pages;
    a.d_err = (int*)c.dense_or_none(o[12], at::kInt, {1});
    return block(c, N > 0 && p.sequences > 0, a);
}

// k_pages, v_pages, page_table, cu, start, k_out, v_out, err
PyObject* read_paged4(PyObject* const* o) {
    Call c{device_of(o[5])};
    qwen3_read_paged4_args a{};
    const at::Tensor* k = c.tensor(o[5], 3);
    if (!c.ok) Py_RETURN_NONE;
    const int64_t N = k->size(0), dh = k->size(2);
    const Pages p(c, o[0], o[1], o[2], dh);
    if (!c.ok) Py_RETURN_NONE;
    a.d_k_pages = p.k;
    a.d_v_pages = p.v;
    a.n_pages = p.n_pages;
    a.page_size = p.page_size;
    a.d_page_table = (const int*)p.table;
    a.max_pages = p.max_pages;
    a.d_cu = (const int*)c.dense(o[3], at::kInt, {p.sequences + 1});
    a.d_start = (const int*)c.dense(o[4], at::kInt, {p.sequences});
    a.S = (int32_t)p.sequences;
    a.N = c.i32(N);
    a.Hkv = c.i32(p.Hkv);
    a.dh = (int32_t)dh;
    a.d_k_out = c.dense(o[5], at::kBFloat16, {N, p.Hkv, dh});
    a.d_v_out = c.dense(o[6], at::kBFloat16, {N, p.Hkv, dh});
    a.d_err = (int*)c.dense_or_none(o[7], at::kInt, {1});
    return block(c, N > 0 && p.sequences > 0, a);
}

// q, k_pages, v_pages, page_table, len0, work, out, err
PyObject* attention_decode_paged4(PyObject* const* o) {
    Call c{device_of(o[0])};
    qwen3_attention_decode_paged4_args a{};
    const at::Tensor* q = c.tensor(o[0], 3);
    if (!c.ok) Py_RETURN_NONE;
    const int64_t B = q->size(0), Hq = q->size(1), dh = q->size(2);
    const Pages p(c, o[1], o[2], o[3], dh);
    if (!c.ok) Py_RETURN_NONE;
    c.ok = Hq >= 1 && Hq % p.Hkv == 0 && Hq <= 8 * p.Hkv && p.sequences == B;
    a.d_q = c.dense(o[0], at::kBFloat16, {B, Hq, dh});
    a.d_k_pages = p.k;
    a.d_v_pages = p.v;
    a.n_pages = p.n_pages;
    a.page_size = p.page_size;
    a.d_page_table = (const int*)p.table;
    a.max_pages = p.max_pages;
    a.d_len0 = (const int*)c.dense(o[4], at::kInt, {B});
    a.B = c.i32(B);
    a.Hq = c.i32(Hq);
    a.Hkv = c.i32(p.Hkv);
    a.dh = (int32_t)dh;
    a.d_work = c.scratch(o[5], a.work_bytes);
    a.d_out = c.dense(o[6], at::kBFloat16, {B, Hq * dh});
    a.d_err = (int*)c.dense_or_none(o[7], at::kInt, {1});
    return block(c, B > 0, a);
}

// q, k, v, plan, longest, out, err
PyObject* attention_prefill_packed(PyObject* const* o) {
    Call c{device_of(o[0])};
    qwen3_attention_prefill_packed_args a{};
    int past = 0;  // of a whole number past 64 bits: its sign
    long long longest = PyLong_AsLongLongAndOverflow(o[4], &past);
    if (PyErr_Occurred()) return nullptr;
    if (past) longest = past < 0 ? 0 : std::numeric_limits<int32_t>::max();
    const at::Tensor *q = c.tensor(o[0], 3), *k = c.tensor(o[1], 3), *v = c.tensor(o[2], 3);
    if (!c.ok) Py_RETURN_NONE;
    const int64_t Nq = q->size(0), Hq = q->size(1), dh = q->size(2), Nk = k->size(0), Hkv = k->size(1);
    for (const at::Tensor* t : {q, k, v})  // rows may be further apart
        c.ok = c.ok && t->scalar_type() == at::kBFloat16 && t->size(2) == dh && t->stride(2) == 1 &&
               (t->size(1) == 1 || t->stride(1) == dh);
    c.ok = c.ok && v->sizes() == k->sizes() && Hkv >= 1 && Hq >= 1 && Hq % Hkv == 0;
    a.d_q = q->data_ptr();
    a.ldq = Nq == 1 ? Hq * dh : q->stride(0);  // (the stride of a single row says nothing)
    a.d_k = k->data_ptr();
    a.ldk = Nk <= 1 ? Hkv * dh : k->stride(0);
    a.d_v = v->data_ptr();
    a.ldv = Nk <= 1 ? Hkv * dh : v->stride(0);
    a.Nq = c.i32(Nq);
    a.Nk = c.i32(Nk);
    a.Hq = c.i32(Hq);
    a.Hkv = c.i32(Hkv);
    a.dh = c.i32(dh);
    a.d_plan = c.scratch(o[3], a.plan_bytes);
    a.longest = (int32_t)std::clamp<long long>(longest, 0, std::numeric_limits<int32_t>::max());  // (any value is right)
    a.d_out = c.dense(o[5], at::kBFloat16, {Nq, Hq * dh});
    a.d_err = (int*)c.dense_or_none(o[6], at::kInt, {1});
    return block(c, Nq > 0, a);
}

// What torch throws (of a tensor without storage, say) reads as a tensor that is not as wanted.
template <PyObject* (*F)(PyObject* const*), int N>
PyObject* entry(PyObject*, PyObject* const* args, Py_ssize_t n) {
    if (n != N) {
        PyErr_Format(PyExc_TypeError, "%d arguments are wanted, not %zd", N, n);
        return nullptr;
    }
    try {
        return F(args);
    } catch (...) {
        Py_RETURN_NONE;
    }
}
template <PyObject* (*F)(PyObject* const*), int N>
PyMethodDef method(const char* name) {
    return {name, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(entry<F, N>)), METH_FASTCALL, nullptr};
}
PyMethodDef methods[] = {method<append_paged4, 13>("append_paged4"), method<read_paged4, 8>("read_paged4"),
                         method<attention_decode_paged4, 8>("attention_decode_paged4"),
                         method<attention_prefill_packed, 7>("attention_prefill_packed"), {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_tensors", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__tensors() { return PyModule_Create(&module); }
