// fa_binding.cpp -- the common case of the cache and rotary calls (cache.py),
// marshalled natively: tensors on the current device, its current stream.
//
// A decoding step makes these calls for every layer, and their kernels take 3
// to 10 us; in Python the checks, allocations and argument conversions take 8 to 16 us,
// here 3 to 6.  Each function returns what the Python call returns, or an
// int status of the C-ABI that is not FA_OK, or NotImplemented for anything that is
// not the common case (another device, an argument that does not fit): the Python
// code then handles the call or says what was wrong.  No function computes anything.
#include <Python.h>

#include <ATen/ops/empty.h>
#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/autograd/python_variable.h>

#include <cmath>
#include <cstdint>
#include <limits>

#include "fa_gb300.h"

namespace {

// The library's entry points (init gets their addresses from the loaded library).
decltype(&fa_kv4_write) p_write;
decltype(&fa_kv4_read) p_read;
decltype(&fa_kv4_attention_workspace_size) p_workspace;
decltype(&fa_kv4_attention) p_attention;
decltype(&fa_rotary) p_rotary;

PyObject* not_here() { Py_RETURN_NOTIMPLEMENTED; }

const at::Tensor* tensor(PyObject* o) { return THPVariable_Check(o) ? &THPVariable_Unpack(o) : nullptr; }

bool fits(int64_t x) { return x >= 0 && x <= std::numeric_limits<int>::max(); }

// A Python int that fits an int; false otherwise.
bool integer(PyObject* o, int* x) {
    if (!PyLong_Check(o)) return false;
    int over = 0;
    const long long v = PyLong_AsLongLongAndOverflow(o, &over);
    if (over != 0 || v < std::numeric_limits<int>::min() || v > std::numeric_limits<int>::max()) return false;
    *x = static_cast<int>(v);
    return true;
}

bool half_type(const at::Tensor& t, int* dtype) {
    if (t.scalar_type() == at::kBFloat16) *dtype = FA_BF16;
    else if (t.scalar_type() == at::kHalf) *dtype = FA_F16;
    else return false;
    return true;
}

// A contiguous CUDA tensor of one type on `dev`.
bool plain(const at::Tensor* t, at::ScalarType type, c10::Device dev) {
    return t != nullptr && t->scalar_type() == type && t->is_contiguous() && t->device() == dev;
}

// The cache's arguments: codes, scales, page_table, seq_lens, cu_seqlens, max_seqlen.
bool parse_cache(PyObject* const* a, int64_t rows, fa_kv4_cache_t* c, c10::Device* device) {
    const at::Tensor *codes = tensor(a[0]), *scales = tensor(a[1]), *table = tensor(a[2]), *lens = tensor(a[3]);
    if (codes == nullptr || !codes->is_cuda()) return false;
    const c10::Device dev = codes->device();
    if (dev.index() != c10::cuda::current_device()) return false;
    if (!plain(codes, at::kByte, dev) || !plain(scales, at::kBFloat16, dev) || !plain(table, at::kInt, dev) ||
        !plain(lens, at::kInt, dev) || codes->dim() != 5 || scales->dim() != 5 || table->dim() != 2 || lens->dim() != 1)
        return false;
    const auto s = codes->sizes(), t = scales->sizes();
    const int64_t B = table->size(0), D = s[4] * 2;
    if (s[1] != 2 || t[0] != s[0] || t[1] != 2 || t[2] != s[2] || t[3] != s[3] || t[4] != s[4] / 16 || lens->size(0) != B)
        return false;
    if (!fits(s[0]) || !fits(s[2]) || !fits(s[3]) || !fits(D) || !fits(B) || !fits(table->size(1)) || !fits(rows)) return false;
    c->codes = codes->data_ptr();
    c->scales = scales->data_ptr();
    c->page_table = static_cast<const int*>(table->data_ptr());
    c->seq_lens = static_cast<const int*>(lens->data_ptr());
    c->cu_seqlens = nullptr;
    c->B = static_cast<int>(B);
    c->max_seqlen = static_cast<int>(rows);
    c->total = 0;
    if (a[4] != Py_None) {
        const at::Tensor* cu = tensor(a[4]);
        if (!plain(cu, at::kInt, dev) || cu->dim() != 1 || cu->size(0) != B + 1) return false;
        c->cu_seqlens = static_cast<const int*>(cu->data_ptr());
        c->total = static_cast<int>(rows);
        if (a[5] != Py_None && !integer(a[5], &c->max_seqlen)) return false;
    }
    c->pages = static_cast<int>(s[0]);
    c->max_pages = static_cast<int>(table->size(1));
    c->page_size = static_cast<int>(s[3]);
    c->H_kv = static_cast<int>(s[2]);
    c->D = static_cast<int>(D);
    *device = dev;
    return true;
}

// A tensor of the call's rows, [B, S, heads, D] or packed [total, heads, D]; its strides.
bool rows_of(const at::Tensor& t, const fa_kv4_cache_t& c, c10::Device dev, long long* strides) {
    const int dim = c.cu_seqlens != nullptr ? 3 : 4;
    if (t.dim() != dim || t.device() != dev || t.size(dim - 1) != c.D || t.stride(dim - 1) != 1) return false;
    if (dim == 4 && t.size(0) != c.B) return false;
    strides[0] = dim == 4 ? t.stride(0) : 0;
    strides[1] = t.stride(dim - 3);
    strides[2] = t.stride(dim - 2);
    return true;
}

fa_stream_t stream_of(c10::Device dev) {
    return reinterpret_cast<fa_stream_t>(c10::cuda::getCurrentCUDAStream(dev.index()).stream());
}

// k, v, codes, scales, page_table, seq_lens, cu_seqlens, max_seqlen, k_out, v_out -> None
PyObject* kv4_write(PyObject*, PyObject* const* a, Py_ssize_t n) {
    try {
        if (n != 10) return not_here();
        const at::Tensor *k = tensor(a[0]), *v = tensor(a[1]);
        int dtype = 0;
        if (k == nullptr || v == nullptr || k->dim() < 3 || k->sizes() != v->sizes() || k->scalar_type() != v->scalar_type() ||
            !half_type(*k, &dtype) || k->numel() == 0)
            return not_here();
        fa_kv4_cache_t c;
        c10::Device dev(c10::kCPU);
        long long ks[3], vs[3];
        if (!parse_cache(a + 2, k->size(-3), &c, &dev) || !rows_of(*k, c, dev, ks) || !rows_of(*v, c, dev, vs) ||
            k->size(-2) != c.H_kv)
            return not_here();
        void *ko = nullptr, *vo = nullptr;
        if (a[8] != Py_None || a[9] != Py_None) {
            const at::Tensor *o = tensor(a[8]), *p = tensor(a[9]);
            if (!plain(o, k->scalar_type(), dev) || !plain(p, k->scalar_type(), dev) || o->sizes() != k->sizes() ||
                p->sizes() != k->sizes())
                return not_here();
            ko = o->data_ptr();
            vo = p->data_ptr();
        }
        const int rc = p_write(&c, k->data_ptr(), v->data_ptr(), ks, vs, ko, vo, dtype, stream_of(dev));
        if (rc != FA_OK) return PyLong_FromLong(rc);
        Py_RETURN_NONE;
    } catch (...) {
        return not_here();
    }
}

// codes, scales, page_table, seq_lens, cu_seqlens, max_seqlen, rows, bf16 -> (k, v)
PyObject* kv4_read(PyObject*, PyObject* const* a, Py_ssize_t n) {
    try {
        int rows = 0;
        if (n != 8 || !integer(a[6], &rows) || rows < 1) return not_here();
        const bool bf16 = a[7] == Py_True;
        fa_kv4_cache_t c;
        c10::Device dev(c10::kCPU);
        if (!parse_cache(a, rows, &c, &dev) || c.B < 1 || c.H_kv < 1 || c.D < 1) return not_here();
        const auto opt = at::TensorOptions().dtype(bf16 ? at::kBFloat16 : at::kHalf).device(dev);
        at::Tensor k, v;
        if (c.cu_seqlens != nullptr) {
            k = at::empty({rows, c.H_kv, c.D}, opt);
            v = at::empty({rows, c.H_kv, c.D}, opt);
        } else {
            k = at::empty({c.B, rows, c.H_kv, c.D}, opt);
            v = at::empty({c.B, rows, c.H_kv, c.D}, opt);
        }
        const int rc = p_read(&c, k.data_ptr(), v.data_ptr(), bf16 ? FA_BF16 : FA_F16, stream_of(dev));
        if (rc != FA_OK) return PyLong_FromLong(rc);
        return Py_BuildValue("(NN)", THPVariable_Wrap(std::move(k)), THPVariable_Wrap(std::move(v)));
    } catch (...) {
        return not_here();
    }
}

// q, codes, scales, page_table, seq_lens, cu_seqlens, max_seqlen, window_left, scale, out, lse, with_lse -> (out, lse)
PyObject* kv4_attention(PyObject*, PyObject* const* a, Py_ssize_t n) {
    try {
        const at::Tensor* q = n == 12 ? tensor(a[0]) : nullptr;
        int dtype = 0, window = 0;
        if (q == nullptr || q->dim() < 3 || !half_type(*q, &dtype) || q->numel() == 0 || !integer(a[7], &window))
            return not_here();
        fa_kv4_cache_t c;
        c10::Device dev(c10::kCPU);
        long long qs[3];
        const int64_t rows = q->size(-3), H = q->size(-2);
        if (!parse_cache(a + 1, rows, &c, &dev) || !rows_of(*q, c, dev, qs) || !fits(H) || c.H_kv < 1 || c.D < 1 ||
            H % c.H_kv != 0)
            return not_here();
        double scale = 1.0 / std::sqrt(static_cast<double>(c.D));
        if (a[8] != Py_None) {
            if (!PyFloat_Check(a[8])) return not_here();
            scale = PyFloat_AsDouble(a[8]);
        }
        at::Tensor out, lse;
        if (a[9] != Py_None) {
            const at::Tensor* o = tensor(a[9]);
            if (!plain(o, q->scalar_type(), dev) || o->sizes() != q->sizes()) return not_here();
            out = *o;
        }
        const bool packed = c.cu_seqlens != nullptr;
        if (a[10] != Py_None) {
            const at::Tensor* l = tensor(a[10]);
            if (!plain(l, at::kFloat, dev)) return not_here();
            if (packed ? (l->dim() != 2 || l->size(0) != H || l->size(1) != rows)
                       : (l->dim() != 3 || l->size(0) != c.B || l->size(1) != H || l->size(2) != rows))
                return not_here();
            lse = *l;
        }
        size_t bytes = 0;
        int rc = p_workspace(&c, static_cast<int>(H), dtype, &bytes);
        if (rc != FA_OK) return PyLong_FromLong(rc);
        const auto opt = q->options();
        if (!out.defined()) out = at::empty(q->sizes(), opt);
        if (!lse.defined() && a[11] != Py_False) {
            const auto f32 = opt.dtype(at::kFloat);
            lse = packed ? at::empty({H, rows}, f32) : at::empty({c.B, H, rows}, f32);
        }
        // not kept: two captured graphs never share one
        at::Tensor ws;
        if (bytes > 0) ws = at::empty({static_cast<int64_t>(bytes)}, opt.dtype(at::kByte));
        rc = p_attention(&c, q->data_ptr(), qs, out.data_ptr(), lse.defined() ? static_cast<float*>(lse.data_ptr()) : nullptr,
                         static_cast<int>(H), window, static_cast<float>(scale), dtype, bytes > 0 ? ws.data_ptr() : nullptr, bytes, stream_of(dev));
        if (rc != FA_OK) return PyLong_FromLong(rc);
        PyObject* l = lse.defined() ? THPVariable_Wrap(std::move(lse)) : Py_NewRef(Py_None);
        return Py_BuildValue("(NN)", THPVariable_Wrap(std::move(out)), l);
    } catch (...) {
        return not_here();
    }
}

// The strides (token, head) of t [T, heads, D] or [B, S, heads, D] with evenly spaced tokens.
bool tokens_of(const at::Tensor& t, long long* strides) {
    const int64_t dim = t.dim();
    if (t.stride(dim - 1) != 1) return false;
    if (dim == 4 && t.size(0) != 1 && t.size(1) != 1 && t.stride(0) != t.stride(1) * t.size(1)) return false;
    strides[0] = dim == 4 && t.size(1) == 1 ? t.stride(0) : t.stride(dim - 3);
    strides[1] = t.stride(dim - 2);
    return true;
}

// q, positions, inv_freq, axes, k, interleaved, inverse, q_out, k_out -> q_out or (q_out, k_out)
PyObject* rotary(PyObject*, PyObject* const* a, Py_ssize_t n) {
    try {
        if (n != 9 || !PyBool_Check(a[5]) || !PyBool_Check(a[6])) return not_here();
        const at::Tensor *q = tensor(a[0]), *pos = tensor(a[1]), *freq = tensor(a[2]), *axes = tensor(a[3]);
        const at::Tensor* k = a[4] == Py_None ? nullptr : tensor(a[4]);
        int dtype = 0;
        if (q == nullptr || pos == nullptr || !q->is_cuda() || (a[4] != Py_None && k == nullptr) || !half_type(*q, &dtype))
            return not_here();
        const c10::Device dev = q->device();
        const int64_t dim = q->dim();
        if (dev.index() != c10::cuda::current_device() || (dim != 3 && dim != 4) || q->numel() == 0 ||
            !plain(pos, at::kInt, dev) || !plain(freq, at::kDouble, dev) || !plain(axes, at::kInt, dev) ||
            pos->dim() != dim - 1 || freq->dim() != 1 || axes->dim() != 1 || freq->size(0) != axes->size(0))
            return not_here();
        const int64_t A = pos->size(dim - 2), F = freq->size(0), H = q->size(dim - 2), D = q->size(dim - 1);
        int64_t T = 1;
        for (int64_t i = 0; i < dim - 2; ++i) {
            if (pos->size(i) != q->size(i)) return not_here();
            T *= q->size(i);
        }
        if (A < 1 || F < 1 || 2 * F > D || !fits(T) || !fits(H) || !fits(D) || !fits(A)) return not_here();
        if (k != nullptr) {
            if (k->dim() != dim || k->scalar_type() != q->scalar_type() || k->device() != dev || k->numel() == 0 ||
                k->size(dim - 1) != D || !fits(k->size(dim - 2)))
                return not_here();
            for (int64_t i = 0; i < dim - 2; ++i)
                if (k->size(i) != q->size(i)) return not_here();
        }
        const at::Tensor* in[2] = {q, k};
        at::Tensor out[2];
        long long xs[2][2] = {}, ys[2][2] = {};
        for (int i = 0; i < 2; ++i) {
            PyObject* o = a[7 + i];
            if (in[i] == nullptr) {
                if (o != Py_None) return not_here();
                continue;
            }
            if (o != Py_None) {
                const at::Tensor* t = tensor(o);
                if (t == nullptr || t->sizes() != in[i]->sizes() || t->scalar_type() != in[i]->scalar_type() || t->device() != dev)
                    return not_here();
                out[i] = *t;
            } else {
                out[i] = at::empty(in[i]->sizes(), in[i]->options());
            }
            if (!tokens_of(*in[i], xs[i]) || !tokens_of(out[i], ys[i])) return not_here();
        }
        const int rc = p_rotary(q->data_ptr(), xs[0], out[0].data_ptr(), ys[0], static_cast<int>(H),
                                k != nullptr ? k->data_ptr() : nullptr, xs[1], k != nullptr ? out[1].data_ptr() : nullptr, ys[1],
                                k != nullptr ? static_cast<int>(k->size(dim - 2)) : 0, static_cast<const int*>(pos->data_ptr()),
                                static_cast<const double*>(freq->data_ptr()), static_cast<const int*>(axes->data_ptr()),
                                static_cast<int>(T), static_cast<int>(A), static_cast<int>(F), static_cast<int>(D),
                                a[5] == Py_True, a[6] == Py_True, dtype, stream_of(dev));
        if (rc != FA_OK) return PyLong_FromLong(rc);
        PyObject* y = THPVariable_Wrap(std::move(out[0]));
        return k == nullptr ? y : Py_BuildValue("(NN)", y, THPVariable_Wrap(std::move(out[1])));
    } catch (...) {
        return not_here();
    }
}

// init(address of fa_kv4_write, fa_kv4_read, fa_kv4_attention_workspace_size, fa_kv4_attention, fa_rotary)
PyObject* init(PyObject*, PyObject* const* a, Py_ssize_t n) {
    if (n != 5) {
        PyErr_SetString(PyExc_TypeError, "init takes five addresses");
        return nullptr;
    }
    void* p[5];
    for (int i = 0; i < 5; ++i) {
        p[i] = PyLong_AsVoidPtr(a[i]);
        if (p[i] == nullptr) {
            if (!PyErr_Occurred()) PyErr_SetString(PyExc_ValueError, "a null address");
            return nullptr;
        }
    }
    p_write = reinterpret_cast<decltype(p_write)>(p[0]);
    p_read = reinterpret_cast<decltype(p_read)>(p[1]);
    p_workspace = reinterpret_cast<decltype(p_workspace)>(p[2]);
    p_attention = reinterpret_cast<decltype(p_attention)>(p[3]);
    p_rotary = reinterpret_cast<decltype(p_rotary)>(p[4]);
    Py_RETURN_NONE;
}

#define FAST(f) {#f, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(f)), METH_FASTCALL, nullptr}
PyMethodDef methods[] = {FAST(init), FAST(kv4_write), FAST(kv4_read), FAST(kv4_attention), FAST(rotary),
                         {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "fa_binding", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit_fa_binding() { return PyModule_Create(&module); }
