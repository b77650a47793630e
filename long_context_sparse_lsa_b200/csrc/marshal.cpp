// marshal.cpp — the tensor checks and argument lists of binding.py's calls on
// 4-bit caches and whole prompts, compiled: checked in Python, the 11 to 30
// tensors of such a call cost 8 to 24 us, more than most of these kernels run
// (a decode store 16 us a call, 6 us this way; its kernel takes 3).
//
// binding.py hands over the address of the C-ABI function (this module is not
// linked to liblsa.so), the caller's tensors as they are, and gets the status
// back. Wrong types and layouts raise TypeError, wrong sizes and devices
// ValueError, before anything is launched.
#define PY_SSIZE_T_CLEAN
#include <Python.h>
#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/autograd/python_variable.h>

#include <cstring>
#include <string>
#include <vector>

#include "built_for.h"  // written by the build
#include "lsa.h"

namespace {

struct Refusal {
    PyObject* type;
    std::string text;
};
struct PythonError {};  // a Python exception is set

[[noreturn]] void type_error(const std::string& s) { throw Refusal{PyExc_TypeError, s}; }
[[noreturn]] void value_error(const std::string& s) { throw Refusal{PyExc_ValueError, s}; }

const at::Tensor& tensor(const char* name, PyObject* o) {
    if (!THPVariable_Check(o)) type_error(std::string(name) + " must be a tensor");
    const at::Tensor& t = THPVariable_Unpack(o);
    if (t.layout() != c10::kStrided) type_error(std::string(name) + " must be a strided tensor");
    return t;
}

int64_t integer(PyObject* o) {
    const long long v = PyLong_AsLongLong(o);
    if (v == -1 && PyErr_Occurred()) throw PythonError{};
    return v;
}
int32_t integer32(const char* name, PyObject* o) {
    const int64_t v = integer(o);
    if (v < INT32_MIN || v > INT32_MAX) value_error(std::string(name) + " does not fit 32 bits");
    return (int32_t)v;
}

// The device of the call: that of its first tensor, which has to be the
// current one; every other tensor is held to it.
struct Device {
    int dev = -2;
    void* use(const at::Tensor& t) {
        const int d = t.is_cuda() ? (int)t.get_device() : -1;
        if (dev == -2) {
            if (d < 0 || d != (int)c10::cuda::current_device()) value_error("tensors must be on the current CUDA device");
            dev = d;
        } else if (d != dev) {
            value_error("tensors must be on the current CUDA device");
        }
        return t.data_ptr();
    }
    void* stream(PyObject* o) const {
        if (o == Py_None) return c10::cuda::getCurrentCUDAStream((c10::DeviceIndex)dev).stream();
        if (PyLong_Check(o)) return reinterpret_cast<void*>((uintptr_t)integer(o));
        PyObject* raw = PyObject_GetAttrString(o, "cuda_stream");
        if (raw == nullptr) throw PythonError{};
        const long long v = PyLong_AsLongLong(raw);
        Py_DECREF(raw);
        if (v == -1 && PyErr_Occurred()) throw PythonError{};
        return reinterpret_cast<void*>((uintptr_t)v);
    }
};

// What a call's tensors are checked for: shape and layout first, for all of
// them, then the devices (a call on host tensors of a wrong shape names the shape).
struct Lists {
    Device where;
    std::vector<const at::Tensor*> seen;
    int layers = 0;

    const at::Tensor& note(const at::Tensor& t) {
        seen.push_back(&t);
        return t;
    }
    // a sequence's items (borrowed: the caller's frame holds the sequence)
    static PyObject* const* items(const char* name, PyObject* o, int* n) {
        if (!PyList_Check(o) && !PyTuple_Check(o)) type_error(std::string(name) + " must be a list, one tensor per layer");
        *n = (int)PySequence_Fast_GET_SIZE(o);
        return PySequence_Fast_ITEMS(o);
    }
    const at::Tensor& first(const char* name, PyObject* o) {
        PyObject* const* it = items(name, o, &layers);
        if (layers < 1 || layers > LSA_MAX_LAYERS) value_error("1 to 8 layers");
        return tensor(name, it[0]);
    }
    // contiguous tensors of one shape, one per layer
    template <class T>
    void whole(const char* name, PyObject* o, at::ScalarType dtype, at::IntArrayRef shape, T** ptrs) {
        int n;
        PyObject* const* it = items(name, o, &n);
        if (n != layers) value_error(std::string(name) + " must hold one tensor per layer");
        for (int g = 0; g < n; ++g) {
            const at::Tensor& t = note(tensor(name, it[g]));
            if (t.scalar_type() != dtype || t.sizes() != shape || !t.is_contiguous())
                type_error(std::string(name) + " must hold contiguous tensors of one type and shape");
            ptrs[g] = static_cast<T*>(t.data_ptr());
        }
    }
    // bf16 [rows, H, d] views with one row stride
    int64_t rows(const char* name, PyObject* o, at::IntArrayRef shape, const uint16_t** ptrs) {
        int n;
        int64_t stride = -1;
        PyObject* const* it = items(name, o, &n);
        if (n != layers) value_error(std::string(name) + " must hold one tensor per layer");
        for (int g = 0; g < n; ++g) {
            const at::Tensor& t = note(tensor(name, it[g]));
            if (t.scalar_type() != at::kBFloat16 || t.sizes() != shape)
                type_error(std::string(name) + " must hold bfloat16 tensors of one shape");
            const int64_t s = row_stride(name, t);
            if (g > 0 && s != stride) value_error(std::string(name) + ": every layer must have the same row stride");
            stride = s;
            ptrs[g] = static_cast<const uint16_t*>(t.data_ptr());
        }
        return stride;
    }
    // elements from one token to the next of a [tokens, H, d] view whose heads are contiguous
    static int64_t row_stride(const char* name, const at::Tensor& t) {
        const int64_t H = t.size(1), d = t.size(2);
        if (t.stride(2) != 1 || (H > 1 && t.stride(1) != d))
            value_error(std::string(name) + ": the heads of a token must be contiguous");
        return t.size(0) > 1 ? t.stride(0) : H * d;
    }
    template <class T>
    T* flat(const char* name, PyObject* o, at::ScalarType dtype, int64_t* n) {
        const at::Tensor& t = note(tensor(name, o));
        if (t.scalar_type() != dtype || !t.is_contiguous()) type_error(std::string(name) + " must be a contiguous tensor of its type");
        *n = t.numel();
        return static_cast<T*>(t.data_ptr());
    }
    void* optional(const char* name, PyObject* o, size_t* bytes) {
        *bytes = 0;
        if (o == Py_None) return nullptr;
        const at::Tensor& t = note(tensor(name, o));
        // (an expanded tensor has fewer bytes behind its address than elements)
        if (!t.is_contiguous()) type_error(std::string(name) + " must be a contiguous tensor");
        *bytes = (size_t)t.nbytes();
        return t.data_ptr();
    }
    int32_t* status(PyObject* o) {
        if (o == Py_None) return nullptr;
        const at::Tensor& t = note(tensor("dev_status", o));
        if (t.scalar_type() != at::kInt || t.numel() < 1) type_error("dev_status must be an int32 tensor");
        return static_cast<int32_t*>(t.data_ptr());
    }
    void scales(const char* name, PyObject* o, float* to) {
        int n;
        PyObject* const* it = items(name, o, &n);
        if (n != layers) value_error("k_scale and v_scale must hold one scale per layer");
        for (int g = 0; g < n; ++g) {
            const double v = PyFloat_AsDouble(it[g]);
            if (v == -1.0 && PyErr_Occurred()) throw PythonError{};
            to[g] = (float)v;
        }
    }
    // args: row_offset, kv_offset, seq_lens, n_rows, max_len, total_tokens
    lsa_prompts_t prompts(PyObject* const* a) {
        lsa_prompts_t p;
        std::memset(&p, 0, sizeof p);
        int64_t nr, nk, ns;
        p.row_offset = flat<int32_t>("row_offset", a[0], at::kInt, &nr);
        p.kv_offset = flat<int64_t>("kv_offset", a[1], at::kLong, &nk);
        p.seq_lens = flat<int32_t>("seq_lens", a[2], at::kInt, &ns);
        if (nr != ns + 1 || nk != ns) value_error("row_offset must hold n_seq + 1 values, kv_offset and seq_lens n_seq");
        if (ns > INT32_MAX) value_error("too many sequences");
        p.n_seq = (int32_t)ns;
        p.n_rows = integer32("n_rows", a[3]);
        p.max_len = integer32("max_len", a[4]);
        p.total_tokens = integer(a[5]);
        return p;
    }
    void* finish(PyObject* stream) {
        for (const at::Tensor* t : seen) where.use(*t);
        return where.stream(stream);
    }
};

template <class F>
PyObject* guarded(Py_ssize_t n_args, Py_ssize_t want, F&& f) {
    if (n_args != want) {
        PyErr_SetString(PyExc_TypeError, "wrong number of arguments");
        return nullptr;
    }
    try {
        return PyLong_FromLong(f());
    } catch (const Refusal& r) {
        PyErr_SetString(r.type, r.text.c_str());
    } catch (const PythonError&) {
    } catch (const std::exception& e) {
        PyErr_SetString(PyExc_RuntimeError, e.what());
    }
    return nullptr;
}

template <class F>
F function(PyObject* o) {
    return reinterpret_cast<F>((uintptr_t)integer(o));
}
template <class F>
long unlocked(F&& f) {
    long st;
    Py_BEGIN_ALLOW_THREADS
    st = f();
    Py_END_ALLOW_THREADS
    return st;
}

// address, k_new, v_new, k, k_group, v, v_group, k_scale, v_scale, prompts (6), k_round, v_round, dev_status, stream
PyObject* store_fp4(PyObject*, PyObject* const* a, Py_ssize_t n) {
    return guarded(n, 19, [&]() -> long {
        Lists x;
        const auto fn = function<decltype(&lsa_store_fp4)>(a[0]);
        const at::Tensor& first = x.first("k_new", a[1]);
        if (first.dim() != 3) type_error("k_new must hold [n_rows, H_kv, d] tensors");
        const std::vector<int64_t> rows = first.sizes().vec();
        const uint16_t *kn[LSA_MAX_LAYERS], *vn[LSA_MAX_LAYERS];
        uint16_t *kr[LSA_MAX_LAYERS], *vr[LSA_MAX_LAYERS];
        uint8_t *k[LSA_MAX_LAYERS], *kg[LSA_MAX_LAYERS], *v[LSA_MAX_LAYERS], *vg[LSA_MAX_LAYERS];
        float ks[LSA_MAX_LAYERS], vs[LSA_MAX_LAYERS];
        const int64_t k_stride = x.rows("k_new", a[1], rows, kn), v_stride = x.rows("v_new", a[2], rows, vn);
        int n_k;
        PyObject* const* k_items = Lists::items("k", a[3], &n_k);
        if (n_k < 1) value_error("k must hold one tensor per layer");
        const at::Tensor& k0 = tensor("k", k_items[0]);
        if (k0.dim() != 3) type_error("k must hold [T, H_kv, d / 2] tensors");
        const int64_t T = k0.size(0), H = rows[1], d = rows[2];
        const lsa_prompts_t p = x.prompts(a + 9);
        if (rows[0] != p.n_rows || T < p.total_tokens)
            value_error("k_new must hold prompts.n_rows rows and the caches prompts.total_tokens");
        if (H > INT32_MAX || d > INT32_MAX) value_error("too many heads or channels");
        x.whole("k", a[3], at::kByte, {T, H, d / 2}, k);
        x.whole("k_group", a[4], at::kByte, {T, H, d / 16}, kg);
        x.whole("v", a[5], at::kByte, {T, H, d / 2}, v);
        x.whole("v_group", a[6], at::kByte, {T, H, d / 16}, vg);
        x.scales("k_scale", a[7], ks);
        x.scales("v_scale", a[8], vs);
        const bool round = a[15] != Py_None;
        if (round != (a[16] != Py_None)) value_error("k_round and v_round come together");
        if (round) {
            x.whole("k_round", a[15], at::kBFloat16, rows, kr);
            x.whole("v_round", a[16], at::kBFloat16, rows, vr);
        }
        int32_t* status = x.status(a[17]);
        void* stream = x.finish(a[18]);
        return unlocked([&] {
            return (long)fn(kn, k_stride, vn, v_stride, (int32_t)H, (int32_t)d, &p, x.layers, ks, vs, k, kg, v, vg,
                            round ? kr : nullptr, round ? vr : nullptr, status, stream);
        });
    });
}

// address, q, k, k_group, v, v_group, k_scale, v_scale, index_sets, kv_offset, seq_lens, q_seq, q_len, max_len,
// total_tokens, out, workspace, dev_status, stream
PyObject* attend_fp4(PyObject*, PyObject* const* a, Py_ssize_t n) {
    return guarded(n, 19, [&]() -> long {
        Lists x;
        const auto fn = function<decltype(&lsa_attend_fp4)>(a[0]);
        const at::Tensor& first = x.first("q", a[1]);
        if (first.dim() != 3) type_error("q must hold [n_q, H_q, d] tensors");
        const std::vector<int64_t> rows = first.sizes().vec();
        const uint16_t* q[LSA_MAX_LAYERS];
        const uint8_t *k[LSA_MAX_LAYERS], *kg[LSA_MAX_LAYERS], *v[LSA_MAX_LAYERS], *vg[LSA_MAX_LAYERS];
        float* out[LSA_MAX_LAYERS];
        float ks[LSA_MAX_LAYERS], vs[LSA_MAX_LAYERS];
        x.whole("q", a[1], at::kBFloat16, rows, q);
        int n_k;
        PyObject* const* k_items = Lists::items("k", a[2], &n_k);
        if (n_k < 1) value_error("k must hold one tensor per layer");
        const at::Tensor& k0 = tensor("k", k_items[0]);
        if (k0.dim() != 3) type_error("k must hold [T, H_kv, d / 2] tensors");
        const int64_t T = k0.size(0), H_kv = k0.size(1), d = rows[2];
        if (H_kv > INT32_MAX || rows[1] > INT32_MAX || d > INT32_MAX) value_error("too many heads or channels");
        const at::Tensor& sets = x.note(tensor("index_sets", a[8]));
        if (sets.scalar_type() != at::kInt || sets.dim() != 2 || !sets.is_contiguous() || sets.size(0) != rows[0] ||
            sets.size(1) > INT32_MAX)
            type_error("index_sets must be a contiguous int32 [n_q, budget] tensor");
        lsa_batch_t b;
        std::memset(&b, 0, sizeof b);
        int64_t nk, ns, nq, nl;
        b.kv_offset = x.flat<int64_t>("kv_offset", a[9], at::kLong, &nk);
        b.seq_lens = x.flat<int32_t>("seq_lens", a[10], at::kInt, &ns);
        b.q_seq = x.flat<int32_t>("q_seq", a[11], at::kInt, &nq);
        b.q_len = x.flat<int32_t>("q_len", a[12], at::kInt, &nl);
        if (nk != ns || nq != nl || ns > INT32_MAX || nq > INT32_MAX)
            value_error("kv_offset and seq_lens must hold n_seq values, q_seq and q_len n_q");
        b.n_seq = (int32_t)ns;
        b.n_q = (int32_t)nq;
        b.max_len = integer32("max_len", a[13]);
        b.total_tokens = integer(a[14]);
        if (T < b.total_tokens || nq != rows[0]) value_error("the caches must hold batch.total_tokens rows, q the batch's rows");
        x.whole("k", a[2], at::kByte, {T, H_kv, d / 2}, k);
        x.whole("k_group", a[3], at::kByte, {T, H_kv, d / 16}, kg);
        x.whole("v", a[4], at::kByte, {T, H_kv, d / 2}, v);
        x.whole("v_group", a[5], at::kByte, {T, H_kv, d / 16}, vg);
        x.scales("k_scale", a[6], ks);
        x.scales("v_scale", a[7], vs);
        x.whole("out", a[15], at::kFloat, rows, out);
        size_t ws_bytes;
        void* ws = x.optional("workspace", a[16], &ws_bytes);
        int32_t* status = x.status(a[17]);
        void* stream = x.finish(a[18]);
        return unlocked([&] {
            return (long)fn(q, k, kg, v, vg, ks, vs, (int32_t)rows[1], (int32_t)H_kv, (int32_t)d,
                            static_cast<const int32_t*>(sets.data_ptr()), (int32_t)sets.size(1), &b, x.layers, out, ws,
                            ws_bytes, status, stream);
        });
    });
}

uint16_t* bits(const at::Tensor& t) { return static_cast<uint16_t*>(t.data_ptr()); }

// address, q, k, v, prompts (6), out, workspace, lse, dev_status, stream
PyObject* attend_prompt(PyObject*, PyObject* const* a, Py_ssize_t n) {
    return guarded(n, 15, [&]() -> long {
        Lists x;
        const auto fn = function<decltype(&lsa_attend_prompt)>(a[0]);
        const at::Tensor &q = x.note(tensor("q", a[1])), &k = x.note(tensor("k", a[2])), &v = x.note(tensor("v", a[3])),
                         &out = x.note(tensor("out", a[10]));
        for (const at::Tensor* t : {&q, &k, &v, &out})
            if (t->scalar_type() != at::kBFloat16 || t->dim() != 3) type_error("q, k, v and out must be bfloat16 [rows, heads, d] tensors");
        const int64_t n_rows = q.size(0), H_q = q.size(1), d = q.size(2), T = k.size(0), H_kv = k.size(1);
        if (k.size(2) != d || v.sizes() != k.sizes() || out.sizes() != q.sizes() || !out.is_contiguous())
            value_error("k and v must be [T, H_kv, d], out contiguous [n_rows, H_q, d]");
        if (H_q > INT32_MAX || H_kv > INT32_MAX || d > INT32_MAX) value_error("too many heads or channels");
        const lsa_prompts_t p = x.prompts(a + 4);
        if (n_rows != p.n_rows || T < p.total_tokens) value_error("q must hold prompts.n_rows rows, k and v prompts.total_tokens");
        float* lse = nullptr;
        if (a[12] != Py_None) {
            const at::Tensor& t = x.note(tensor("lse", a[12]));
            if (t.scalar_type() != at::kFloat || t.dim() != 2 || t.size(0) != n_rows || t.size(1) != H_q || !t.is_contiguous())
                type_error("lse must be a contiguous float32 [n_rows, H_q] tensor");
            lse = static_cast<float*>(t.data_ptr());
        }
        const int64_t qs = Lists::row_stride("q", q), ks = Lists::row_stride("k", k), vs = Lists::row_stride("v", v);
        size_t ws_bytes;
        void* ws = x.optional("workspace", a[11], &ws_bytes);
        int32_t* status = x.status(a[13]);
        void* stream = x.finish(a[14]);
        return unlocked([&] {
            return (long)fn(bits(q), qs, bits(k), ks, bits(v), vs, (int32_t)H_q, (int32_t)H_kv, (int32_t)d, &p, bits(out), lse,
                            ws, ws_bytes, status, stream);
        });
    });
}

#define LSA_METHOD(name) {#name, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(name)), METH_FASTCALL, nullptr}
PyMethodDef methods[] = {LSA_METHOD(store_fp4), LSA_METHOD(attend_fp4), LSA_METHOD(attend_prompt), {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_marshal", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__marshal(void) {
    PyObject* m = PyModule_Create(&module);
    if (m != nullptr && PyModule_AddStringConstant(m, "built_for", LSA_BUILT_FOR) != 0) {
        Py_DECREF(m);
        return nullptr;
    }
    return m;
}
