// qar_torch.cpp -- the serving calls of include/qar.h on torch tensors, a
// Python extension module (block_wise_int8_amd/_qar_torch.so).
//
// These calls are short: a token's append, attention or product takes 3 to 10
// us on the GPU, so what the host does before a launch is most of the time.
// The same steps in Python through ctypes (checks, allocation of outputs and
// workspaces, marshalling) took 7 to 9 us a call.
//
// Each function either makes its call, or, where an argument does not fit it
// (another type, shape or device, not contiguous), returns None with nothing
// enqueued; qar.py then finds out which and raises.  A status other than
// QAR_OK comes back as an int.
#include <torch/csrc/Dtype.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include <ATen/hip/EmptyTensor.h>
#include <c10/hip/HIPFunctions.h>
#include <c10/hip/HIPStream.h>

#include <cmath>

#include "qar.h"

namespace {

struct Refused {};

void require(bool ok) {
    if (!ok) throw Refused{};
}

// ---------------------------------------------------------------------------
// arguments

const at::Tensor& tensor(PyObject* o) {
    require(THPVariable_Check(o));
    return THPVariable_Unpack(o);
}

uint32_t u32(int64_t v) {
    require(v >= 0 && v <= UINT32_MAX);
    return (uint32_t)v;
}

// Python's whole numbers and NumPy's.  A truth value is none (as in qar.py), and
// a tensor would be waited for.
int64_t whole(PyObject* o) {
    require(!PyBool_Check(o) && !THPVariable_Check(o));
    PyObject* n = PyNumber_Index(o);
    if (!n) {
        PyErr_Clear();
        throw Refused{};
    }
    const int64_t v = PyLong_AsLongLong(n);
    Py_DECREF(n);
    if (v == -1 && PyErr_Occurred()) {
        PyErr_Clear();
        throw Refused{};
    }
    return v;
}

at::ScalarType dtype_of(PyObject* o) {
    require(THPDtype_Check(o));
    return reinterpret_cast<THPDtype*>(o)->scalar_type;
}

qar_dtype data_code(at::ScalarType t) {
    require(t == at::kBFloat16 || t == at::kFloat);
    return t == at::kBFloat16 ? QAR_BF16 : QAR_F32;
}

// The GPU that a call runs on: its first tensor's, which has to be the current one.
struct Gpu {
    c10::Device device;
    void* stream;
    explicit Gpu(const at::Tensor& first) : device(first.device()) {
        require(device.is_cuda() && device.index() == c10::hip::current_device());
        stream = c10::hip::getCurrentHIPStream(device.index()).stream();
    }
    const at::Tensor& check(const at::Tensor& t) const {
        require(t.device() == device && t.is_contiguous());
        return t;
    }
    const at::Tensor& check(const at::Tensor& t, at::ScalarType type) const {
        require(t.scalar_type() == type);
        return check(t);
    }
    // contiguous, of this type and shape
    void* shaped(const at::Tensor& t, at::ScalarType type, at::IntArrayRef shape) const {
        check(t, type);
        require(t.sizes() == shape);
        return t.data_ptr();
    }
    // contiguous, of this type, with so many elements
    void* filled(const at::Tensor& t, at::ScalarType type, int64_t numel) const {
        check(t, type);
        require(t.numel() == numel);
        return t.data_ptr();
    }
    at::Tensor empty(at::IntArrayRef shape, at::ScalarType type) const {
        return at::Tensor(at::detail::empty_cuda(shape, type, device, std::nullopt));
    }
};

// The caller's workspace or a new one, whose memory the allocator hands out
// again only behind the work already on this stream.
struct Workspace {
    at::Tensor held;
    void* data = nullptr;
    size_t bytes = 0;
    Workspace(const Gpu& gpu, PyObject* given, size_t need) {
        if (given == Py_None) {
            if (!need) return;
            held = gpu.empty({(int64_t)need}, at::kByte);
        } else {
            held = gpu.check(tensor(given));
        }
        data = held.data_ptr();
        bytes = held.nbytes();
    }
};

// ---------------------------------------------------------------------------
// results

struct Released {
    PyThreadState* state = PyEval_SaveThread();
    ~Released() { PyEval_RestoreThread(state); }
};

template <class F>
qar_status made(F f) {
    Released other_threads_run;
    return f();
}

PyObject* status(qar_status st) { return PyLong_FromLong(st); }

PyObject* result(qar_status st, const at::Tensor& t) { return st == QAR_OK ? THPVariable_Wrap(t) : status(st); }

PyObject* result(qar_status st, const at::Tensor& a, const at::Tensor& b) {
    if (st != QAR_OK) return status(st);
    PyObject* pair = PyTuple_New(2);
    if (!pair) return nullptr;
    PyTuple_SET_ITEM(pair, 0, THPVariable_Wrap(a));
    PyTuple_SET_ITEM(pair, 1, THPVariable_Wrap(b));
    return pair;
}

// ---------------------------------------------------------------------------
// the cache: a KvCache object's six tensors

constexpr const char* kFields[6] = {"k", "k_scales", "v", "v_scales", "page_table", "lengths"};
PyObject* field_names[6];

struct Cache {
    at::Tensor t[6];
    qar_kv8_cache c;
    explicit Cache(PyObject* o) {
        for (int i = 0; i < 6; ++i) {
            PyObject* field = PyObject_GetAttr(o, field_names[i]);
            if (!field) {
                PyErr_Clear();
                throw Refused{};
            }
            const bool is_tensor = THPVariable_Check(field);
            if (is_tensor) t[i] = THPVariable_Unpack(field);
            Py_DECREF(field);
            require(is_tensor);
        }
        require(t[0].dim() == 4 && t[0].size(2) == QAR_KV8_PAGE && t[4].dim() == 2);
        c.pages = u32(t[0].size(0)), c.kv_heads = u32(t[0].size(1)), c.dim = u32(t[0].size(3));
        c.batch = u32(t[4].size(0)), c.table_width = u32(t[4].size(1));
    }
    void fill(const Gpu& gpu) {
        const int64_t flat = (int64_t)c.pages * c.kv_heads;
        c.k = (int8_t*)gpu.check(t[0], at::kChar).data_ptr();
        c.k_scales = (float*)gpu.filled(t[1], at::kFloat, flat);
        c.v = (int8_t*)gpu.shaped(t[2], at::kChar, {c.pages, c.kv_heads, c.dim, QAR_KV8_PAGE});
        c.v_scales = (float*)gpu.filled(t[3], at::kFloat, flat);
        c.page_table = (const int32_t*)gpu.check(t[4], at::kInt).data_ptr();
        c.lengths = (int32_t*)gpu.filled(t[5], at::kInt, c.batch);
    }
};

// cache, starts, k_new, v_new
PyObject* kv8_append(PyObject* const* a) {
    Cache cache(a[0]);
    const Gpu gpu(cache.t[0]);
    cache.fill(gpu);
    const at::Tensor &starts = tensor(a[1]), &k = tensor(a[2]), &v = tensor(a[3]);
    require(k.dim() == 4);
    const qar_kv8_cache& c = cache.c;
    const uint32_t tokens = u32(k.size(1));
    const int64_t shape[4] = {c.batch, tokens, c.kv_heads, c.dim};
    const at::ScalarType type = k.scalar_type();
    const qar_dtype code = data_code(type);
    const void *kp = gpu.shaped(k, type, shape), *vp = gpu.shaped(v, type, shape);
    const int32_t* sp = (const int32_t*)gpu.shaped(starts, at::kInt, {c.batch});
    return status(made([&] { return qar_kv8_append(&c, sp, kp, vp, code, tokens, gpu.stream); }));
}

// cache, starts, tokens, out_dtype, out (None or a pair)
PyObject* kv8_read(PyObject* const* a) {
    Cache cache(a[0]);
    const Gpu gpu(cache.t[0]);
    cache.fill(gpu);
    const qar_kv8_cache& c = cache.c;
    const uint32_t tokens = u32(whole(a[2]));
    const int32_t* sp = (const int32_t*)gpu.shaped(tensor(a[1]), at::kInt, {c.batch});
    const int64_t shape[4] = {c.batch, tokens, c.kv_heads, c.dim};
    at::Tensor k, v;
    qar_dtype code;
    if (a[4] == Py_None) {
        const at::ScalarType type = dtype_of(a[3]);
        code = data_code(type);
        k = gpu.empty(shape, type);
        v = gpu.empty(shape, type);
    } else {
        require(PyTuple_Check(a[4]) && PyTuple_GET_SIZE(a[4]) == 2);
        k = tensor(PyTuple_GET_ITEM(a[4], 0));
        v = tensor(PyTuple_GET_ITEM(a[4], 1));
        code = data_code(k.scalar_type());
        gpu.shaped(k, k.scalar_type(), shape);
        gpu.shaped(v, k.scalar_type(), shape);
    }
    void *kp = k.data_ptr(), *vp = v.data_ptr();
    return result(made([&] { return qar_kv8_read(&c, sp, tokens, kp, vp, code, gpu.stream); }), k, v);
}

// cache, q, q_lens, scale, weights, out, workspace (all but the first two may be None)
PyObject* kv8_attention(PyObject* const* a) {
    Cache cache(a[0]);
    const Gpu gpu(cache.t[0]);
    cache.fill(gpu);
    const qar_kv8_cache& c = cache.c;
    const at::Tensor& q = tensor(a[1]);
    require(q.dim() == 4);
    const uint32_t queries = u32(q.size(1)), heads = u32(q.size(2));
    const int64_t shape[4] = {c.batch, queries, heads, c.dim};
    const at::ScalarType type = q.scalar_type();
    const qar_dtype code = data_code(type);
    const void* qp = gpu.shaped(q, type, shape);
    const int32_t* lens = nullptr;
    if (a[2] != Py_None) lens = (const int32_t*)gpu.shaped(tensor(a[2]), at::kInt, {c.batch});
    float scale = (float)(1.0 / std::sqrt((double)c.dim));
    if (a[3] != Py_None) {
        const double given = PyFloat_AsDouble(a[3]);
        if (given == -1.0 && PyErr_Occurred()) {
            PyErr_Clear();
            throw Refused{};
        }
        scale = (float)given;
    }
    float* weights = nullptr;
    if (a[4] != Py_None)
        weights = (float*)gpu.shaped(tensor(a[4]), at::kFloat, {c.batch, c.kv_heads, (int64_t)c.table_width * QAR_KV8_PAGE});
    at::Tensor out;
    if (a[5] == Py_None)
        out = gpu.empty(shape, type);
    else
        gpu.shaped(out = tensor(a[5]), type, shape);
    const Workspace ws(gpu, a[6], qar_kv8_attention_workspace_bytes(c.batch, queries, heads, c.kv_heads, c.dim,
                                                                    c.table_width, code, weights != nullptr));
    void* op = out.data_ptr();
    return result(made([&] {
                      return qar_kv8_attention(&c, qp, code, queries, heads, lens, scale, weights, op, ws.data, ws.bytes,
                                               gpu.stream);
                  }),
                  out);
}

// cache, into, weights, recent, keep, kept, moved (the last two may be None)
PyObject* kv8_evict(PyObject* const* a) {
    Cache cache(a[0]), into(a[1]);
    const Gpu gpu(cache.t[0]);
    cache.fill(gpu);
    into.fill(gpu);
    const qar_kv8_cache& c = cache.c;
    const uint32_t recent = u32(whole(a[3])), keep = u32(whole(a[4]));
    require(keep >= 1 && keep <= INT32_MAX);
    const float* wp =
        (const float*)gpu.shaped(tensor(a[2]), at::kFloat, {c.batch, c.kv_heads, (int64_t)c.table_width * QAR_KV8_PAGE});
    const int64_t shape[3] = {c.batch, c.kv_heads, keep};
    at::Tensor kept, moved;
    if (a[5] == Py_None)
        kept = gpu.empty(shape, at::kInt);
    else
        gpu.shaped(kept = tensor(a[5]), at::kInt, shape);
    if (a[6] == Py_None)
        moved = gpu.empty(shape, at::kFloat);
    else
        gpu.shaped(moved = tensor(a[6]), at::kFloat, shape);
    int32_t* kp = (int32_t*)kept.data_ptr();
    float* mp = (float*)moved.data_ptr();
    return result(made([&] { return qar_kv8_evict(&c, &into.c, wp, recent, keep, kp, mp, gpu.stream); }), kept, moved);
}

// ---------------------------------------------------------------------------
// microscaled 4-bit

int64_t mx4_blocks(int64_t cols) { return (cols + QAR_MX4_BLOCK - 1) / QAR_MX4_BLOCK; }

// x, codes, scales (the last two may be None)
PyObject* mx4_quantize(PyObject* const* a) {
    const at::Tensor& x = tensor(a[0]);
    const Gpu gpu(x);
    gpu.check(x);
    require(x.dim() == 2);
    const qar_dtype code = data_code(x.scalar_type());
    const int64_t rows = x.size(0), cols = x.size(1), nb = mx4_blocks(cols);
    at::Tensor codes, scales;
    if (a[1] == Py_None)
        codes = gpu.empty({rows, nb * 16}, at::kByte);
    else
        gpu.filled(codes = tensor(a[1]), at::kByte, rows * nb * 16);
    if (a[2] == Py_None)
        scales = gpu.empty({rows, nb}, at::kByte);
    else
        gpu.filled(scales = tensor(a[2]), at::kByte, rows * nb);
    const void* xp = x.data_ptr();
    uint8_t *cp = (uint8_t*)codes.data_ptr(), *sp = (uint8_t*)scales.data_ptr();
    return result(made([&] { return qar_mx4_quantize(xp, code, rows, cols, cp, sp, gpu.stream); }), codes, scales);
}

// The codes and scales of `rows` rows of nb blocks.
struct Mx4 {
    const uint8_t *codes, *scales;
    Mx4(const Gpu& gpu, const at::Tensor& c, PyObject* s, int64_t nb) {
        codes = (const uint8_t*)gpu.filled(c, at::kByte, c.size(0) * nb * 16);
        scales = (const uint8_t*)gpu.filled(tensor(s), at::kByte, c.size(0) * nb);
    }
};

// codes, scales, cols, out (or None), out_dtype
PyObject* mx4_dequantize(PyObject* const* a) {
    const at::Tensor& c = tensor(a[0]);
    const Gpu gpu(c);
    require(c.dim() == 2);
    const int64_t rows = c.size(0), cols = whole(a[2]);
    require(cols >= 0);
    const Mx4 m(gpu, c, a[1], mx4_blocks(cols));
    at::Tensor out;
    if (a[3] == Py_None) {
        const at::ScalarType type = dtype_of(a[4]);
        data_code(type);
        out = gpu.empty({rows, cols}, type);
    } else {
        out = tensor(a[3]);
        gpu.filled(out, out.scalar_type(), rows * cols);
    }
    const qar_dtype code = data_code(out.scalar_type());
    void* op = out.data_ptr();
    return result(made([&] { return qar_mx4_dequantize(m.codes, m.scales, rows, cols, op, code, gpu.stream); }), out);
}

// x, codes, scales, out, out_dtype, workspace (the last three may be None)
PyObject* mx4_linear(PyObject* const* a) {
    const at::Tensor &x = tensor(a[0]), &c = tensor(a[1]);
    const Gpu gpu(x);
    gpu.check(x);
    require(x.dim() == 2 && c.dim() == 2);
    const int64_t rows = x.size(0), inner = x.size(1), cols = c.size(0);
    const qar_dtype code = data_code(x.scalar_type());
    const Mx4 m(gpu, c, a[2], mx4_blocks(inner));
    at::Tensor out;
    if (a[3] == Py_None) {
        const at::ScalarType type = a[4] == Py_None ? x.scalar_type() : dtype_of(a[4]);
        data_code(type);
        out = gpu.empty({rows, cols}, type);
    } else {
        out = tensor(a[3]);
        gpu.filled(out, out.scalar_type(), rows * cols);
    }
    const qar_dtype out_code = data_code(out.scalar_type());
    const Workspace ws(gpu, a[5], qar_mx4_linear_workspace_bytes(rows, inner, cols));
    const void* xp = x.data_ptr();
    void* op = out.data_ptr();
    return result(made([&] {
                      return qar_mx4_linear(xp, code, rows, inner, m.codes, m.scales, cols, op, out_code, ws.data, ws.bytes,
                                            gpu.stream);
                  }),
                  out);
}

// ---------------------------------------------------------------------------
// the module

// No C++ exception leaves: what torch throws (no memory left) becomes the
// Python exception that it is there.
template <PyObject* (*F)(PyObject* const*), int N>
PyObject* entry(PyObject*, PyObject* const* args, Py_ssize_t count) {
    HANDLE_TH_ERRORS
    if (count != N) {
        PyErr_Format(PyExc_TypeError, "%d arguments expected, not %zd", N, count);
        return nullptr;
    }
    try {
        return F(args);
    } catch (const Refused&) {
        Py_RETURN_NONE;
    }
    END_HANDLE_TH_ERRORS
}

template <PyObject* (*F)(PyObject* const*), int N>
PyMethodDef method(const char* name) {
    return {name, (PyCFunction)(void (*)(void))entry<F, N>, METH_FASTCALL, nullptr};
}

PyMethodDef methods[] = {method<kv8_append, 4>("kv8_append"),         method<kv8_read, 5>("kv8_read"),
                         method<kv8_attention, 7>("kv8_attention"),   method<kv8_evict, 7>("kv8_evict"),
                         method<mx4_quantize, 3>("mx4_quantize"),     method<mx4_dequantize, 5>("mx4_dequantize"),
                         method<mx4_linear, 6>("mx4_linear"),         {nullptr, nullptr, 0, nullptr}};

PyModuleDef module = {PyModuleDef_HEAD_INIT, "_qar_torch", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

} // namespace

PyMODINIT_FUNC PyInit__qar_torch(void) {
    for (int i = 0; i < 6; ++i)
        if (!(field_names[i] = PyUnicode_InternFromString(kFields[i]))) return nullptr;
    return PyModule_Create(&module);
}
