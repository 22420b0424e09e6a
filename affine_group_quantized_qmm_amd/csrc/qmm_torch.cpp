// The step operators' Python calls: checks of the tensors and the call into the
// C ABI, compiled. A decode step makes these calls for every layer, with
// kernels of a few microseconds. One token through the norm and rotation takes
// 4 to 4.5 us a call, its kernel 3.0; with the same checks in Python it took 10.5.
// Nothing here computes or launches anything itself.
//
// Every function takes its arguments by position (the package's Python
// functions name and default them), raises TypeError or ValueError for a tensor
// that does not fit, and returns the output (the caller's, or a new tensor) or,
// where the C function refuses the call, its code.
#include <torch/csrc/autograd/python_variable.h>

#include <ATen/core/Tensor.h>
#include <ATen/ops/empty.h>

#include <cmath>
#include <initializer_list>
#include <stdexcept>
#include <string>

// the HIP runtime's stream type is all that the header needs of it
#include "qmm.h"

namespace {

struct Refused : std::runtime_error {
    PyObject *type;
    Refused(PyObject *t, const std::string &what) : std::runtime_error(what), type(t) {}
};

std::string shape_text(at::IntArrayRef s)
{
    std::string t = "(";
    for (size_t i = 0; i < s.size(); ++i)
        t += (i ? ", " : "") + std::to_string(s[i]);
    return t + ")";
}

const at::Tensor &tensor(PyObject *o, const char *name)
{
    if (!THPVariable_Check(o))
        throw Refused(PyExc_TypeError, std::string(name) + " must be a torch.Tensor");
    return THPVariable_Unpack(o);
}

int type_code(at::ScalarType t)
{
    return t == at::kHalf ? QMM_F16 : t == at::kBFloat16 ? QMM_BF16 : t == at::kFloat ? QMM_F32 : -1;
}

// What has to hold for every tensor of a call.
struct Call {
    c10::Device device;

    void fits(const at::Tensor &t, const char *name, at::ScalarType type, at::IntArrayRef shape) const
    {
        if (t.scalar_type() != type)
            throw Refused(PyExc_TypeError, std::string(name) + " must have dtype " + c10::toString(type) + ", got " +
                                               c10::toString(t.scalar_type()));
        if (t.device() != device)
            throw Refused(PyExc_ValueError, std::string(name) + " must be on the GPU device " + device.str() + ", got " +
                                                t.device().str());
        if (t.sizes() != shape)
            throw Refused(PyExc_ValueError, std::string(name) + " must have shape " + shape_text(shape) + ", got " +
                                                shape_text(t.sizes()));
    }
    void *whole(const at::Tensor &t, const char *name, at::ScalarType type, at::IntArrayRef shape) const
    {
        fits(t, name, type, shape);
        if (!t.is_contiguous())
            throw Refused(PyExc_ValueError, std::string(name) + " must be contiguous");
        return t.data_ptr();
    }
    void *whole(PyObject *o, const char *name, at::ScalarType type, std::initializer_list<int64_t> shape) const
    {
        return whole(tensor(o, name), name, type, at::IntArrayRef(shape.begin(), shape.size()));
    }
    void *whole_or_null(PyObject *o, const char *name, at::ScalarType type, std::initializer_list<int64_t> shape) const
    {
        return o == Py_None ? nullptr : whole(o, name, type, shape);
    }
    // Rows may lie apart; returns their distance.
    int64_t rows(const at::Tensor &t, const char *name, at::ScalarType type, at::IntArrayRef shape) const
    {
        fits(t, name, type, shape);
        int64_t dense = 1;
        for (int64_t i = (int64_t)shape.size() - 1; i > 0; --i) {
            if (shape[i] != 1 && t.stride(i) != dense)
                throw Refused(PyExc_ValueError, std::string(name) + " must be contiguous within a row");
            dense *= shape[i];
        }
        return shape[0] == 1 ? dense : t.stride(0);
    }
};

Call on_gpu(const at::Tensor &t, const char *name)
{
    if (!t.is_cuda())
        throw Refused(PyExc_ValueError, std::string(name) + " must be on the GPU, got " + t.device().str());
    return Call{t.device()};
}

int as_int(PyObject *o, const char *name)
{
    const long long v = PyLong_AsLongLong(o);
    if (v == -1 && PyErr_Occurred())
        throw Refused(nullptr, "");
    if (v < INT32_MIN || v > INT32_MAX)
        throw Refused(PyExc_ValueError, std::string(name) + " does not fit 32 bits");
    return (int)v;
}
float as_float(PyObject *o)
{
    const double v = PyFloat_AsDouble(o);
    if (v == -1.0 && PyErr_Occurred())
        throw Refused(nullptr, "");
    return (float)v;
}
hipStream_t as_stream(PyObject *o)
{
    void *p = PyLong_AsVoidPtr(o);
    if (!p && PyErr_Occurred())
        throw Refused(nullptr, "");
    return static_cast<hipStream_t>(p);
}

struct Caches {
    const at::Tensor &k, &v;
    int pages, Hkv, page_size;
    at::ScalarType type;
};
Caches caches(const Call &c, PyObject *ko, PyObject *vo, int64_t D)
{
    const at::Tensor &k = tensor(ko, "k_cache"), &v = tensor(vo, "v_cache");
    if (k.dim() != 4)
        throw Refused(PyExc_ValueError, "the caches must be 4-D [num_pages, Hkv, page_size, D]");
    const at::ScalarType type = k.scalar_type();
    if (type != at::kHalf && type != at::kBFloat16)
        throw Refused(PyExc_TypeError, std::string("the caches must be float16 or bfloat16, got ") + c10::toString(type));
    if (k.size(3) != D)
        throw Refused(PyExc_ValueError, "the caches' D is " + std::to_string(k.size(3)) + ", the queries' " +
                                            std::to_string(D));
    if (k.size(0) > INT32_MAX || k.size(1) > INT32_MAX || k.size(2) > INT32_MAX)
        throw Refused(PyExc_ValueError, "the caches' sizes do not fit 32 bits");
    c.whole(k, "k_cache", type, k.sizes());
    c.whole(v, "v_cache", type, k.sizes());
    return Caches{k, v, (int)k.size(0), (int)k.size(1), (int)k.size(2), type};
}

void args(Py_ssize_t n, Py_ssize_t want)
{
    if (n != want)
        throw Refused(PyExc_TypeError, "takes " + std::to_string(want) + " arguments");
}

// An output: the caller's, or a new tensor from torch's allocator.
struct Output {
    PyObject *given;
    at::Tensor t;
    void *data;
    Output(const Call &c, PyObject *o, const char *name, at::ScalarType type, std::initializer_list<int64_t> shape)
        : given(o)
    {
        const at::IntArrayRef s(shape.begin(), shape.size());
        if (o == Py_None) {
            t = at::empty(s, at::TensorOptions().dtype(type).device(c.device));
            data = t.data_ptr();
        } else {
            data = c.whole(tensor(o, name), name, type, s);
        }
    }
    PyObject *result(int code) const
    {
        if (code)
            return PyLong_FromLong(code);
        return given == Py_None ? THPVariable_Wrap(t) : (Py_INCREF(given), given);
    }
};

template <typename F>
PyObject *guarded(F f)
{
    try {
        return f();
    } catch (const Refused &e) {
        if (e.type)
            PyErr_SetString(e.type, e.what());
        return nullptr;
    } catch (const std::exception &e) {
        PyErr_SetString(PyExc_RuntimeError, e.what());
        return nullptr;
    }
}

// (q, k, v, q_weight, k_weight, positions, inv_freq or None, slots, k_cache,
//  v_cache, out or None, eps, weight_offset, interleaved, stream)
PyObject *qk_norm_rope(PyObject *, PyObject *const *a, Py_ssize_t n)
{
    return guarded([&]() -> PyObject * {
        args(n, 15);
        const at::Tensor &q = tensor(a[0], "q"), &k = tensor(a[1], "k"), &v = tensor(a[2], "v");
        if (q.dim() != 3 || k.dim() != 3 || v.dim() != 3)
            throw Refused(PyExc_ValueError, "q, k and v must be 3-D [M, heads, D]");
        const Call c = on_gpu(q, "q");
        const at::ScalarType type = q.scalar_type();
        if (type_code(type) < 0)
            throw Refused(PyExc_TypeError, std::string("q must be float32, float16 or bfloat16, got ") + c10::toString(type));
        const int64_t M = q.size(0), Hq = q.size(1), D = q.size(2);
        if (M > INT32_MAX || Hq > INT32_MAX || D > INT32_MAX)
            throw Refused(PyExc_ValueError, "q's sizes do not fit 32 bits");
        const Caches kv = caches(c, a[8], a[9], D);
        const int64_t qs = c.rows(q, "q", type, q.sizes());
        const int64_t keys[3] = {M, kv.Hkv, D};
        const int64_t ks = c.rows(k, "k", type, keys), vs = c.rows(v, "v", type, keys);
        int R = 0;
        const float *freq = nullptr;
        if (a[6] != Py_None) {
            const int64_t half = tensor(a[6], "inv_freq").numel();
            R = (int)(half < 4096 ? 2 * half : 8192);
            freq = static_cast<const float *>(c.whole(a[6], "inv_freq", at::kFloat, {half}));
        }
        const Output out(c, a[10], "out", kv.type, {M, Hq, D});
        const int code =
            qmm_qk_norm_rope(q.data_ptr(), k.data_ptr(), v.data_ptr(), qs, ks, vs, type_code(type),
                                static_cast<const float *>(c.whole(a[3], "q_weight", at::kFloat, {D})),
                                static_cast<const float *>(c.whole(a[4], "k_weight", at::kFloat, {D})), as_float(a[11]),
                                as_float(a[12]), static_cast<const int32_t *>(c.whole(a[5], "positions", at::kInt, {M})),
                                freq, R, PyObject_IsTrue(a[13]),
                                static_cast<const int32_t *>(c.whole(a[7], "slots", at::kInt, {M})),
                                out.data, kv.k.data_ptr(), kv.v.data_ptr(),
                                type_code(kv.type), (int)M, (int)Hq, kv.Hkv, (int)D, kv.pages, kv.page_size,
                                as_stream(a[14]));
        return out.result(code);
    });
}

// A workspace of `need` bytes: the caller's, or one from torch's allocator on
// the current stream, which is the call's (freed to that stream's pool when the
// call returns: what runs on it next runs after).
struct Workspace {
    at::Tensor own;
    void *data = nullptr;
    size_t bytes = 0;
    Workspace(PyObject *given, size_t need, const c10::Device &device)
    {
        if (given != Py_None) {
            const at::Tensor &t = tensor(given, "workspace");
            if (t.device() != device || !t.is_contiguous())
                throw Refused(PyExc_ValueError, "workspace must be contiguous on the GPU device " + device.str());
            data = t.data_ptr();
            bytes = t.numel() * t.element_size();
        } else if (need > 0) {
            own = at::empty({(int64_t)need}, at::TensorOptions().dtype(at::kByte).device(device));
            data = own.data_ptr();
            bytes = need;
        }
    }
};

// (q, k_cache, v_cache, block_table, context_lens, row_starts, max_rows,
//  max_context, scale or None, window, sinks, out or None, lse or None, workspace or
//  None, stream)
PyObject *paged_attention(PyObject *, PyObject *const *a, Py_ssize_t n)
{
    return guarded([&]() -> PyObject * {
        args(n, 15);
        const at::Tensor &q = tensor(a[0], "q"), &table = tensor(a[3], "block_table");
        if (q.dim() != 3 || table.dim() != 2)
            throw Refused(PyExc_ValueError, "q must be 3-D [T, Hq, D] and block_table 2-D [B, max_pages]");
        const Call c = on_gpu(q, "q");
        const int64_t T = q.size(0), Hq = q.size(1), D = q.size(2), B = table.size(0), max_pages = table.size(1);
        if (T > INT32_MAX || Hq > INT32_MAX || D > INT32_MAX || B > INT32_MAX || max_pages > INT32_MAX)
            throw Refused(PyExc_ValueError, "sizes of q or block_table do not fit 32 bits");
        const Caches kv = caches(c, a[1], a[2], D);
        const int64_t qs = c.rows(q, "q", kv.type, q.sizes());
        const int max_rows = as_int(a[6], "max_rows"), max_context = as_int(a[7], "max_context");
        const int window = as_int(a[9], "window"), sinks = as_int(a[10], "sinks");
        const int32_t *blocks = static_cast<const int32_t *>(c.whole(table, "block_table", at::kInt, table.sizes()));
        const int32_t *lens = static_cast<const int32_t *>(c.whole(a[4], "context_lens", at::kInt, {B}));
        const int32_t *starts = static_cast<const int32_t *>(c.whole(a[5], "row_starts", at::kInt, {B + 1}));
        const Output out(c, a[11], "out", kv.type, {T, Hq, D});
        float *lse = static_cast<float *>(c.whole_or_null(a[12], "lse", at::kFloat, {T, Hq}));
        const float scale = a[8] == Py_None ? (float)(1.0 / std::sqrt((double)D)) : as_float(a[8]);
        const hipStream_t stream = as_stream(a[14]);
        const Workspace ws(a[13],
                           qmm_paged_attention_workspace_bytes((int)T, (int)B, (int)Hq, kv.Hkv, (int)D, max_rows,
                                                               max_context, window, sinks),
                           c.device);
        return out.result(
            qmm_paged_attention(q.data_ptr(), qs, kv.k.data_ptr(), kv.v.data_ptr(), type_code(kv.type), blocks, lens,
                                   starts, out.data, lse, (int)T, (int)B, (int)Hq, kv.Hkv, (int)D, kv.pages, kv.page_size,
                                   (int)max_pages, max_rows, max_context, scale, window, sinks, ws.data, ws.bytes, stream));
    });
}

// (logits, u, temperature, top_k, top_p, min_p or None each, tokens
//  or None, logprobs or None, workspace or None, stream)
PyObject *sample(PyObject *, PyObject *const *a, Py_ssize_t n)
{
    return guarded([&]() -> PyObject * {
        args(n, 10);
        const at::Tensor &x = tensor(a[0], "logits");
        if (x.dim() != 2)
            throw Refused(PyExc_ValueError, "logits must be 2-D [M, V]");
        const Call c = on_gpu(x, "logits");
        const at::ScalarType type = x.scalar_type();
        if (type_code(type) < 0)
            throw Refused(PyExc_TypeError,
                          std::string("logits must be float32, float16 or bfloat16, got ") + c10::toString(type));
        const int64_t M = x.size(0), V = x.size(1);
        if (M > INT32_MAX || V > INT32_MAX)
            throw Refused(PyExc_ValueError, "sizes of logits do not fit 32 bits");
        const int64_t stride = c.rows(x, "logits", type, x.sizes());
        const float *u = static_cast<const float *>(c.whole(a[1], "u", at::kFloat, {M}));
        const float *t = static_cast<const float *>(c.whole_or_null(a[2], "temperature", at::kFloat, {M}));
        const int32_t *k = static_cast<const int32_t *>(c.whole_or_null(a[3], "top_k", at::kInt, {M}));
        const float *p = static_cast<const float *>(c.whole_or_null(a[4], "top_p", at::kFloat, {M}));
        const float *mp = static_cast<const float *>(c.whole_or_null(a[5], "min_p", at::kFloat, {M}));
        const Output tokens(c, a[6], "tokens", at::kInt, {M});
        float *lp = static_cast<float *>(c.whole_or_null(a[7], "logprobs", at::kFloat, {M}));
        const hipStream_t stream = as_stream(a[9]);
        const Workspace ws(a[8], qmm_sample_workspace_bytes((int)M, (int)V), c.device);
        return tokens.result(qmm_sample(x.data_ptr(), stride, type_code(type), u, t, k, p, mp,
                                        static_cast<int32_t *>(tokens.data), lp, (int)M, (int)V, ws.data, ws.bytes,
                                        stream));
    });
}

PyMethodDef methods[] = {
    {"qk_norm_rope", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(qk_norm_rope)), METH_FASTCALL, nullptr},
    {"paged_attention", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(paged_attention)), METH_FASTCALL,
     nullptr},
    {"sample", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(sample)), METH_FASTCALL, nullptr},
    {nullptr, nullptr, 0, nullptr},
};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_qmm_torch", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__qmm_torch() { return PyModule_Create(&module); }
