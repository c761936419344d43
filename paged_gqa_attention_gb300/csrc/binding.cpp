// binding.cpp -- the usual case of the small serving calls, without Python between a call and its
// launch.
//
// A decode step of a few sequences takes the GPU 2 to 5 us; checking a dozen tensors and
// marshalling as many pointers through ctypes takes the host 14 to 27.  The functions here check
// the arguments of paged_rope_append(_fp8), paged_attn_decode_window(_fp8) and
// paged_attn_prefill_window against the one form that callers use in practice (plain CUDA tensors
// of the right types and shapes on one device, options of the right Python types), allocate the
// output, take the device's current stream and make the C call.  Anything else is not judged
// here: they return None, and ops.py goes through its own checks, which say what is wrong.
// Returns: the output tensor, None, or the call's status as an int when it is not PA_OK.
#include <Python.h>

#include <ATen/ATen.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include "pagedattn.h"

namespace {

constexpr pa_shape kShape = {32, 8, 128, 256};
constexpr int64_t kHq = 32, kHkv = 8, kD = 128, kBlock = 256;

// The tensor behind a Python object, or nullptr when it is not a plain one.
const at::Tensor *tensor(PyObject *o) { return THPVariable_CheckExact(o) ? &THPVariable_Unpack(o) : nullptr; }

// A contiguous tensor of this type on device `dev` (-1: on any GPU).
bool plain(const at::Tensor *t, at::ScalarType type, int dev) {
    return t && t->defined() && t->is_cuda() && t->scalar_type() == type && (dev < 0 || t->get_device() == dev) &&
           t->is_contiguous();
}

bool sized(const at::Tensor &t, std::initializer_list<int64_t> want) {   // -1: any size
    if (t.dim() != (int64_t)want.size()) return false;
    int64_t i = 0;
    for (int64_t n : want) {
        if (n >= 0 && t.size(i) != n) return false;
        ++i;
    }
    return true;
}

bool fits32(int64_t n) { return n >= 0 && n <= INT32_MAX; }

bool as_int32(PyObject *o, int32_t *x) {
    if (!PyLong_CheckExact(o)) return false;
    int overflow = 0;
    const long long v = PyLong_AsLongLongAndOverflow(o, &overflow);
    if (overflow || v < INT32_MIN || v > INT32_MAX) return false;
    *x = (int32_t)v;
    return true;
}

bool as_float(PyObject *o, double *x) {
    if (PyFloat_CheckExact(o)) {
        *x = PyFloat_AS_DOUBLE(o);
        return true;
    }
    int32_t i;
    if (!as_int32(o, &i)) return false;
    *x = i;
    return true;
}

// [tokens][heads][128] bf16 rows on dev, whole and a multiple of 8 elements apart.
bool rows(const at::Tensor *t, int64_t tokens, int64_t heads, int dev, int64_t *stride) {
    if (!t || !t->defined() || !t->is_cuda() || t->scalar_type() != at::kBFloat16 || t->get_device() != dev ||
        !sized(*t, {tokens, heads, kD}) || t->stride(2) != 1 || t->stride(1) != kD)
        return false;
    *stride = tokens == 1 ? heads * kD : t->stride(0);
    return *stride >= heads * kD && *stride % 8 == 0;
}

// The cache's tensors (k_pool, v_pool or k_codes, v_codes, k_scale, v_scale) and their device.
struct Cache {
    const at::Tensor *t[4];
    int dev = -1;
    int32_t blocks = 0;

    bool take(PyObject *const *o, bool eight_bit) {
        const at::ScalarType type = eight_bit ? at::kByte : at::kBFloat16;
        for (int i = 0; i < 2; ++i) {
            t[i] = tensor(o[i]);
            if (!plain(t[i], type, dev) || !sized(*t[i], {i ? blocks : -1, kBlock, kHkv, kD})) return false;
            dev = t[i]->get_device();
            if (!fits32(t[i]->size(0))) return false;
            blocks = (int32_t)t[i]->size(0);
        }
        for (int i = 2; eight_bit && i < 4; ++i) {
            t[i] = tensor(o[i]);
            if (!plain(t[i], at::kFloat, dev) || !sized(*t[i], {blocks, kHkv, kBlock})) return false;
        }
        return true;
    }
    void *ptr(int i) const { return t[i]->data_ptr(); }
    float *scale(int i) const { return static_cast<float *>(t[i]->data_ptr()); }
};

const int32_t *ints(const at::Tensor *t) { return static_cast<const int32_t *>(t->data_ptr()); }

// `out` as given (None: a new tensor of that shape); false when it is not a plain one of it.
bool output(PyObject *o, at::IntArrayRef shape, int dev, at::Tensor *out) {
    if (o == Py_None) {
        *out = at::empty(shape, at::TensorOptions().dtype(at::kBFloat16).device(at::kCUDA, dev));
        return true;
    }
    const at::Tensor *t = tensor(o);
    if (!plain(t, at::kBFloat16, dev) || t->sizes() != shape) return false;
    *out = *t;
    return true;
}

PyObject *answer(pa_status st, const at::Tensor &out) {
    return st == PA_OK ? THPVariable_Wrap(out) : PyLong_FromLong((long)st);
}

// Exceptions of torch (out of memory) become Python's; none crosses into the interpreter.
template <typename F>
PyObject *guarded(F f) {
    HANDLE_TH_ERRORS
    return f();
    END_HANDLE_TH_ERRORS
}

// rope_append(eight_bit, q, k_new, v_new, k, v, k_scale, v_scale, block_table, cu_q_lens, seq_lens, workspace,
//             rope_theta, positions, pair_axis, q_norm_weight, k_norm_weight, norm_eps, q_out)
PyObject *rope_append(PyObject *, PyObject *const *o, Py_ssize_t n) {
    if (n != 19) Py_RETURN_NONE;
    return guarded([&]() -> PyObject * {
        const bool eight_bit = o[0] == Py_True;
        Cache cache;
        if (!cache.take(o + 4, eight_bit)) Py_RETURN_NONE;
        const int dev = cache.dev;
        const at::Tensor *q = tensor(o[1]), *k = tensor(o[2]), *v = tensor(o[3]);
        const at::Tensor *table = tensor(o[8]), *cu = tensor(o[9]), *lens = tensor(o[10]), *ws = tensor(o[11]);
        if (!q || q->dim() != 3) Py_RETURN_NONE;
        const int64_t tokens = q->size(0);
        int64_t qs, ks, vs;
        if (!fits32(tokens) || !rows(q, tokens, kHq, dev, &qs) || !rows(k, tokens, kHkv, dev, &ks) ||
            !rows(v, tokens, kHkv, dev, &vs) || !plain(table, at::kInt, dev) || !sized(*table, {-1, -1}) ||
            !fits32(table->size(0)) || !fits32(table->size(1)) || !plain(ws, at::kByte, dev))
            Py_RETURN_NONE;
        const int64_t seqs = table->size(0);
        if (!plain(cu, at::kInt, dev) || !sized(*cu, {seqs + 1}) || !plain(lens, at::kInt, dev) || !sized(*lens, {seqs}))
            Py_RETURN_NONE;
        double theta, eps;
        if (!as_float(o[12], &theta) || !as_float(o[17], &eps)) Py_RETURN_NONE;
        const int32_t *positions = nullptr;
        int32_t axes = 1;
        if (o[13] != Py_None) {
            const at::Tensor *p = tensor(o[13]);
            if (!plain(p, at::kInt, dev) || p->dim() < 1 || p->dim() > 2 || p->size(p->dim() - 1) != tokens ||
                !fits32(p->size(0)))
                Py_RETURN_NONE;
            if (p->dim() == 2) axes = (int32_t)p->size(0);
            positions = ints(p);
        }
        const uint8_t *pair_axis = nullptr;
        if (o[14] != Py_None) {
            if (!PyBytes_CheckExact(o[14]) || PyBytes_GET_SIZE(o[14]) != kD / 2) Py_RETURN_NONE;
            pair_axis = reinterpret_cast<const uint8_t *>(PyBytes_AS_STRING(o[14]));
        }
        const void *gains[2] = {nullptr, nullptr};
        if ((o[15] == Py_None) != (o[16] == Py_None)) Py_RETURN_NONE;
        for (int i = 0; i < 2; ++i) {
            if (o[15 + i] == Py_None) continue;
            const at::Tensor *g = tensor(o[15 + i]);
            if (!plain(g, at::kBFloat16, dev) || !sized(*g, {kD})) Py_RETURN_NONE;
            gains[i] = g->data_ptr();
        }
        at::Tensor out;
        if (!output(o[18], {tokens, kHq, kD}, dev, &out)) Py_RETURN_NONE;
        const c10::cuda::OptionalCUDAGuard on(c10::Device(c10::kCUDA, (c10::DeviceIndex)dev));
        void *stream = c10::cuda::getCurrentCUDAStream((c10::DeviceIndex)dev).stream();
        const pa_status st =
            eight_bit ? paged_rope_append_fp8(kShape, (float)theta, positions, axes, pair_axis, gains[0], gains[1],
                                              (float)eps, out.data_ptr(), q->data_ptr(), qs, k->data_ptr(), ks,
                                              v->data_ptr(), vs, cache.ptr(0), cache.ptr(1), cache.scale(2),
                                              cache.scale(3), ints(table), (int32_t)table->size(1), cache.blocks,
                                              ints(cu), ints(lens), (int32_t)seqs, (int32_t)tokens, ws->data_ptr(),
                                              (size_t)ws->numel(), stream)
                      : paged_rope_append(kShape, (float)theta, positions, axes, pair_axis, gains[0], gains[1],
                                          (float)eps, out.data_ptr(), q->data_ptr(), qs, k->data_ptr(), ks,
                                          v->data_ptr(), vs, cache.ptr(0), cache.ptr(1), ints(table),
                                          (int32_t)table->size(1), cache.blocks, ints(cu), ints(lens), (int32_t)seqs,
                                          (int32_t)tokens, ws->data_ptr(), (size_t)ws->numel(), stream);
        return answer(st, out);
    });
}

// What the attention calls share: q, the block table, the lengths, out, lse and the workspace.
struct Attention {
    Cache cache;
    const at::Tensor *q, *table, *lens, *ws;
    float *lse = nullptr;
    at::Tensor out;
    int64_t tokens;

    bool take(bool eight_bit, PyObject *const *k, PyObject *q_, PyObject *table_, PyObject *lens_, PyObject *ws_,
              PyObject *out_, PyObject *lse_) {
        if (!cache.take(k, eight_bit)) return false;
        const int dev = cache.dev;
        q = tensor(q_), table = tensor(table_), lens = tensor(lens_), ws = tensor(ws_);
        if (!plain(q, at::kBFloat16, dev) || !sized(*q, {-1, kHq, kD}) || !fits32(q->size(0)) ||
            !plain(table, at::kInt, dev) || !sized(*table, {-1, -1}) || !fits32(table->size(0)) ||
            !fits32(table->size(1)) || !plain(lens, at::kInt, dev) || !sized(*lens, {table->size(0)}) ||
            !plain(ws, at::kByte, dev))
            return false;
        tokens = q->size(0);
        if (lse_ != Py_None) {
            const at::Tensor *l = tensor(lse_);
            if (!plain(l, at::kFloat, dev) || !sized(*l, {tokens, kHq})) return false;
            lse = static_cast<float *>(l->data_ptr());
        }
        return output(out_, q->sizes(), dev, &out);
    }
};

// decode_window(eight_bit, q, k, v, k_scale, v_scale, block_table, seq_lens, workspace, window, sinks, scale,
//               split_tokens, out, lse)
PyObject *decode_window(PyObject *, PyObject *const *o, Py_ssize_t n) {
    if (n != 15) Py_RETURN_NONE;
    return guarded([&]() -> PyObject * {
        const bool eight_bit = o[0] == Py_True;
        Attention a;
        int32_t window, sinks, split;
        double scale;
        if (!as_int32(o[9], &window) || !as_int32(o[10], &sinks) || !as_float(o[11], &scale) ||
            !as_int32(o[12], &split) || !a.take(eight_bit, o + 2, o[1], o[6], o[7], o[8], o[13], o[14]) ||
            a.table->size(0) != a.tokens)
            Py_RETURN_NONE;
        const c10::cuda::OptionalCUDAGuard on(c10::Device(c10::kCUDA, (c10::DeviceIndex)a.cache.dev));
        void *stream = c10::cuda::getCurrentCUDAStream((c10::DeviceIndex)a.cache.dev).stream();
        const int32_t width = (int32_t)a.table->size(1), batch = (int32_t)a.tokens;
        const pa_status st =
            eight_bit ? paged_attn_decode_window_fp8(kShape, a.out.data_ptr(), a.lse, a.q->data_ptr(), a.cache.ptr(0),
                                                     a.cache.ptr(1), a.cache.scale(2), a.cache.scale(3),
                                                     ints(a.table), width, a.cache.blocks, ints(a.lens), batch, window,
                                                     sinks, (float)scale, split, a.ws->data_ptr(),
                                                     (size_t)a.ws->numel(), stream)
                      : paged_attn_decode_window(kShape, a.out.data_ptr(), a.lse, a.q->data_ptr(), a.cache.ptr(0),
                                                 a.cache.ptr(1), ints(a.table), width, a.cache.blocks, ints(a.lens),
                                                 batch, window, sinks, (float)scale, split, a.ws->data_ptr(),
                                                 (size_t)a.ws->numel(), stream);
        return answer(st, a.out);
    });
}

// prefill_window(q, k_pool, v_pool, block_table, cu_q_lens, seq_lens, max_q_len, workspace, window, sinks, scale,
//                out, lse)
PyObject *prefill_window(PyObject *, PyObject *const *o, Py_ssize_t n) {
    if (n != 13) Py_RETURN_NONE;
    return guarded([&]() -> PyObject * {
        Attention a;
        int32_t max_q_len, window, sinks;
        double scale;
        if (!as_int32(o[6], &max_q_len) || !as_int32(o[8], &window) || !as_int32(o[9], &sinks) ||
            !as_float(o[10], &scale) || !a.take(false, o + 1, o[0], o[3], o[5], o[7], o[11], o[12]))
            Py_RETURN_NONE;
        const at::Tensor *cu = tensor(o[4]);
        if (!plain(cu, at::kInt, a.cache.dev) || !sized(*cu, {a.table->size(0) + 1})) Py_RETURN_NONE;
        const c10::cuda::OptionalCUDAGuard on(c10::Device(c10::kCUDA, (c10::DeviceIndex)a.cache.dev));
        void *stream = c10::cuda::getCurrentCUDAStream((c10::DeviceIndex)a.cache.dev).stream();
        const pa_status st = paged_attn_prefill_window(
            kShape, a.out.data_ptr(), a.lse, a.q->data_ptr(), a.cache.ptr(0), a.cache.ptr(1), ints(a.table),
            (int32_t)a.table->size(1), a.cache.blocks, ints(cu), ints(a.lens), (int32_t)a.table->size(0),
            (int32_t)a.tokens, max_q_len, window, sinks, (float)scale, a.ws->data_ptr(), (size_t)a.ws->numel(), stream);
        return answer(st, a.out);
    });
}

template <typename F>
PyCFunction fastcall(F f) { return reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(f)); }

PyMethodDef methods[] = {
    {"rope_append", fastcall(rope_append), METH_FASTCALL, "paged_rope_append(_fp8) in the usual case, else None"},
    {"decode_window", fastcall(decode_window), METH_FASTCALL, "paged_attn_decode_window(_fp8) in the usual case, else None"},
    {"prefill_window", fastcall(prefill_window), METH_FASTCALL, "paged_attn_prefill_window in the usual case, else None"},
    {nullptr, nullptr, 0, nullptr}};

PyModuleDef module = {PyModuleDef_HEAD_INIT, "_binding", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__binding(void) { return PyModule_Create(&module); }
