// torch_calls.cpp -- the calls of the 8-bit cache and of the query / key preparation for torch
// tensors.
//
// These calls sit in decode loops whose kernels take two to five microseconds, where
// testing ten tensors' attributes and converting twenty arguments in Python costs
// three to four times that.  Each function here tests its arguments, allocates what the
// caller did not pass, and calls the C ABI on the current stream of the tensors'
// device, with that device current.  It returns the result, or an integer: a
// pkv_status, or -1 where an argument is not what it should be; the Python wrapper
// then names it.
#define PY_SSIZE_T_CLEAN
#include <Python.h>

#include <ATen/cuda/EmptyTensor.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/Dtype.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include <climits>

#include "pkv.h"

namespace {

using at::ScalarType;
using at::Tensor;

// A tensor argument; none where the object is not a tensor (None included).
const Tensor* tensor(PyObject* o) { return THPVariable_Check(o) ? &THPVariable_Unpack(o) : nullptr; }

// Type, device and density of a tensor of any shape.
bool is(const Tensor* t, ScalarType type, at::DeviceIndex dev) {
    return t && t->scalar_type() == type && t->is_cuda() && t->get_device() == dev && t->is_contiguous();
}
bool is(const Tensor* t, ScalarType type, at::DeviceIndex dev, at::IntArrayRef shape) {
    return is(t, type, dev) && t->sizes() == shape;
}

bool optional(PyObject* o, ScalarType type, at::DeviceIndex dev, at::IntArrayRef shape) {
    return o == Py_None || is(tensor(o), type, dev, shape);
}
template <typename T = void>
T* pointer(PyObject* o) {
    return o == Py_None ? nullptr : static_cast<T*>(THPVariable_Unpack(o).data_ptr());
}

bool float_code(ScalarType t, pkv_dtype* code) {
    *code = t == ScalarType::Float ? PKV_F32 : PKV_BF16;
    return t == ScalarType::Float || t == ScalarType::BFloat16;
}

// An 8-bit cache, or (k_scale and v_scale None) one of rows of type `plain`.
struct Cache {
    const Tensor *k, *v;
    float *ks = nullptr, *vs = nullptr;
    int NB, Hkv, BS, D;
    at::DeviceIndex dev;
    pkv_dtype code;

    bool take(PyObject* ko, PyObject* vo, PyObject* kso, PyObject* vso, const ScalarType* plain) {
        k = tensor(ko);
        v = tensor(vo);
        if (!k || !k->is_cuda() || k->dim() != 4) return false;
        dev = k->get_device();
        const ScalarType type = k->scalar_type();
        if (!is(k, type, dev) || !is(v, type, dev, k->sizes())) return false;
        for (int i = 0; i < 4; ++i)
            if (k->size(i) > INT_MAX) return false;
        NB = static_cast<int>(k->size(0));
        Hkv = static_cast<int>(k->size(1));
        BS = static_cast<int>(k->size(2));
        D = static_cast<int>(k->size(3));
        if (plain && kso == Py_None && vso == Py_None) return type == *plain && float_code(type, &code);
        if (type != ScalarType::Float8_e4m3fn && type != ScalarType::Char) return false;
        code = type == ScalarType::Char ? PKV_I8 : PKV_E4M3;
        const at::IntArrayRef rows = k->sizes().slice(0, 3);
        if (!is(tensor(kso), ScalarType::Float, dev, rows) || !is(tensor(vso), ScalarType::Float, dev, rows)) return false;
        ks = pointer<float>(kso);
        vs = pointer<float>(vso);
        return true;
    }
};

struct Sequences {
    int B, max_blocks;
    int32_t *tables, *lens, *status;

    bool take(PyObject* bto, PyObject* slo, PyObject* sto, at::DeviceIndex dev) {
        const Tensor *bt = tensor(bto), *sl = tensor(slo);
        if (!is(bt, ScalarType::Int, dev) || !is(sl, ScalarType::Int, dev) || bt->dim() != 2 || sl->dim() != 1 ||
            bt->size(0) != sl->size(0) || bt->size(0) > INT_MAX || bt->size(1) > INT_MAX ||
            !optional(sto, ScalarType::Int, dev, {1}))
            return false;
        B = static_cast<int>(sl->size(0));
        max_blocks = static_cast<int>(bt->size(1));
        tables = bt->data_ptr<int32_t>();
        lens = sl->data_ptr<int32_t>();
        status = pointer<int32_t>(sto);
        return true;
    }
};

void* stream_of(at::DeviceIndex dev) { return c10::cuda::getCurrentCUDAStream(dev).stream(); }

PyObject* code(long c) { return PyLong_FromLong(c); }

// A new tensor beside `like` (on its device, which is current).
Tensor fresh(at::IntArrayRef shape, ScalarType type, const Tensor* like) {
    return at::detail::empty_cuda(shape, type, like->device(), std::nullopt);
}

// append(k_new, v_new, k_cache, v_cache, k_scale, v_scale, block_tables, seq_lens, q_start, status)
PyObject* append(PyObject*, PyObject* const* a, Py_ssize_t n) {
    HANDLE_TH_ERRORS
    Cache c;
    Sequences s;
    const Tensor *kn = nullptr, *vn = nullptr;
    pkv_dtype dtype;
    if (n != 10 || !c.take(a[2], a[3], a[4], a[5], nullptr) || !s.take(a[6], a[7], a[9], c.dev) ||
        !(kn = tensor(a[0])) || !(vn = tensor(a[1])) || !float_code(kn->scalar_type(), &dtype) || kn->dim() != 3)
        return code(-1);
    const int64_t T = kn->size(0);
    if (T > INT_MAX || !is(kn, kn->scalar_type(), c.dev, {T, c.Hkv, c.D}) ||
        !is(vn, kn->scalar_type(), c.dev, kn->sizes()) || !optional(a[8], ScalarType::Int, c.dev, {s.B + 1}) ||
        (a[8] == Py_None && T != s.B))
        return code(-1);
    const c10::cuda::OptionalCUDAGuard guard(c.k->device());
    return code(pkv_kv_append_q8(kn->data_ptr(), vn->data_ptr(), c.k->data_ptr(), c.v->data_ptr(), c.ks, c.vs, s.tables,
                                 s.max_blocks, s.lens, pointer<int32_t>(a[8]), s.B, static_cast<int>(T), c.Hkv, c.D,
                                 c.BS, c.NB, dtype, c.code, s.status, stream_of(c.dev)));
    END_HANDLE_TH_ERRORS
}

// read(k_cache, v_cache, k_scale, v_scale, blocks, k_out, v_out, dtype, status) -> (k, v)
PyObject* read(PyObject*, PyObject* const* a, Py_ssize_t n) {
    HANDLE_TH_ERRORS
    Cache c;
    const Tensor* ids = nullptr;
    if (n != 9 || !c.take(a[0], a[1], a[2], a[3], nullptr) || !(ids = tensor(a[4])) ||
        !is(ids, ScalarType::Int, c.dev) || ids->dim() != 1 || ids->size(0) > INT_MAX ||
        !optional(a[8], ScalarType::Int, c.dev, {1}))
        return code(-1);
    const int64_t shape[4] = {ids->size(0), c.Hkv, c.BS, c.D};
    ScalarType type;
    if (a[5] != Py_None || a[6] != Py_None) {
        const Tensor* t = tensor(a[5] != Py_None ? a[5] : a[6]);
        if (!t) return code(-1);
        type = t->scalar_type();
    } else {
        if (!THPDtype_Check(a[7])) return code(-1);
        type = reinterpret_cast<THPDtype*>(a[7])->scalar_type;
    }
    pkv_dtype dtype;
    if (!float_code(type, &dtype) || !optional(a[5], type, c.dev, shape) || !optional(a[6], type, c.dev, shape))
        return code(-1);
    const c10::cuda::OptionalCUDAGuard guard(c.k->device());
    const Tensor ko = a[5] != Py_None ? THPVariable_Unpack(a[5]) : fresh(shape, type, c.k);
    const Tensor vo = a[6] != Py_None ? THPVariable_Unpack(a[6]) : fresh(shape, type, c.k);
    const pkv_status r = pkv_kv_read_blocks_q8(
        ko.data_ptr(), vo.data_ptr(), c.k->data_ptr(), c.v->data_ptr(), c.ks, c.vs, ids->data_ptr<int32_t>(),
        static_cast<int>(ids->size(0)), c.Hkv, c.D, c.BS, c.NB, dtype, c.code, pointer<int32_t>(a[8]), stream_of(c.dev));
    if (r != PKV_OK) return code(r);
    PyObject* out = PyTuple_New(2);
    if (!out) return nullptr;
    PyTuple_SET_ITEM(out, 0, THPVariable_Wrap(ko));
    PyTuple_SET_ITEM(out, 1, THPVariable_Wrap(vo));
    return out;
    END_HANDLE_TH_ERRORS
}

// attend(q, k_cache, v_cache, k_scale, v_scale, block_tables, seq_lens, out, scale, workspace, status) -> out
PyObject* attend(PyObject*, PyObject* const* a, Py_ssize_t n) {
    HANDLE_TH_ERRORS
    Cache c;
    Sequences s;
    const Tensor* q = nullptr;
    pkv_dtype dtype;
    if (n != 11 || !c.take(a[1], a[2], a[3], a[4], nullptr) || !s.take(a[5], a[6], a[10], c.dev) ||
        !(q = tensor(a[0])) || !float_code(q->scalar_type(), &dtype) || q->dim() != 3 || q->size(1) > INT_MAX ||
        !is(q, q->scalar_type(), c.dev, {s.B, q->size(1), c.D}) ||
        !optional(a[7], q->scalar_type(), c.dev, q->sizes()))
        return code(-1);
    const double scale = PyFloat_AsDouble(a[8]);
    if (scale == -1.0 && PyErr_Occurred()) return nullptr;
    const Tensor* ws = nullptr;
    if (a[9] != Py_None && (!(ws = tensor(a[9])) || !is(ws, ws->scalar_type(), c.dev))) return code(-1);
    const c10::cuda::OptionalCUDAGuard guard(c.k->device());
    const int Hq = static_cast<int>(q->size(1));
    Tensor out = a[7] != Py_None ? THPVariable_Unpack(a[7]) : fresh(q->sizes(), q->scalar_type(), q);
    Tensor own;
    size_t bytes;
    if (!ws) {
        bytes = pkv_decode_q8_workspace_bytes(s.B, Hq, c.Hkv, c.D, 0);
        own = fresh({static_cast<int64_t>(bytes < 16 ? 16 : bytes)}, ScalarType::Byte, q);
        ws = &own;
    } else {
        bytes = ws->nbytes();
    }
    const pkv_status r = pkv_paged_decode_attention_q8(
        out.data_ptr(), q->data_ptr(), c.k->data_ptr(), c.v->data_ptr(), c.ks, c.vs, s.tables, s.max_blocks, s.lens, s.B,
        Hq, c.Hkv, c.D, c.BS, c.NB, static_cast<float>(scale), dtype, c.code, ws->data_ptr(), bytes, s.status,
        stream_of(c.dev));
    return r != PKV_OK ? code(r) : THPVariable_Wrap(std::move(out));
    END_HANDLE_TH_ERRORS
}

// Elements between the tokens of a [T, H, D] view whose heads are dense; -1 if it is none.
int64_t token_stride(const Tensor* t, ScalarType type, at::DeviceIndex dev, int64_t T, int64_t H, int64_t D) {
    if (!t || t->scalar_type() != type || !t->is_cuda() || t->get_device() != dev || t->dim() != 3 || t->size(0) != T ||
        t->size(1) != H || t->size(2) != D || (D > 1 && t->stride(2) != 1) || (H > 1 && t->stride(1) != D))
        return -1;
    if (T <= 1) return H * D;
    return t->stride(0) >= H * D ? t->stride(0) : -1;
}

// prepare(q, k_new, v_new, q_weight, k_weight, eps, freqs, k_cache, v_cache, block_tables, seq_lens, q_start,
//         k_scale, v_scale, interleaved, q_out, status) -> q_out
PyObject* prepare(PyObject*, PyObject* const* a, Py_ssize_t n) {
    HANDLE_TH_ERRORS
    Cache c;
    Sequences s;
    const Tensor* q = n == 17 ? tensor(a[0]) : nullptr;
    pkv_dtype dtype;
    if (!q || q->dim() != 3 || q->size(0) > INT_MAX || q->size(1) > INT_MAX || !float_code(q->scalar_type(), &dtype))
        return code(-1);
    const ScalarType type = q->scalar_type();
    if (!c.take(a[7], a[8], a[12], a[13], &type) || !s.take(a[9], a[10], a[16], c.dev)) return code(-1);
    const int64_t T = q->size(0), Hq = q->size(1);
    const int64_t qs = token_stride(q, type, c.dev, T, Hq, c.D), ks = token_stride(tensor(a[1]), type, c.dev, T, c.Hkv, c.D),
                  vs = token_stride(tensor(a[2]), type, c.dev, T, c.Hkv, c.D);
    const Tensor* freqs = a[6] == Py_None ? nullptr : tensor(a[6]);
    if (qs < 0 || ks < 0 || vs < 0 || !optional(a[3], type, c.dev, {c.D}) || !optional(a[4], type, c.dev, {c.D}) ||
        (a[6] != Py_None && (!is(freqs, ScalarType::Long, c.dev) || freqs->dim() != 1 || freqs->size(0) > INT_MAX / 2)) ||
        !optional(a[11], ScalarType::Int, c.dev, {s.B + 1}) || (a[11] == Py_None && T != s.B) ||
        !optional(a[15], type, c.dev, q->sizes()))
        return code(-1);
    const double eps = PyFloat_AsDouble(a[5]);
    if (eps == -1.0 && PyErr_Occurred()) return nullptr;
    const int interleaved = PyObject_IsTrue(a[14]);
    if (interleaved < 0) return nullptr;
    const c10::cuda::OptionalCUDAGuard guard(c.k->device());
    Tensor out = a[15] != Py_None ? THPVariable_Unpack(a[15]) : fresh(q->sizes(), type, q);
    const pkv_status r = pkv_qk_norm_rope_append(
        out.data_ptr(), q->data_ptr(), qs, pointer<>(a[1]), ks, pointer<>(a[2]), vs, pointer<>(a[3]), pointer<>(a[4]),
        static_cast<float>(eps), freqs ? freqs->data_ptr<int64_t>() : nullptr,
        freqs ? 2 * static_cast<int>(freqs->size(0)) : 0, interleaved, c.k->data_ptr(), c.v->data_ptr(), c.ks, c.vs,
        s.tables, s.max_blocks, s.lens, pointer<int32_t>(a[11]), s.B, static_cast<int>(T), static_cast<int>(Hq), c.Hkv,
        c.D, c.BS, c.NB, dtype, c.code, s.status, stream_of(c.dev));
    return r != PKV_OK ? code(r) : THPVariable_Wrap(std::move(out));
    END_HANDLE_TH_ERRORS
}

PyMethodDef methods[] = {
    {"append", reinterpret_cast<PyCFunction>(reinterpret_cast<void*>(append)), METH_FASTCALL, nullptr},
    {"read", reinterpret_cast<PyCFunction>(reinterpret_cast<void*>(read)), METH_FASTCALL, nullptr},
    {"attend", reinterpret_cast<PyCFunction>(reinterpret_cast<void*>(attend)), METH_FASTCALL, nullptr},
    {"prepare", reinterpret_cast<PyCFunction>(reinterpret_cast<void*>(prepare)), METH_FASTCALL, nullptr},
    {nullptr, nullptr, 0, nullptr},
};

PyModuleDef module = {PyModuleDef_HEAD_INIT, "_torch_calls", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__torch_calls(void) { return PyModule_Create(&module); }
