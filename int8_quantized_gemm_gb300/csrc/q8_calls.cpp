// The common calls of the 4-bit operators without the interpreter's steps: a decode step makes many of them, and the kernels of
// small batches take less time than the marshalling in Python (one token quantized: 11.3 us a call there). Each function checks its
// arguments as the binding does, allocates the results on the current stream and calls the C ABI. What it does not take (other
// arguments than the common ones, wrong ones, any error) it leaves to the binding by returning None before anything is queued; the
// binding then names what is wrong.
#include <Python.h>

#include <ATen/core/Tensor.h>
#include <ATen/ops/empty.h>
#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/Dtype.h>
#include <torch/csrc/autograd/python_variable.h>

#include "../../include/q8.h"

namespace {

decltype(&q8_quantize_fp4) quantize_entry = nullptr;
decltype(&q8_swiglu_quantize_fp4) swiglu_entry = nullptr;
decltype(&q8_dequantize_fp4) dequantize_entry = nullptr;
decltype(&q8_gemm_fp4) gemm_entry = nullptr;
decltype(&q8_gemm_fp4_grouped) grouped_entry = nullptr;

constexpr int64_t kSpan = 256;   // K that a row's scales are padded to

int64_t cdiv(int64_t a, int64_t b) { return (a + b - 1) / b; }
int64_t pitch_of(int64_t K, int block) { return cdiv(K, kSpan) * (kSpan / block); }

// A plain tensor (no subclass), or nullptr.
const at::Tensor* plain(PyObject* o) { return THPVariable_CheckExact(o) ? &THPVariable_Unpack(o) : nullptr; }

bool float_type(at::ScalarType t, q8_float_type& type) {
    switch (t) {
        case at::kFloat: type = Q8_F32; return true;
        case at::kBFloat16: type = Q8_BF16; return true;
        case at::kHalf: type = Q8_F16; return true;
        default: return false;
    }
}

// A contiguous tensor of this type and shape on the device.
bool dense(const at::Tensor* t, at::ScalarType type, c10::IntArrayRef shape, int device) {
    return t && t->scalar_type() == type && t->is_cuda() && t->get_device() == device && t->sizes() == shape && t->is_contiguous();
}

at::Tensor fresh(c10::IntArrayRef shape, at::ScalarType type, int device) {
    return at::empty(shape, at::TensorOptions().dtype(type).device(at::kCUDA, (c10::DeviceIndex)device));
}

q8_stream_t current_stream(int device) {
    return reinterpret_cast<q8_stream_t>(c10::cuda::getCurrentCUDAStream((c10::DeviceIndex)device).stream());
}

template <class T>
T* address(const at::Tensor& t) { return static_cast<T*>(t.data_ptr()); }

// A matrix of floats with unit stride along its rows, on the current device.
struct Rows {
    const void* x;
    q8_float_type type;
    int64_t M, cols, pitch;
    int device;
};
bool rows_of(PyObject* o, Rows& r) {
    const at::Tensor* t = plain(o);
    if (!t || !t->is_cuda() || t->dim() != 2 || !float_type(t->scalar_type(), r.type)) return false;
    r.M = t->size(0);
    r.cols = t->size(1);
    r.device = t->get_device();
    if ((t->stride(1) != 1 && r.cols > 1) || r.device != c10::cuda::current_device()) return false;
    r.pitch = r.M <= 1 ? r.cols : t->stride(0);
    if (r.pitch < r.cols) return false;
    r.x = t->data_ptr();
    return true;
}

// Codes, block scales and row scales of `rows` rows, as a tuple (q, sf, s or None).
struct Codes {
    at::Tensor q, sf, s;
    Codes(int64_t rows, int64_t K, int block, int device)
        : q(fresh({rows, K / 2}, at::kByte, device)),
          sf(fresh({rows, pitch_of(K, block)}, block == 16 ? at::kFloat8_e4m3fn : at::kFloat8_e8m0fnu, device)) {
        if (block == 16) s = fresh({rows}, at::kFloat, device);
    }
    float* row_scales() const { return s.defined() ? address<float>(s) : nullptr; }
    PyObject* tuple() {
        PyObject* a = THPVariable_Wrap(std::move(q));
        PyObject* b = THPVariable_Wrap(std::move(sf));
        PyObject* c = s.defined() ? THPVariable_Wrap(std::move(s)) : Py_NewRef(Py_None);
        PyObject* r = a && b && c ? PyTuple_Pack(3, a, b, c) : nullptr;
        Py_XDECREF(a);
        Py_XDECREF(b);
        Py_XDECREF(c);
        return r;
    }
};

bool block_of(PyObject* o, int& block) {
    if (!PyLong_CheckExact(o)) return false;
    const long v = PyLong_AsLong(o);
    if (v != 16 && v != 32) {
        PyErr_Clear();
        return false;
    }
    block = (int)v;
    return true;
}

// Runs a call; whatever goes wrong in it is left to the binding.
template <class F>
PyObject* guarded(F f) {
    try {
        PyObject* r = f();
        if (r) return r;
    } catch (...) {
    }
    PyErr_Clear();
    Py_RETURN_NONE;
}

// quantize_fp4(x, block, slots or None)
PyObject* quantize_fp4(PyObject*, PyObject* const* a, Py_ssize_t n) {
    return guarded([&]() -> PyObject* {
        Rows r;
        int block;
        if (n != 3 || !rows_of(a[0], r) || !block_of(a[1], block) || r.cols % 32) return nullptr;
        int64_t rows = r.M, top_k = 0;
        const int32_t* to = nullptr;
        if (a[2] != Py_None) {
            const at::Tensor* slots = plain(a[2]);
            if (!slots || slots->dim() != 2) return nullptr;
            top_k = slots->size(1);
            if (!dense(slots, at::kInt, {r.M, top_k}, r.device)) return nullptr;
            to = address<const int32_t>(*slots);
            rows = r.M * top_k;
        }
        Codes c(rows, r.cols, block, r.device);
        if (quantize_entry(r.x, r.type, block, r.M, r.cols, r.pitch, to, top_k, rows, address<uint8_t>(c.q), address<uint8_t>(c.sf),
                           c.row_scales(), current_stream(r.device)) != Q8_OK)
            return nullptr;
        return c.tuple();
    });
}

// swiglu_quantize_fp4(h, block)
PyObject* swiglu_quantize_fp4(PyObject*, PyObject* const* a, Py_ssize_t n) {
    return guarded([&]() -> PyObject* {
        Rows r;
        int block;
        if (n != 2 || !rows_of(a[0], r) || !block_of(a[1], block) || r.cols % 64) return nullptr;
        Codes c(r.M, r.cols / 2, block, r.device);
        if (swiglu_entry(r.x, r.type, block, r.M, r.cols / 2, r.pitch, address<uint8_t>(c.q), address<uint8_t>(c.sf), c.row_scales(),
                         current_stream(r.device)) != Q8_OK)
            return nullptr;
        return c.tuple();
    });
}

// dequantize_fp4(q, out_dtype): the codes alone
PyObject* dequantize_fp4(PyObject*, PyObject* const* a, Py_ssize_t n) {
    return guarded([&]() -> PyObject* {
        const at::Tensor* q = n == 2 ? plain(a[0]) : nullptr;
        if (!q || !THPDtype_Check(a[1]) || q->scalar_type() != at::kByte || !q->is_cuda() || q->dim() != 2 || !q->is_contiguous())
            return nullptr;
        const at::ScalarType out = reinterpret_cast<THPDtype*>(a[1])->scalar_type;
        q8_float_type type;
        if (out == at::kFloat8_e4m3fn) type = Q8_E4M3;
        else if (!float_type(out, type)) return nullptr;
        const int device = q->get_device();
        if (device != c10::cuda::current_device()) return nullptr;
        const int64_t rows = q->size(0), K = 2 * q->size(1);
        at::Tensor y = fresh({rows, K}, out, device);
        if (dequantize_entry(address<const uint8_t>(*q), nullptr, nullptr, 16, rows, K, 0, y.data_ptr(), type, current_stream(device)) !=
            Q8_OK)
            return nullptr;
        return THPVariable_Wrap(std::move(y));
    });
}

// gemm_fp4(qa, sfa, sa or None, qw, sfw, sw or None, offsets or None, out_dtype)
PyObject* gemm_fp4(PyObject*, PyObject* const* a, Py_ssize_t n) {
    return guarded([&]() -> PyObject* {
        if (n != 8 || !THPDtype_Check(a[7])) return nullptr;
        const bool grouped = a[6] != Py_None;
        const at::Tensor *qa = plain(a[0]), *sfa = plain(a[1]), *qw = plain(a[3]);
        const at::ScalarType out = reinterpret_cast<THPDtype*>(a[7])->scalar_type;
        q8_float_type type;
        if (!qa || !sfa || !qw || !qa->is_cuda() || qa->dim() != 2 || qw->dim() != (grouped ? 3 : 2) || !float_type(out, type))
            return nullptr;
        const at::ScalarType scales = sfa->scalar_type();
        if (scales != at::kFloat8_e4m3fn && scales != at::kFloat8_e8m0fnu) return nullptr;
        const int block = scales == at::kFloat8_e4m3fn ? 16 : 32, device = qa->get_device();
        const int64_t M = qa->size(0), half = qa->size(1), K = 2 * half, E = grouped ? qw->size(0) : 1, N = qw->size(-2);
        const int64_t pitch = pitch_of(K, block);
        if (device != c10::cuda::current_device() || !dense(qa, at::kByte, {M, half}, device) ||
            !dense(sfa, scales, {M, pitch}, device))
            return nullptr;
        const float *sa = nullptr, *sw = nullptr;
        if (a[2] != Py_None) {
            const at::Tensor* t = plain(a[2]);
            if (!dense(t, at::kFloat, {M}, device)) return nullptr;
            sa = address<const float>(*t);
        }
        const at::Tensor *sfw = plain(a[4]), *tw = a[5] == Py_None ? nullptr : plain(a[5]);
        if (a[5] != Py_None && !tw) return nullptr;
        const int32_t* offsets = nullptr;
        if (grouped) {
            const at::Tensor* t = plain(a[6]);
            if (!dense(qw, at::kByte, {E, N, half}, device) || !dense(sfw, scales, {E, cdiv(N, 128), pitch / 4, 32, 4, 4}, device) ||
                (tw && !dense(tw, at::kFloat, {E, N}, device)) || !dense(t, at::kInt, {E + 1}, device))
                return nullptr;
            offsets = address<const int32_t>(*t);
        } else if (!dense(qw, at::kByte, {N, half}, device) || !dense(sfw, scales, {cdiv(N, 128), pitch / 4, 32, 4, 4}, device) ||
                   (tw && !dense(tw, at::kFloat, {N}, device))) {
            return nullptr;
        }
        if (tw) sw = address<const float>(*tw);
        at::Tensor y = fresh({M, N}, out, device);
        const uint8_t *pa = address<const uint8_t>(*qa), *psa = address<const uint8_t>(*sfa), *pw = address<const uint8_t>(*qw),
                      *psw = address<const uint8_t>(*sfw);
        const q8_stream_t stream = current_stream(device);
        const q8_status st = grouped ? grouped_entry(pa, psa, sa, pw, psw, sw, offsets, block, M, E, N, K, y.data_ptr(), type, stream)
                                     : gemm_entry(pa, psa, sa, pw, psw, sw, block, M, N, K, y.data_ptr(), type, stream);
        return st == Q8_OK ? THPVariable_Wrap(std::move(y)) : nullptr;
    });
}

// entries(addresses of the five C entry points, in the order of their declaration above)
PyObject* entries(PyObject*, PyObject* const* a, Py_ssize_t n) {
    void* p[5];
    if (n != 5) {
        PyErr_SetString(PyExc_TypeError, "five addresses");
        return nullptr;
    }
    for (int i = 0; i < 5; ++i) {
        p[i] = PyLong_AsVoidPtr(a[i]);
        if (!p[i]) {
            if (!PyErr_Occurred()) PyErr_SetString(PyExc_ValueError, "no address");
            return nullptr;
        }
    }
    quantize_entry = reinterpret_cast<decltype(quantize_entry)>(p[0]);
    swiglu_entry = reinterpret_cast<decltype(swiglu_entry)>(p[1]);
    dequantize_entry = reinterpret_cast<decltype(dequantize_entry)>(p[2]);
    gemm_entry = reinterpret_cast<decltype(gemm_entry)>(p[3]);
    grouped_entry = reinterpret_cast<decltype(grouped_entry)>(p[4]);
    Py_RETURN_NONE;
}

#define Q8_FAST(f) reinterpret_cast<PyCFunction>(reinterpret_cast<void*>(f)), METH_FASTCALL, nullptr
PyMethodDef methods[] = {{"entries", Q8_FAST(entries)},
                         {"quantize_fp4", Q8_FAST(quantize_fp4)},
                         {"swiglu_quantize_fp4", Q8_FAST(swiglu_quantize_fp4)},
                         {"dequantize_fp4", Q8_FAST(dequantize_fp4)},
                         {"gemm_fp4", Q8_FAST(gemm_fp4)},
                         {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_q8_calls", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__q8_calls() { return PyModule_Create(&module); }
