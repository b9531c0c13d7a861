// torch_calls.cpp -- the well-formed calls of the mx4 and expert-grouped
// operators, marshalled from torch tensors into the C ABI without the
// interpreter.  A product of one token runs for 5 us on the GPU; the call takes
// 11 us of host time through the interpreter and 4.3 us here, 3 of them the launch.
//
// Every function returns None for a call that is not well-formed (types,
// shapes, strides, devices) or that the library refuses; the Python binding
// then makes the same call itself and reports what is wrong.  No computation
// happens here and no state is kept.
#include <Python.h>

#include <ATen/ATen.h>
#include <ATen/ops/empty.h>
#include <c10/hip/HIPFunctions.h>
#include <c10/hip/HIPStream.h>
#include <torch/csrc/Dtype.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include "ssgemm.h"

namespace {

struct Mat {
    void* p;
    int64_t rows, cols, ld;
};
struct Stack {
    void* p;
    int64_t mats, rows, cols, ld, stride;
};

// The current device if a tensor is on it, else -1 (also on a machine without one).
int device_of(PyObject* o) {
    if (!THPVariable_Check(o)) return -1;
    const at::Tensor& t = THPVariable_Unpack(o);
    if (!t.is_cuda()) return -1;
    const int dev = c10::hip::current_device();
    return t.get_device() == dev ? dev : -1;
}

// A tensor on the device, else nullptr.
const at::Tensor* tensor(PyObject* o, int device) {
    if (!THPVariable_Check(o)) return nullptr;
    const at::Tensor& t = THPVariable_Unpack(o);
    return t.is_cuda() && t.get_device() == device ? &t : nullptr;
}

// Row stride of rows x cols; that of a single row, or of rows without columns,
// means nothing.  False for rows that repeat or overlap, and for columns apart.
bool row_stride(int64_t rows, int64_t cols, int64_t ld, int64_t unit, int64_t* out) {
    if (cols > 1 && unit != 1) return false;
    const bool any = rows <= 1 || cols == 0;
    *out = any ? cols : ld;
    return any || ld >= cols;
}

bool mat(const at::Tensor& t, Mat* m) {
    if (t.dim() != 2) return false;
    m->rows = t.size(0);
    m->cols = t.size(1);
    if (!row_stride(m->rows, m->cols, t.stride(0), t.stride(1), &m->ld)) return false;
    m->p = t.data_ptr();
    return true;
}

bool stack(const at::Tensor& t, Stack* s) {
    if (t.dim() != 3) return false;
    s->mats = t.size(0);
    s->rows = t.size(1);
    s->cols = t.size(2);
    if (!row_stride(s->rows, s->cols, t.stride(1), t.stride(2), &s->ld)) return false;
    s->stride = s->mats > 1 ? t.stride(0) : s->rows * s->ld;
    s->p = t.data_ptr();
    return true;
}

int dtype_code(at::ScalarType t) {
    switch (t) {
        case at::kHalf: return SSG_F16;
        case at::kBFloat16: return SSG_BF16;
        case at::kFloat: return SSG_F32;
        default: return -1;
    }
}
bool is16(int dt) { return dt == SSG_F16 || dt == SSG_BF16; }

PyObject* none() { Py_RETURN_NONE; }

// `call` with a workspace (pointer, bytes): none first, then of the size that `need` gives.
template <typename Call, typename Need>
int with_workspace(const at::Tensor& like, Call&& call, Need&& need) {
    int rc = call(nullptr, SSG_WS_ASK);
    if (rc == SSG_ERR_WORKSPACE) {
        const size_t n = need();
        const at::Tensor ws = at::empty({(int64_t)n}, like.options().dtype(at::kByte));
        rc = call(ws.data_ptr(), n);
    }
    return rc;
}

// mx4 products: (X, xscales or None, W, scales, offs or None, out dtype)
PyObject* mx4_product(PyObject*, PyObject* const* args, Py_ssize_t n) {
    if (n != 6 || !THPDtype_Check(args[5])) return none();
    const int dev = device_of(args[0]);
    if (dev < 0) return none();
    const bool grouped = args[4] != Py_None, mx = args[1] != Py_None;
    const at::Tensor *X = tensor(args[0], dev), *W = tensor(args[2], dev), *S = tensor(args[3], dev);
    if (!X || !W || !S || W->scalar_type() != at::kByte || S->scalar_type() != at::kByte) return none();
    const at::ScalarType out = reinterpret_cast<THPDtype*>(args[5])->scalar_type;
    const int y = dtype_code(out), x = mx ? SSG_MX4 : dtype_code(X->scalar_type());
    Mat mx_x, mx_s{nullptr, 0, 0, 0};
    if (y < 0 || x < 0 || !mat(*X, &mx_x) || (mx && X->scalar_type() != at::kByte) || (!mx && !is16(x))) return none();
    const int64_t K = mx ? 2 * mx_x.cols : mx_x.cols, nb = (K + 31) / 32, N = mx_x.rows;
    if (mx) {
        const at::Tensor* xs = tensor(args[1], dev);
        if (mx_x.cols % 16) return none();             // mx4 rows are whole blocks
        if (!xs || xs->scalar_type() != at::kByte || !mat(*xs, &mx_s) || mx_s.rows != N || mx_s.cols != nb) return none();
    }
    uint8_t* const xs = (uint8_t*)mx_s.p;
    void* const stream = (void*)c10::hip::getCurrentHIPStream((c10::DeviceIndex)dev).stream();
    if (!grouped) {
        Mat w, s;
        if (!mat(*W, &w) || !mat(*S, &s) || w.cols != 16 * nb || s.rows != w.rows || s.cols != nb) return none();
        at::Tensor Y = at::empty({N, w.rows}, X->options().dtype(out));
        const int rc = with_workspace(
            *X,
            [&](void* ws, size_t bytes) {
                return ssg_mm_mx4(x, y, w.rows, N, K, mx_x.p, mx_x.ld, xs, mx_s.ld, (uint8_t*)w.p, w.ld, (uint8_t*)s.p,
                                  s.ld, Y.data_ptr(), w.rows, ws, bytes, stream);
            },
            [&] {
                return ssg_mm_mx4_workspace_bytes(x, w.rows, N, K, mx_x.p, mx_x.ld, xs, mx_s.ld, (uint8_t*)w.p, w.ld,
                                                  (uint8_t*)s.p, s.ld);
            });
        return rc == SSG_OK ? THPVariable_Wrap(std::move(Y)) : none();
    }
    Stack w, s;
    const at::Tensor* offs = tensor(args[4], dev);
    if (!offs || offs->scalar_type() != at::kInt || offs->dim() != 1 || !offs->is_contiguous()) return none();
    if (!stack(*W, &w) || !stack(*S, &s) || w.cols != 16 * nb || s.mats != w.mats || s.rows != w.rows || s.cols != nb ||
        offs->size(0) != w.mats + 1)
        return none();
    const int32_t* const o = (const int32_t*)offs->data_ptr();
    at::Tensor Y = at::empty({N, w.rows}, X->options().dtype(out));
    const int rc = with_workspace(
        *X,
        [&](void* ws, size_t bytes) {
            return ssg_grouped_mm_mx4(x, y, w.mats, w.rows, N, K, mx_x.p, mx_x.ld, xs, mx_s.ld, (uint8_t*)w.p, w.ld,
                                      w.stride, (uint8_t*)s.p, s.ld, s.stride, o, Y.data_ptr(), w.rows, ws, bytes,
                                      stream);
        },
        [&] {
            return ssg_grouped_mm_mx4_workspace_bytes(x, w.mats, w.rows, N, K, mx_x.p, mx_x.ld, xs, mx_s.ld,
                                                      (uint8_t*)w.p, w.ld, w.stride, (uint8_t*)s.p, s.ld, s.stride, o);
        });
    return rc == SSG_OK ? THPVariable_Wrap(std::move(Y)) : none();
}

// 16-bit products: (kind, A, B, offs, out dtype); kind 0: Y = A B_e^T, 1: dX = A B_e,
// 2: dW_e = A_e^T B_e
PyObject* grouped_product(PyObject*, PyObject* const* args, Py_ssize_t n) {
    if (n != 5 || !THPDtype_Check(args[4])) return none();
    const long kind = PyLong_AsLong(args[0]);
    const int dev = device_of(args[1]);
    if (dev < 0) return none();
    const at::Tensor *A = tensor(args[1], dev), *B = tensor(args[2], dev), *offs = tensor(args[3], dev);
    if (!A || !B || !offs || A->scalar_type() != B->scalar_type()) return none();
    const at::ScalarType out = reinterpret_cast<THPDtype*>(args[4])->scalar_type;
    const int x = dtype_code(A->scalar_type()), y = dtype_code(out);
    Mat a;
    if (!is16(x) || y < 0 || !mat(*A, &a)) return none();
    if (offs->scalar_type() != at::kInt || offs->dim() != 1 || offs->size(0) < 1 || !offs->is_contiguous()) return none();
    const int64_t E = offs->size(0) - 1;
    const int32_t* const o = (const int32_t*)offs->data_ptr();
    void* const stream = (void*)c10::hip::getCurrentHIPStream((c10::DeviceIndex)dev).stream();
    at::Tensor Y;
    int rc;
    if (kind == 2) {
        Mat b;
        if (!mat(*B, &b) || b.rows != a.rows) return none();
        const int64_t M = a.cols, K = b.cols;
        Y = at::empty({E, M, K}, A->options().dtype(out));
        rc = with_workspace(
            *A,
            [&](void* ws, size_t bytes) {
                return ssg_grouped_mm_dw(x, y, E, M, a.rows, K, a.p, a.ld, b.p, b.ld, o, Y.data_ptr(), K, M * K, ws,
                                         bytes, stream);
            },
            [&] { return ssg_grouped_mm_dw_workspace_bytes(x, E, M, a.rows, K, a.p, a.ld, b.p, b.ld, o); });
    } else {
        Stack b;
        if (!stack(*B, &b) || b.mats != E || a.cols != (kind == 0 ? b.cols : b.rows)) return none();
        const int64_t M = b.rows, K = b.cols, q = kind == 0 ? M : K;
        Y = at::empty({a.rows, q}, A->options().dtype(out));
        auto* const f = kind == 0 ? ssg_grouped_mm : ssg_grouped_mm_dx;
        auto* const g = kind == 0 ? ssg_grouped_mm_workspace_bytes : ssg_grouped_mm_dx_workspace_bytes;
        rc = with_workspace(
            *A,
            [&](void* ws, size_t bytes) {
                return f(x, y, E, M, a.rows, K, a.p, a.ld, b.p, b.ld, b.stride, o, Y.data_ptr(), q, ws, bytes, stream);
            },
            [&] { return g(x, E, M, a.rows, K, a.p, a.ld, b.p, b.ld, b.stride, o); });
    }
    return rc == SSG_OK ? THPVariable_Wrap(std::move(Y)) : none();
}

// (A) -> (elems, scales)
PyObject* mx4_quantize(PyObject*, PyObject* arg) {
    const int dev = device_of(arg);
    if (dev < 0) return none();
    const at::Tensor* A = tensor(arg, dev);
    Mat a;
    if (!A || dtype_code(A->scalar_type()) < 0 || !mat(*A, &a)) return none();
    const int64_t nb = (a.cols + 31) / 32;
    const auto u8 = A->options().dtype(at::kByte);
    at::Tensor e = at::empty({a.rows, 16 * nb}, u8), s = at::empty({a.rows, nb}, u8);
    const int rc = ssg_mx4_quantize(dtype_code(A->scalar_type()), a.rows, a.cols, a.p, a.ld, (uint8_t*)e.data_ptr(),
                                    16 * nb, (uint8_t*)s.data_ptr(), nb,
                                    (void*)c10::hip::getCurrentHIPStream((c10::DeviceIndex)dev).stream());
    if (rc != SSG_OK) return none();
    return Py_BuildValue("(NN)", THPVariable_Wrap(std::move(e)), THPVariable_Wrap(std::move(s)));
}

// (elems, scales, K, dtype) -> values
PyObject* mx4_dequantize(PyObject*, PyObject* const* args, Py_ssize_t n) {
    if (n != 4 || !PyLong_Check(args[2]) || !THPDtype_Check(args[3])) return none();
    const int dev = device_of(args[0]);
    if (dev < 0) return none();
    const at::Tensor *E = tensor(args[0], dev), *S = tensor(args[1], dev);
    const int64_t K = PyLong_AsLongLong(args[2]);
    const at::ScalarType out = reinterpret_cast<THPDtype*>(args[3])->scalar_type;
    Mat e, s;
    if (!E || !S || K < 0 || dtype_code(out) < 0 || E->scalar_type() != at::kByte || S->scalar_type() != at::kByte ||
        !mat(*E, &e) || !mat(*S, &s))
        return none();
    const int64_t nb = (K + 31) / 32;
    if (e.cols != 16 * nb || s.cols != nb || s.rows != e.rows) return none();
    at::Tensor D = at::empty({e.rows, K}, E->options().dtype(out));
    const int rc = ssg_mx4_dequantize(dtype_code(out), e.rows, K, (uint8_t*)e.p, e.ld, (uint8_t*)s.p, s.ld,
                                      D.data_ptr(), K,
                                      (void*)c10::hip::getCurrentHIPStream((c10::DeviceIndex)dev).stream());
    return rc == SSG_OK ? THPVariable_Wrap(std::move(D)) : none();
}

// C++ exceptions (an allocation that fails) become torch's Python ones.
template <PyObject* (*F)(PyObject*, PyObject* const*, Py_ssize_t)>
PyObject* guarded(PyObject* self, PyObject* const* args, Py_ssize_t n) {
    HANDLE_TH_ERRORS
    return F(self, args, n);
    END_HANDLE_TH_ERRORS
}
PyObject* quantize_one(PyObject* self, PyObject* const* args, Py_ssize_t n) {
    return n == 1 ? mx4_quantize(self, args[0]) : none();
}

PyMethodDef kMethods[] = {
    {"mx4_product", (PyCFunction)(void*)guarded<mx4_product>, METH_FASTCALL, nullptr},
    {"grouped_product", (PyCFunction)(void*)guarded<grouped_product>, METH_FASTCALL, nullptr},
    {"mx4_quantize", (PyCFunction)(void*)guarded<quantize_one>, METH_FASTCALL, nullptr},
    {"mx4_dequantize", (PyCFunction)(void*)guarded<mx4_dequantize>, METH_FASTCALL, nullptr},
    {nullptr, nullptr, 0, nullptr},
};
PyModuleDef kModule = {PyModuleDef_HEAD_INIT, "_torch_calls", nullptr, -1, kMethods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

extern "C" __attribute__((visibility("default"))) PyObject* PyInit__torch_calls() { return PyModule_Create(&kModule); }
