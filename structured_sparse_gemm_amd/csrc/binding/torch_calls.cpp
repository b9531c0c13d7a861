// torch_calls.cpp -- the well-formed calls of the mx4, 8-bit float and expert
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
// means nothing, nor does any stride of no rows.  False for rows that repeat or
// overlap, and for columns apart.
bool row_stride(int64_t rows, int64_t cols, int64_t ld, int64_t unit, int64_t* out) {
    if (rows > 0 && cols > 1 && unit != 1) return false;
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

// ------------------------------------------------------------------ around the experts' products

bool integer(PyObject* o, int64_t* v) {
    if (!PyLong_Check(o)) return false;
    int over = 0;
    *v = PyLong_AsLongLongAndOverflow(o, &over);
    return !over;
}
bool word(PyObject* o, const char* w) { return PyUnicode_Check(o) && PyUnicode_CompareWithASCIIString(o, w) == 0; }
// The place of a word in a list of two, else -1.
int either(PyObject* o, const char* first, const char* second) { return word(o, first) ? 0 : word(o, second) ? 1 : -1; }
void* stream_of(int dev) { return (void*)c10::hip::getCurrentHIPStream((c10::DeviceIndex)dev).stream(); }

// A contiguous vector or matrix (cols >= 0) of this type and shape.
bool whole(const at::Tensor* t, at::ScalarType dt, int64_t rows, int64_t cols = -1) {
    return t && t->scalar_type() == dt && t->dim() == (cols < 0 ? 1 : 2) && t->size(0) == rows &&
           (cols < 0 || t->size(1) == cols) && t->is_contiguous();
}
// A matrix of this type and shape whose rows may be apart.
bool rows_of(const at::Tensor* t, at::ScalarType dt, int64_t rows, int64_t cols, Mat* m) {
    return t && t->scalar_type() == dt && mat(*t, m) && m->rows == rows && m->cols == cols;
}

// (logits, k, score, bias or None, groups, top_groups, group_score, renorm, scale) -> (weights, experts)
PyObject* route(PyObject*, PyObject* const* args, Py_ssize_t n) {
    if (n != 9) return none();
    const int dev = device_of(args[0]);
    int64_t k, groups, top_groups;
    const int score = either(args[2], "softmax", "sigmoid"), group_score = either(args[6], "max", "top2");
    if (dev < 0 || !integer(args[1], &k) || !integer(args[4], &groups) || !integer(args[5], &top_groups) || score < 0 ||
        group_score < 0 || !PyBool_Check(args[7]) || !PyFloat_Check(args[8]))
        return none();
    const at::Tensor* L = tensor(args[0], dev);
    const int dt = dtype_code(L->scalar_type());
    Mat l;
    if (dt < 0 || !mat(*L, &l) || k < 0 || k > l.cols) return none();
    const float* bias = nullptr;
    if (args[3] != Py_None) {
        const at::Tensor* b = tensor(args[3], dev);
        if (!whole(b, at::kFloat, l.cols)) return none();
        bias = (const float*)b->data_ptr();
    }
    at::Tensor W = at::empty({l.rows, k}, L->options().dtype(at::kFloat));
    at::Tensor X = at::empty({l.rows, k}, L->options().dtype(at::kInt));
    const int rc = ssg_route(dt, l.rows, l.cols, l.p, l.ld, bias, score, k, groups, top_groups, group_score,
                             args[7] == Py_True, (float)PyFloat_AS_DOUBLE(args[8]), (float*)W.data_ptr(), k,
                             (int32_t*)X.data_ptr(), k, stream_of(dev));
    if (rc != SSG_OK) return none();
    return Py_BuildValue("(NN)", THPVariable_Wrap(std::move(W)), THPVariable_Wrap(std::move(X)));
}

// (dweights, logits, experts, score, renorm, scale) -> dlogits
PyObject* route_backward(PyObject*, PyObject* const* args, Py_ssize_t n) {
    if (n != 6) return none();
    const int dev = device_of(args[0]), score = either(args[3], "softmax", "sigmoid");
    if (dev < 0 || score < 0 || !PyBool_Check(args[4]) || !PyFloat_Check(args[5])) return none();
    const at::Tensor *L = tensor(args[1], dev), *X = tensor(args[2], dev);
    Mat l, x, w;
    if (!L || !X || dtype_code(L->scalar_type()) < 0 || !mat(*L, &l) || X->dim() != 2) return none();
    const int64_t k = X->size(1);
    if (!rows_of(X, at::kInt, l.rows, k, &x) || !rows_of(tensor(args[0], dev), at::kFloat, l.rows, k, &w)) return none();
    at::Tensor D = at::empty({l.rows, l.cols}, L->options());
    const int rc = ssg_route_backward(dtype_code(L->scalar_type()), l.rows, l.cols, (float*)w.p, w.ld, l.p, l.ld,
                                      (int32_t*)x.p, x.ld, score, k, args[4] == Py_True,
                                      (float)PyFloat_AS_DOUBLE(args[5]), D.data_ptr(), l.cols, stream_of(dev));
    return rc == SSG_OK ? THPVariable_Wrap(std::move(D)) : none();
}

// (experts, E) -> (offs, rows, pos)
PyObject* expert_order(PyObject*, PyObject* const* args, Py_ssize_t n) {
    int64_t E;
    if (n != 2 || !integer(args[1], &E) || E < 0 || E >= 1 << 20) return none();
    const int dev = device_of(args[0]);
    if (dev < 0) return none();
    const at::Tensor* X = tensor(args[0], dev);
    Mat x;
    if (X->scalar_type() != at::kInt || !mat(*X, &x)) return none();
    const int64_t pairs = x.rows * x.cols;
    at::Tensor O = at::empty({E + 1}, X->options()), R = at::empty({pairs}, X->options()),
               P = at::empty({x.rows, x.cols}, X->options());
    const auto call = [&](void* ws, size_t bytes) {
        return ssg_expert_order(x.rows, x.cols, E, (int32_t*)x.p, x.ld, (int32_t*)O.data_ptr(), (int32_t*)R.data_ptr(),
                                (int32_t*)P.data_ptr(), ws, bytes, stream_of(dev));
    };
    const int rc = with_workspace(*X, call, [&] { return ssg_expert_order_workspace_bytes(x.rows, x.cols, E); });
    if (rc != SSG_OK) return none();
    return Py_BuildValue("(NNN)", THPVariable_Wrap(std::move(O)), THPVariable_Wrap(std::move(R)),
                         THPVariable_Wrap(std::move(P)));
}

// (X, pos, rows) -> Y
PyObject* expert_gather(PyObject*, PyObject* const* args, Py_ssize_t n) {
    if (n != 3) return none();
    const int dev = device_of(args[0]);
    if (dev < 0) return none();
    const at::Tensor *X = tensor(args[0], dev), *P = tensor(args[1], dev), *R = tensor(args[2], dev);
    Mat x;
    if (dtype_code(X->scalar_type()) < 0 || !mat(*X, &x) || !P || P->dim() != 2) return none();
    const int64_t k = P->size(1), pairs = x.rows * k;
    if (!whole(P, at::kInt, x.rows, k) || !whole(R, at::kInt, pairs)) return none();
    at::Tensor Y = at::empty({pairs, x.cols}, X->options());
    const int rc = ssg_expert_gather(dtype_code(X->scalar_type()), x.rows, k, x.cols, x.p, x.ld, (int32_t*)P->data_ptr(),
                                     (int32_t*)R->data_ptr(), Y.data_ptr(), x.cols, stream_of(dev));
    return rc == SSG_OK ? THPVariable_Wrap(std::move(Y)) : none();
}

// (Y, pos, weights or None, out dtype or None) -> O
PyObject* expert_combine(PyObject*, PyObject* const* args, Py_ssize_t n) {
    if (n != 4 || !(args[3] == Py_None || THPDtype_Check(args[3]))) return none();
    const int dev = device_of(args[0]);
    if (dev < 0) return none();
    const at::Tensor *Y = tensor(args[0], dev), *P = tensor(args[1], dev);
    const at::ScalarType out =
        args[3] == Py_None ? Y->scalar_type() : reinterpret_cast<THPDtype*>(args[3])->scalar_type;
    Mat y, w{nullptr, 0, 0, 0};
    if (dtype_code(Y->scalar_type()) < 0 || dtype_code(out) < 0 || !mat(*Y, &y) || !P || P->dim() != 2) return none();
    const int64_t N = P->size(0), k = P->size(1);
    if (!whole(P, at::kInt, N, k) || y.rows != N * k) return none();
    if (args[2] != Py_None && !rows_of(tensor(args[2], dev), at::kFloat, N, k, &w)) return none();
    at::Tensor O = at::empty({N, y.cols}, Y->options().dtype(out));
    const int rc = ssg_expert_combine(dtype_code(Y->scalar_type()), dtype_code(out), N, k, y.cols, y.p, y.ld,
                                      (int32_t*)P->data_ptr(), (float*)w.p, w.ld, O.data_ptr(), y.cols, stream_of(dev));
    return rc == SSG_OK ? THPVariable_Wrap(std::move(O)) : none();
}

// (dO, Y, pos, rows, weights) -> (dY, dweights)
PyObject* expert_combine_backward(PyObject*, PyObject* const* args, Py_ssize_t n) {
    if (n != 5) return none();
    const int dev = device_of(args[0]);
    if (dev < 0) return none();
    const at::Tensor *G = tensor(args[0], dev), *P = tensor(args[2], dev), *R = tensor(args[3], dev);
    const at::ScalarType dt = G->scalar_type();
    Mat g, y, w;
    if (dtype_code(dt) < 0 || !mat(*G, &g) || !P || P->dim() != 2) return none();
    const int64_t k = P->size(1), pairs = g.rows * k;
    if (!whole(P, at::kInt, g.rows, k) || !whole(R, at::kInt, pairs) ||
        !rows_of(tensor(args[1], dev), dt, pairs, g.cols, &y) ||
        !rows_of(tensor(args[4], dev), at::kFloat, g.rows, k, &w))
        return none();
    at::Tensor D = at::empty({pairs, g.cols}, G->options()), S = at::empty({g.rows, k}, G->options().dtype(at::kFloat));
    const int rc = ssg_expert_combine_backward(dtype_code(dt), g.rows, k, g.cols, g.p, g.ld, y.p, y.ld,
                                               (int32_t*)P->data_ptr(), (int32_t*)R->data_ptr(), (float*)w.p, w.ld,
                                               D.data_ptr(), g.cols, (float*)S.data_ptr(), k, stream_of(dev));
    if (rc != SSG_OK) return none();
    return Py_BuildValue("(NN)", THPVariable_Wrap(std::move(D)), THPVariable_Wrap(std::move(S)));
}

// ------------------------------------------------------------------ 8-bit floats

struct Scales {
    float* p = nullptr;
    int block = 1;
    int64_t row = 0, blk = 0, mat = 0;
};

// The scales of rows x cols elements (mats < 0: of a matrix, not a stack), for
// each row or each 128 rows; the stride of a single row or block means nothing.
bool scales(const at::Tensor* t, int64_t mats, int64_t rows, int64_t cols, Scales* s) {
    const int lead = mats >= 0;
    if (!t || t->scalar_type() != at::kFloat || t->dim() != 2 + lead || t->size(1 + lead) != (cols + 127) / 128 ||
        (lead && t->size(0) != mats))
        return false;
    const int64_t r = t->size(lead);
    s->block = r == rows ? 1 : 128;
    if (s->block == 128 && r != (rows + 127) / 128) return false;
    const auto stride = [&](int d) { return t->size(d) == 1 ? 1 : t->stride(d); };
    s->p = (float*)t->data_ptr();
    s->row = stride(lead);
    s->blk = stride(1 + lead);
    s->mat = lead ? stride(0) : 0;
    return true;
}

// A matrix as a stack of one, or a stack.
bool as_stack(const at::Tensor& t, Stack* s) {
    if (t.dim() == 3) return stack(t, s);
    Mat m;
    if (!mat(t, &m)) return false;
    *s = Stack{m.p, 1, m.rows, m.cols, m.ld, 0};
    return true;
}

// (A, block, transpose) -> (elems, scales)
PyObject* fp8_quantize(PyObject*, PyObject* const* args, Py_ssize_t n) {
    int64_t block;
    if (n != 3 || !integer(args[1], &block) || (block != 1 && block != 128) || !PyBool_Check(args[2])) return none();
    const int dev = device_of(args[0]);
    if (dev < 0) return none();
    const at::Tensor* A = tensor(args[0], dev);
    Stack a;
    if (dtype_code(A->scalar_type()) < 0 || !as_stack(*A, &a)) return none();
    const bool turn = args[2] == Py_True, lead = A->dim() == 3;
    const int64_t R = turn ? a.cols : a.rows, K = turn ? a.rows : a.cols, nb = (K + 127) / 128;
    const int64_t ld = (K + 15) / 16 * 16, rb = block == 1 ? (R + 3) / 4 * 4 : (R + 127) / 128;
    const auto made = [&](int64_t rows, int64_t cols, at::ScalarType dt) {
        return lead ? at::empty({a.mats, rows, cols}, A->options().dtype(dt)) : at::empty({rows, cols}, A->options().dtype(dt));
    };
    at::Tensor E = made(R, ld, at::kFloat8_e4m3fn);
    at::Tensor S = block == 1 ? made(nb, rb, at::kFloat) : made(rb, nb, at::kFloat);
    if (ld != K) E = E.narrow(-1, 0, K);
    if (block == 1) S = (rb == R ? S : S.narrow(-1, 0, R)).transpose(-1, -2);
    const int64_t row = block == 1 ? 1 : nb, blk = block == 1 ? rb : 1;
    const int rc = ssg_fp8_quantize(dtype_code(A->scalar_type()), a.mats, a.rows, a.cols, a.p, a.ld, a.stride,
                                    (int)block, turn, (uint8_t*)E.data_ptr(), ld, R * ld, (float*)S.data_ptr(), row, blk,
                                    rb * nb, stream_of(dev));
    if (rc != SSG_OK) return none();
    return Py_BuildValue("(NN)", THPVariable_Wrap(std::move(E)), THPVariable_Wrap(std::move(S)));
}

// (elems, scales, dtype) -> values
PyObject* fp8_dequantize(PyObject*, PyObject* const* args, Py_ssize_t n) {
    if (n != 3 || !THPDtype_Check(args[2])) return none();
    const int dev = device_of(args[0]);
    if (dev < 0) return none();
    const at::Tensor* E = tensor(args[0], dev);
    const at::ScalarType out = reinterpret_cast<THPDtype*>(args[2])->scalar_type;
    Stack e;
    Scales s;
    if (E->scalar_type() != at::kFloat8_e4m3fn || dtype_code(out) < 0 || !as_stack(*E, &e) ||
        !scales(tensor(args[1], dev), E->dim() == 3 ? e.mats : -1, e.rows, e.cols, &s))
        return none();
    at::Tensor D = at::empty(E->sizes(), E->options().dtype(out));
    const int rc = ssg_fp8_dequantize(dtype_code(out), e.mats, e.rows, e.cols, (uint8_t*)e.p, e.ld, e.stride, s.block,
                                      s.p, s.row, s.blk, s.mat, D.data_ptr(), e.cols, e.rows * e.cols, stream_of(dev));
    return rc == SSG_OK ? THPVariable_Wrap(std::move(D)) : none();
}

// (X, xscales or None, W, wscales, offs or None, out dtype) -> Y
PyObject* fp8_product(PyObject*, PyObject* const* args, Py_ssize_t n) {
    if (n != 6 || !THPDtype_Check(args[5])) return none();
    const int dev = device_of(args[0]);
    if (dev < 0) return none();
    const bool grouped = args[4] != Py_None;
    const at::Tensor *X = tensor(args[0], dev), *W = tensor(args[2], dev);
    const at::ScalarType out = reinterpret_cast<THPDtype*>(args[5])->scalar_type;
    const int y = dtype_code(out);
    Mat a;
    Stack w;
    Scales xs, s;
    if (!W || W->scalar_type() != at::kFloat8_e4m3fn || y < 0 || !mat(*X, &a) || W->dim() != 2 + grouped ||
        !as_stack(*W, &w) || w.cols != a.cols ||
        !scales(tensor(args[3], dev), grouped ? w.mats : -1, w.rows, w.cols, &s))
        return none();
    int x = dtype_code(X->scalar_type());
    if (args[1] != Py_None) {
        if (X->scalar_type() != at::kFloat8_e4m3fn || !scales(tensor(args[1], dev), -1, a.rows, a.cols, &xs) ||
            xs.block != 1)
            return none();
        x = SSG_E4M3;
    }
    if (x < 0) return none();
    void* const stream = stream_of(dev);
    const int64_t M = w.rows, N = a.rows, K = a.cols;
    if (!grouped) {
        at::Tensor Y = at::empty({N, M}, X->options().dtype(out));
        const int rc = with_workspace(
            *X,
            [&](void* ws, size_t bytes) {
                return ssg_mm_fp8(x, y, M, N, K, a.p, a.ld, xs.p, xs.row, xs.blk, (uint8_t*)w.p, w.ld, s.block, s.p,
                                  s.row, s.blk, Y.data_ptr(), M, ws, bytes, stream);
            },
            [&] {
                return ssg_mm_fp8_workspace_bytes(x, y, M, N, K, a.p, a.ld, xs.p, xs.row, xs.blk, (uint8_t*)w.p, w.ld,
                                                  s.block, s.p, s.row, s.blk);
            });
        return rc == SSG_OK ? THPVariable_Wrap(std::move(Y)) : none();
    }
    const at::Tensor* offs = tensor(args[4], dev);
    if (!whole(offs, at::kInt, w.mats + 1)) return none();
    const int32_t* const o = (const int32_t*)offs->data_ptr();
    at::Tensor Y = at::empty({N, M}, X->options().dtype(out));
    const int rc = with_workspace(
        *X,
        [&](void* ws, size_t bytes) {
            return ssg_grouped_mm_fp8(x, y, w.mats, M, N, K, a.p, a.ld, xs.p, xs.row, xs.blk, (uint8_t*)w.p, w.ld,
                                      w.stride, s.block, s.p, s.row, s.blk, s.mat, o, Y.data_ptr(), M, ws, bytes,
                                      stream);
        },
        [&] {
            return ssg_grouped_mm_fp8_workspace_bytes(x, y, w.mats, M, N, K, a.p, a.ld, xs.p, xs.row, xs.blk,
                                                      (uint8_t*)w.p, w.ld, w.stride, s.block, s.p, s.row, s.blk, s.mat,
                                                      o);
        });
    return rc == SSG_OK ? THPVariable_Wrap(std::move(Y)) : none();
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
    {"route", (PyCFunction)(void*)guarded<route>, METH_FASTCALL, nullptr},
    {"route_backward", (PyCFunction)(void*)guarded<route_backward>, METH_FASTCALL, nullptr},
    {"expert_order", (PyCFunction)(void*)guarded<expert_order>, METH_FASTCALL, nullptr},
    {"expert_gather", (PyCFunction)(void*)guarded<expert_gather>, METH_FASTCALL, nullptr},
    {"expert_combine", (PyCFunction)(void*)guarded<expert_combine>, METH_FASTCALL, nullptr},
    {"expert_combine_backward", (PyCFunction)(void*)guarded<expert_combine_backward>, METH_FASTCALL, nullptr},
    {"fp8_quantize", (PyCFunction)(void*)guarded<fp8_quantize>, METH_FASTCALL, nullptr},
    {"fp8_dequantize", (PyCFunction)(void*)guarded<fp8_dequantize>, METH_FASTCALL, nullptr},
    {"fp8_product", (PyCFunction)(void*)guarded<fp8_product>, METH_FASTCALL, nullptr},
    {nullptr, nullptr, 0, nullptr},
};
PyModuleDef kModule = {PyModuleDef_HEAD_INIT, "_torch_calls", nullptr, -1, kMethods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

extern "C" __attribute__((visibility("default"))) PyObject* PyInit__torch_calls() { return PyModule_Create(&kModule); }
