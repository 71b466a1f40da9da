// The plain calls of gemm_w4, norm_residual and norm_residual_backward from torch tensors:
// checks, allocation of the results and the C entry point in one native call.  On single
// tokens the host's work is the time of a call: read attribute by attribute from Python,
// norm_residual on one row took 18 us, of which the kernel runs 2.6; from here it takes 4.6.
//
// A function returns its results, a status (int) if the entry point reports one, or None
// where the call is not plain (another stream or device, results given, anything that a
// check refuses): the caller then takes the general way, which has the errors' words.
#include <ATen/cuda/EmptyTensor.h>
#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/Dtype.h>
#include <torch/csrc/autograd/python_variable.h>

#include <cstring>
#include <optional>

#include "tgemm.h"

namespace {

decltype(&tg_gemm_w4) g_w4 = nullptr;
decltype(&tg_norm_residual) g_norm = nullptr;
decltype(&tg_norm_residual_backward) g_norm_backward = nullptr;
PyTypeObject* g_grads = nullptr;  // a named tuple of five

// A CUDA tensor with storage of its own, or nullptr.
const at::Tensor* plain(PyObject* o) {
    if (!THPVariable_Check(o)) return nullptr;
    const at::Tensor& t = THPVariable_Unpack(o);
    const c10::TensorImpl* impl = t.unsafeGetTensorImpl();
    return t.is_cuda() && t.layout() == c10::kStrided && !impl->is_python_dispatch() && impl->has_storage()
               ? &t
               : nullptr;
}

struct Matrix {
    void* p = nullptr;
    int64_t ld = 0, rows = 0, cols = 0;
};

// A row-major matrix of this type on this device; rows and cols are its own if negative.
bool matrix(PyObject* o, at::ScalarType type, int64_t rows, int64_t cols, int index, Matrix* m) {
    const at::Tensor* t = plain(o);
    if (t == nullptr || t->scalar_type() != type || t->dim() != 2 || t->get_device() != index) return false;
    m->rows = t->size(0);
    m->cols = t->size(1);
    if ((rows >= 0 && m->rows != rows) || (cols >= 0 && m->cols != cols)) return false;
    if (t->stride(1) != 1 && m->cols > 1) return false;
    m->p = t->data_ptr();
    // a single row's stride is never used
    m->ld = m->rows > 1 ? t->stride(0) : (m->cols + 15) / 16 * 16;
    return true;
}
bool vector(PyObject* o, int64_t size, int index, const float** p) {
    if (o == Py_None) return true;
    const at::Tensor* t = plain(o);
    if (t == nullptr || t->scalar_type() != at::kFloat || t->dim() != 1 || t->size(0) != size ||
        t->get_device() != index || (size > 1 && t->stride(0) != 1))
        return false;
    *p = static_cast<const float*>(t->data_ptr());
    return true;
}
bool code_of(at::ScalarType type, int32_t* code) {
    *code = type == at::kHalf ? TG_DTYPE_F16 : type == at::kBFloat16 ? TG_DTYPE_BF16 : TG_DTYPE_F32;
    return type == at::kHalf || type == at::kBFloat16 || type == at::kFloat;
}
bool integer(PyObject* o, int64_t* v) {
    if (!PyLong_CheckExact(o)) return false;
    int overflow = 0;
    *v = PyLong_AsLongLongAndOverflow(o, &overflow);
    return overflow == 0;
}
bool number(PyObject* o, float* v) {
    if (!PyFloat_CheckExact(o) && !PyLong_CheckExact(o)) return false;
    const double d = PyFloat_AsDouble(o);
    *v = static_cast<float>(d);
    if (d != -1.0 || PyErr_Occurred() == nullptr) return true;
    PyErr_Clear();
    return false;
}
at::Tensor empty(at::IntArrayRef sizes, at::ScalarType type, int index) {
    return at::Tensor(at::detail::empty_cuda(sizes, type, c10::Device(c10::kCUDA, static_cast<c10::DeviceIndex>(index)),
                                             std::nullopt));
}
bool here(int index) { return c10::cuda::current_device() == index; }
void* stream_of(int index) {
    return c10::cuda::getCurrentCUDAStream(static_cast<c10::DeviceIndex>(index)).stream();
}
PyObject* wrap(const at::Tensor& t) {
    if (!t.defined()) Py_RETURN_NONE;
    return THPVariable_Wrap(t);
}
PyObject* tuple_of(const at::Tensor* t, Py_ssize_t n) {
    PyObject* made = PyTuple_New(n);
    if (made == nullptr) return nullptr;
    for (Py_ssize_t i = 0; i < n; ++i) {
        PyObject* o = wrap(t[i]);
        if (o == nullptr) {
            Py_DECREF(made);
            return nullptr;
        }
        PyTuple_SET_ITEM(made, i, o);
    }
    return made;
}

// f(), or None where it throws (out of memory: the general way reports it).
template <typename F>
PyObject* guarded(F f) {
    try {
        return f();
    } catch (...) {
        PyErr_Clear();
        Py_RETURN_NONE;
    }
}

// (gemm_w4, norm_residual, norm_residual_backward: addresses; NormGrads)
PyObject* bind(PyObject*, PyObject* const* a, Py_ssize_t n) {
    if (n != 4 || !PyType_Check(a[3]) || !PyType_IsSubtype(reinterpret_cast<PyTypeObject*>(a[3]), &PyTuple_Type)) {
        PyErr_SetString(PyExc_TypeError, "bind needs three addresses and a named tuple");
        return nullptr;
    }
    g_w4 = reinterpret_cast<decltype(g_w4)>(PyLong_AsVoidPtr(a[0]));
    g_norm = reinterpret_cast<decltype(g_norm)>(PyLong_AsVoidPtr(a[1]));
    g_norm_backward = reinterpret_cast<decltype(g_norm_backward)>(PyLong_AsVoidPtr(a[2]));
    if (PyErr_Occurred()) return nullptr;
    Py_INCREF(a[3]);
    g_grads = reinterpret_cast<PyTypeObject*>(a[3]);
    Py_RETURN_NONE;
}

// (a, bq, bscale, N, group, relu, bzero, bias, residual, out_dtype)
PyObject* gemm_w4(PyObject*, PyObject* const* a, Py_ssize_t count) {
    return guarded([&]() -> PyObject* {
        int64_t N, group;
        const at::Tensor* x = count == 10 && g_w4 != nullptr ? plain(a[0]) : nullptr;
        if (x == nullptr || !integer(a[3], &N) || !integer(a[4], &group) ||
            (group != 32 && group != 64 && group != 128) || N < 0 || !PyBool_Check(a[5]))
            Py_RETURN_NONE;
        const at::ScalarType type = x->scalar_type();
        const int index = x->get_device();
        int32_t code, out_code;
        at::ScalarType out_type = type;
        if (a[9] != Py_None) {
            if (!THPDtype_Check(a[9])) Py_RETURN_NONE;
            out_type = reinterpret_cast<THPDtype*>(a[9])->scalar_type;
        }
        Matrix A, bq, scale, zero, residual;
        if (!code_of(type, &code) || type == at::kFloat || !code_of(out_type, &out_code) ||
            (out_type != type && out_type != at::kFloat) || !here(index) ||
            !matrix(a[0], type, -1, -1, index, &A))
            Py_RETURN_NONE;
        const int64_t groups = (A.cols + group - 1) / group;
        tg_epilogue_ex_t epi;
        std::memset(&epi, 0, sizeof(epi));
        if (!matrix(a[1], at::kByte, N, -1, index, &bq) || bq.cols < (A.cols + 1) / 2 ||
            !matrix(a[2], type, groups, -1, index, &scale) || scale.cols < N ||
            (a[6] != Py_None && (!matrix(a[6], at::kByte, groups, -1, index, &zero) || zero.cols < N)) ||
            !vector(a[7], N, index, &epi.bias) ||
            (a[8] != Py_None && !matrix(a[8], type, A.rows, N, index, &residual)))
            Py_RETURN_NONE;
        epi.activation = a[5] == Py_True ? TG_EPI_RELU : TG_EPI_NONE;
        epi.out_dtype = out_code;
        epi.residual = residual.p;
        epi.ldr = residual.ld;
        const at::Tensor c = empty({A.rows, N}, out_type, index);
        const tg_status_t st =
            g_w4(code, A.p, bq.p, scale.p, zero.p, c.data_ptr(), A.rows, N, A.cols, static_cast<int32_t>(group),
                 A.ld, bq.ld, scale.ld, zero.ld, N, &epi, stream_of(index));
        return st == TG_OK ? wrap(c) : PyLong_FromLong(st);
    });
}

// (x, residual, post_weight, gate, scale, pre_weight, eps) to the C structure.
bool norm_args(PyObject* const* a, tg_norm_t* n, at::ScalarType* type, at::ScalarType* kind, int* index) {
    const at::Tensor* x = plain(a[0]);
    if (x == nullptr) return false;
    *type = *kind = x->scalar_type();
    *index = x->get_device();
    std::memset(n, 0, sizeof(*n));
    Matrix m, r, g;
    if (!code_of(*type, &n->dtype) || !here(*index) || !matrix(a[0], *type, -1, -1, *index, &m) ||
        m.cols > 32768 || !number(a[4], &n->scale) || !number(a[6], &n->eps) || !(n->eps >= 0.0f))
        return false;
    n->stream_dtype = n->dtype;
    if (a[1] != Py_None) {
        const at::Tensor* t = plain(a[1]);
        if (t == nullptr) return false;
        *kind = t->scalar_type();
        if (*kind != *type && *kind != at::kFloat) return false;
        if (!code_of(*kind, &n->stream_dtype) || !matrix(a[1], *kind, m.rows, m.cols, *index, &r)) return false;
    }
    if (a[3] != Py_None) {
        const at::Tensor* t = plain(a[3]);
        if (t == nullptr) return false;
        if (t->dim() == 1) {
            if (t->scalar_type() != *type || t->size(0) != m.cols || t->get_device() != *index ||
                (m.cols > 1 && t->stride(0) != 1))
                return false;
            g.p = t->data_ptr();
            g.rows = 1;
            g.ld = (m.cols + 15) / 16 * 16;
        } else if (!matrix(a[3], *type, -1, m.cols, *index, &g)) {
            return false;
        }
        if (g.rows < 1 || (m.rows > 0 && (g.rows > m.rows || m.rows % g.rows != 0))) return false;
    }
    n->rows = m.rows;
    n->cols = m.cols;
    n->x = m.p;
    n->ldx = m.ld;
    n->residual = r.p;
    n->ldr = r.ld;
    n->gate = g.p;
    n->ldg = g.ld;
    n->gate_rows = g.rows;
    return vector(a[2], m.cols, *index, &n->post_weight) && vector(a[5], m.cols, *index, &n->pre_weight);
}

// (x, residual, post_weight, gate, scale, pre_weight, eps)
PyObject* norm_residual(PyObject*, PyObject* const* a, Py_ssize_t count) {
    return guarded([&]() -> PyObject* {
        tg_norm_t n;
        at::ScalarType type, kind;
        int index;
        if (count != 7 || g_norm == nullptr || !norm_args(a, &n, &type, &kind, &index)) Py_RETURN_NONE;
        at::Tensor made[2];
        made[0] = empty({n.rows, n.cols}, kind, index);
        if (a[5] != Py_None) made[1] = empty({n.rows, n.cols}, type, index);
        const tg_status_t st = g_norm(&n, made[0].data_ptr(), n.cols,
                                      made[1].defined() ? made[1].data_ptr() : nullptr, n.cols, stream_of(index));
        return st == TG_OK ? tuple_of(made, 2) : PyLong_FromLong(st);
    });
}

// (dy, dh, x, residual, post_weight, gate, scale, pre_weight, eps)
PyObject* norm_residual_backward(PyObject*, PyObject* const* a, Py_ssize_t count) {
    return guarded([&]() -> PyObject* {
        tg_norm_t n;
        tg_norm_grad_t g;
        at::ScalarType type, kind;
        int index;
        if (count != 9 || g_norm_backward == nullptr || !norm_args(a + 2, &n, &type, &kind, &index))
            Py_RETURN_NONE;
        std::memset(&g, 0, sizeof(g));
        Matrix dy, dh;
        if ((a[0] != Py_None && !matrix(a[0], kind, n.rows, n.cols, index, &dy)) ||
            (a[1] != Py_None && (a[7] == Py_None || !matrix(a[1], type, n.rows, n.cols, index, &dh))))
            Py_RETURN_NONE;
        g.dy = dy.p;
        g.lddy = dy.ld;
        g.dh = dh.p;
        g.lddh = dh.ld;
        at::Tensor made[5];
        made[0] = empty({n.rows, n.cols}, type, index);
        g.dx = made[0].data_ptr();
        if (a[3] != Py_None) {
            made[1] = empty({n.rows, n.cols}, kind, index);
            g.dresidual = made[1].data_ptr();
        }
        if (a[5] != Py_None) {
            made[2] = empty(THPVariable_Unpack(a[5]).sizes(), type, index);
            g.dgate = made[2].data_ptr();
        }
        if (a[4] != Py_None) {
            made[3] = empty({n.cols}, at::kFloat, index);
            g.dpost_weight = static_cast<float*>(made[3].data_ptr());
        }
        if (a[7] != Py_None) {
            made[4] = empty({n.cols}, at::kFloat, index);
            g.dpre_weight = static_cast<float*>(made[4].data_ptr());
        }
        g.lddx = g.lddr = g.lddg = n.cols;
        const tg_status_t st = g_norm_backward(&n, &g, stream_of(index));
        if (st != TG_OK) return PyLong_FromLong(st);
        PyObject* five = tuple_of(made, 5);
        if (five == nullptr) return nullptr;
        PyObject* args = PyTuple_Pack(1, five);
        Py_DECREF(five);
        if (args == nullptr) return nullptr;
        PyObject* grads = PyTuple_Type.tp_new(g_grads, args, nullptr);
        Py_DECREF(args);
        return grads;
    });
}

template <typename F>
PyCFunction fast(F f) {
    return reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(f));
}

PyMethodDef g_methods[] = {
    {"bind", fast(bind), METH_FASTCALL, nullptr},
    {"gemm_w4", fast(gemm_w4), METH_FASTCALL, nullptr},
    {"norm_residual", fast(norm_residual), METH_FASTCALL, nullptr},
    {"norm_residual_backward", fast(norm_residual_backward), METH_FASTCALL, nullptr},
    {nullptr, nullptr, 0, nullptr}};
PyModuleDef g_module = {PyModuleDef_HEAD_INIT, "_calls", nullptr, -1, g_methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__calls() {
    PyObject* m = PyModule_Create(&g_module);
    // also how build.py tells that the file is another PyTorch's
    if (m != nullptr && PyModule_AddStringConstant(m, "built_against", TG_BUILT_AGAINST) != 0) Py_CLEAR(m);
    return m;
}
