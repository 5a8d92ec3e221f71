// Calls of the 8-bit layer and the block norms straight from Python objects:
// the checks that an ordinary call passes, the outputs and the scratch, and
// the C API, in one C function each.
//
// On a few tokens these calls take 2 to 10 us of device time, and the same
// steps through Python attribute tests, tensor constructors and ctypes took
// 8 to 11 us of the host's (here 3 to 4).  A function here returns the call's result; the
// library's status (an int) where the library refuses the call; or None where
// an argument is not what an ordinary call has, and then the Python binding
// makes the call with its own checks, which say what is wrong.
#include <Python.h>

#include <ATen/core/Tensor.h>
#include <ATen/cuda/EmptyTensor.h>
#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include "w4a16.h"

namespace {

struct Api {
    decltype(&w8_quantize_rows) quantize_rows;
    decltype(&w8a8_workspace_bytes) gemm_workspace;
    decltype(&w8a8_linear_workspace_bytes) linear_workspace;
    decltype(&w8a8_gemm) gemm;
    decltype(&w8a8_linear) linear;
    decltype(&w4_block_norm) norm;
    decltype(&w4_block_norm_workspace_bytes) norm_workspace;
    decltype(&w4_block_norm_backward) norm_backward;
} api;

PyTypeObject* block_norm_type = nullptr;         // named tuples of the Python module
PyTypeObject* block_norm_grad_type = nullptr;

constexpr int64_t kMost = 1ll << 30;

const at::Tensor* tensor(PyObject* o) { return THPVariable_Check(o) ? &THPVariable_Unpack(o) : nullptr; }

// A dense tensor of this type on device `dev`.
bool dense(const at::Tensor* t, at::ScalarType type, c10::DeviceIndex dev) {
    return t && t->scalar_type() == type && t->is_cuda() && t->get_device() == dev && t->is_contiguous();
}
bool vector(const at::Tensor* t, at::ScalarType type, c10::DeviceIndex dev, int64_t n) {
    return dense(t, type, dev) && t->dim() == 1 && t->size(0) == n;
}
bool matrix(const at::Tensor* t, at::ScalarType type, c10::DeviceIndex dev, int64_t rows, int64_t cols) {
    return dense(t, type, dev) && t->dim() == 2 && t->size(0) == rows && t->size(1) == cols;
}
// An optional argument: None, or a tensor that `ok` holds for.
template <class F>
bool optional(PyObject* o, const at::Tensor** t, F ok) {
    *t = nullptr;
    if (o == Py_None) return true;
    *t = tensor(o);
    return *t && ok(*t);
}
void* ptr(const at::Tensor* t) { return t ? t->data_ptr() : nullptr; }

// The device of a call: the first tensor's, if that is the current one.
bool here(const at::Tensor* t, c10::DeviceIndex* dev) {
    if (!t || !t->is_cuda()) return false;
    *dev = static_cast<c10::DeviceIndex>(t->get_device());
    return *dev == c10::cuda::current_device();
}

int64_t round16(int64_t n) { return (n + 15) / 16 * 16; }

// int8 rows: their stride if they are laid out as w8_quantize_rows lays them out, else 0.
int64_t codes_stride(const at::Tensor* t, c10::DeviceIndex dev) {
    if (!t || t->scalar_type() != at::kChar || !t->is_cuda() || t->get_device() != dev || t->dim() != 2) return 0;
    const int64_t R = t->size(0), C = t->size(1), ld = t->stride(0);
    if (R < 2 || C < 1 || R > kMost || C > kMost || t->stride(1) != 1 || ld % 16 != 0 || ld < round16(C)) return 0;
    const int64_t end = t->storage_offset() + (R - 1) * ld + round16(C);
    return static_cast<int64_t>(t->storage().nbytes()) >= end ? ld : 0;
}

at::Tensor empty_like_type(const at::Tensor& like, at::IntArrayRef sizes, at::ScalarType type) {
    // what at::empty comes to on a CUDA device, without the dispatcher
    return at::detail::empty_cuda(sizes, type, like.device(), c10::nullopt);
}
at::Tensor empty_codes(const at::Tensor& like, int64_t R, int64_t C) {
    at::Tensor q = empty_like_type(like, {R, round16(C)}, at::kChar);
    if (C != round16(C)) {
        const int64_t sizes[2] = {R, C}, strides[2] = {round16(C), 1};
        q.unsafeGetTensorImpl()->set_sizes_and_strides(at::IntArrayRef(sizes), at::IntArrayRef(strides));
    }
    return q;
}

void* stream(c10::DeviceIndex dev) { return c10::cuda::getCurrentCUDAStream(dev).stream(); }

PyObject* wrap(const at::Tensor& t) {
    if (!t.defined()) Py_RETURN_NONE;
    return THPVariable_Wrap(t);
}
// The tensors as a tuple, or as the named tuple `type`.
PyObject* tuple(std::initializer_list<at::Tensor> ts, PyTypeObject* type = &PyTuple_Type) {
    const Py_ssize_t n = static_cast<Py_ssize_t>(ts.size());
    PyObject* r = type == &PyTuple_Type ? PyTuple_New(n) : type->tp_alloc(type, n);
    if (!r) return nullptr;
    Py_ssize_t i = 0;
    for (const at::Tensor& t : ts) {
        PyObject* o = wrap(t);
        if (!o) {
            Py_DECREF(r);
            return nullptr;
        }
        PyTuple_SET_ITEM(r, i++, o);
    }
    return r;
}

// (X, channel_scales)
PyObject* quantize_rows(PyObject*, PyObject* const* args, Py_ssize_t n) {
    HANDLE_TH_ERRORS
    c10::DeviceIndex dev;
    const at::Tensor *X = n == 2 ? tensor(args[0]) : nullptr, *channel;
    if (!here(X, &dev) || !dense(X, at::kBFloat16, dev) || X->dim() != 2) Py_RETURN_NONE;
    const int64_t R = X->size(0), C = X->size(1);
    if (R < 1 || C < 1 || R > kMost || C > kMost) Py_RETURN_NONE;
    if (!optional(args[1], &channel, [&](const at::Tensor* t) { return vector(t, at::kFloat, dev, C); })) Py_RETURN_NONE;
    at::Tensor codes = empty_codes(*X, R, C), scales = empty_like_type(*X, {R}, at::kFloat);
    int st;
    Py_BEGIN_ALLOW_THREADS
    st = api.quantize_rows(X->data_ptr(), static_cast<int>(R), static_cast<int>(C), static_cast<float*>(ptr(channel)),
                           static_cast<int8_t*>(codes.data_ptr()), round16(C), static_cast<float*>(scales.data_ptr()),
                           stream(dev));
    Py_END_ALLOW_THREADS
    if (st != W4_OK) return PyLong_FromLong(st);
    return tuple({codes, scales});
    END_HANDLE_TH_ERRORS
}

// What gemm and linear share; A is int8 with a_scales and lda, or bf16 with neither.
PyObject* product(const at::Tensor* A, c10::DeviceIndex dev, const at::Tensor* a_scales, int64_t lda, PyObject* codes_o,
                  PyObject* scales_o, PyObject* bias_o, PyObject* transposed_o, PyObject* out_o) {
    const int tr = PyObject_IsTrue(transposed_o);
    if (tr < 0) return nullptr;
    const at::Tensor *W = tensor(codes_o), *scales, *bias, *given;
    const int64_t ldw = codes_stride(W, dev);
    if (!ldw) Py_RETURN_NONE;
    const int64_t N = W->size(0), K = W->size(1), M = A->size(0);
    const int64_t in = tr ? N : K, out_len = tr ? K : N;
    if (A->size(1) != in || M < 1 || M > kMost) Py_RETURN_NONE;
    if (!optional(scales_o, &scales, [&](const at::Tensor* t) { return vector(t, at::kFloat, dev, N); })) Py_RETURN_NONE;
    // linear always has the weights' scales, gemm has them unless transposed
    if ((scales != nullptr) != (a_scales == nullptr || !tr)) Py_RETURN_NONE;
    if (!optional(bias_o, &bias, [&](const at::Tensor* t) { return vector(t, at::kBFloat16, dev, out_len); }))
        Py_RETURN_NONE;
    if (!optional(out_o, &given, [&](const at::Tensor* t) { return matrix(t, at::kBFloat16, dev, M, out_len); }))
        Py_RETURN_NONE;
    const int m = static_cast<int>(M), nn = static_cast<int>(N), k = static_cast<int>(K);
    const at::Tensor out = given ? *given : empty_like_type(*A, {M, out_len}, at::kBFloat16);
    const size_t bytes = a_scales ? api.gemm_workspace(m, nn, k, tr) : api.linear_workspace(m, nn, k, tr);
    at::Tensor ws;
    if (bytes) ws = empty_like_type(*A, {static_cast<int64_t>(bytes)}, at::kByte);
    void* wsp = bytes ? ws.data_ptr() : nullptr;
    const int8_t* w = static_cast<const int8_t*>(W->data_ptr());
    const float* s = static_cast<const float*>(ptr(scales));
    void* y = out.data_ptr();
    void* st_ = stream(dev);
    int st;
    Py_BEGIN_ALLOW_THREADS
    st = a_scales ? api.gemm(static_cast<const int8_t*>(A->data_ptr()), lda, static_cast<const float*>(ptr(a_scales)), m,
                             nn, k, w, ldw, s, ptr(bias), tr, y, wsp, bytes, st_)
                  : api.linear(A->data_ptr(), m, nn, k, w, ldw, s, ptr(bias), tr, y, wsp, bytes, st_);
    Py_END_ALLOW_THREADS
    if (st != W4_OK) return PyLong_FromLong(st);
    if (given) {
        Py_INCREF(out_o);
        return out_o;
    }
    return wrap(out);
}

// (A, a_scales, codes, scales, bias, transposed, out)
PyObject* gemm(PyObject*, PyObject* const* args, Py_ssize_t n) {
    HANDLE_TH_ERRORS
    c10::DeviceIndex dev;
    const at::Tensor* A = n == 7 ? tensor(args[0]) : nullptr;
    if (!here(A, &dev)) Py_RETURN_NONE;
    int64_t lda = codes_stride(A, dev);
    if (!lda && A->dim() == 2 && A->size(0) == 1 && A->size(1) >= 1 && A->size(1) <= kMost &&
        A->scalar_type() == at::kChar && A->stride(1) == 1 &&
        static_cast<int64_t>(A->storage().nbytes()) >= A->storage_offset() + round16(A->size(1)))
        lda = round16(A->size(1));      // a single row has no stride of its own
    if (!lda) Py_RETURN_NONE;
    const at::Tensor* a_scales = tensor(args[1]);
    if (!vector(a_scales, at::kFloat, dev, A->size(0))) Py_RETURN_NONE;
    return product(A, dev, a_scales, lda, args[2], args[3], args[4], args[5], args[6]);
    END_HANDLE_TH_ERRORS
}

// (A, codes, scales, bias, transposed, out)
PyObject* linear(PyObject*, PyObject* const* args, Py_ssize_t n) {
    HANDLE_TH_ERRORS
    c10::DeviceIndex dev;
    const at::Tensor* A = n == 6 ? tensor(args[0]) : nullptr;
    if (!here(A, &dev) || !dense(A, at::kBFloat16, dev) || A->dim() != 2) Py_RETURN_NONE;
    return product(A, dev, nullptr, 0, args[1], args[2], args[3], args[4], args[5]);
    END_HANDLE_TH_ERRORS
}

struct NormInputs {
    const at::Tensor *y, *pre, *post, *gate;
    int gate_kind;
    double alpha, off;
};

// y, pre_weight, post_weight, gate, residual_scale, weight_offset
bool norm_inputs(PyObject* const* o, c10::DeviceIndex dev, int64_t M, int64_t C, NormInputs* in) {
    if (!optional(o[0], &in->y, [&](const at::Tensor* t) { return matrix(t, at::kBFloat16, dev, M, C); })) return false;
    in->pre = tensor(o[1]);
    if (!vector(in->pre, at::kBFloat16, dev, C)) return false;
    if (!optional(o[2], &in->post, [&](const at::Tensor* t) { return vector(t, at::kBFloat16, dev, C); })) return false;
    in->gate_kind = W4_GATE_NONE;
    if (!optional(o[3], &in->gate, [&](const at::Tensor* t) {
            in->gate_kind = t->dim() == 1 ? W4_GATE_CHANNEL : W4_GATE_TOKEN;
            return t->dim() == 1 ? vector(t, at::kBFloat16, dev, C) : matrix(t, at::kBFloat16, dev, M, C);
        }))
        return false;
    if (!in->y && (in->post || in->gate)) return false;
    if (!PyFloat_Check(o[4]) || !PyFloat_Check(o[5])) return false;
    in->alpha = PyFloat_AS_DOUBLE(o[4]);
    in->off = PyFloat_AS_DOUBLE(o[5]);
    return true;
}

// (x, y, pre_weight, post_weight, gate, residual_scale, weight_offset, eps, quantize, keep_rstd, residual_out)
PyObject* norm(PyObject*, PyObject* const* args, Py_ssize_t n) {
    HANDLE_TH_ERRORS
    c10::DeviceIndex dev;
    NormInputs in;
    const at::Tensor* x = n == 11 ? tensor(args[0]) : nullptr;
    if (!here(x, &dev) || !dense(x, at::kBFloat16, dev) || x->dim() != 2) Py_RETURN_NONE;
    const int64_t M = x->size(0), C = x->size(1);
    if (M < 1 || C < 1 || M > kMost || C > kMost || !norm_inputs(args + 1, dev, M, C, &in)) Py_RETURN_NONE;
    const at::Tensor* given;
    if (!optional(args[10], &given, [&](const at::Tensor* t) { return in.y && matrix(t, at::kBFloat16, dev, M, C); }) ||
        !PyFloat_Check(args[7]))
        Py_RETURN_NONE;
    const int quantize = PyObject_IsTrue(args[8]), keep = PyObject_IsTrue(args[9]);
    if (quantize < 0 || keep < 0) return nullptr;
    at::Tensor residual, normed, scales, rstd;
    if (in.y) residual = given ? *given : empty_like_type(*x, {M, C}, at::kBFloat16);
    if (quantize) {
        normed = empty_codes(*x, M, C);
        scales = empty_like_type(*x, {M}, at::kFloat);
    } else {
        normed = empty_like_type(*x, {M, C}, at::kBFloat16);
    }
    if (keep) rstd = empty_like_type(*x, {2, M}, at::kFloat);
    void* r = in.y ? residual.data_ptr() : nullptr;
    float* sc = quantize ? static_cast<float*>(scales.data_ptr()) : nullptr;
    float* rs = keep ? static_cast<float*>(rstd.data_ptr()) : nullptr;
    const float eps = static_cast<float>(PyFloat_AS_DOUBLE(args[7]));
    void* st_ = stream(dev);
    int st;
    Py_BEGIN_ALLOW_THREADS
    st = api.norm(x->data_ptr(), ptr(in.y), static_cast<int>(M), static_cast<int>(C), ptr(in.post), ptr(in.gate),
                  in.gate_kind, static_cast<float>(in.alpha), in.pre->data_ptr(), static_cast<float>(in.off), eps, r,
                  normed.data_ptr(), round16(C), sc, rs, st_);
    Py_END_ALLOW_THREADS
    if (st != W4_OK) return PyLong_FromLong(st);
    PyObject* t = tuple({residual, normed, scales, rstd}, block_norm_type);
    // what the caller gave comes back as the caller's own object
    PyObject* own = !in.y ? args[0] : given ? args[10] : nullptr;
    if (t && own) {
        Py_INCREF(own);
        Py_DECREF(PyTuple_GET_ITEM(t, 0));
        PyTuple_SET_ITEM(t, 0, own);
    }
    return t;
    END_HANDLE_TH_ERRORS
}

// (d_normed, residual, rstd, d_residual, y, pre_weight, post_weight, gate, residual_scale, weight_offset)
PyObject* norm_backward(PyObject*, PyObject* const* args, Py_ssize_t n) {
    HANDLE_TH_ERRORS
    c10::DeviceIndex dev;
    NormInputs in;
    const at::Tensor* dn = n == 10 ? tensor(args[0]) : nullptr;
    if (!here(dn, &dev) || !dense(dn, at::kBFloat16, dev) || dn->dim() != 2) Py_RETURN_NONE;
    const int64_t M = dn->size(0), C = dn->size(1);
    if (M < 1 || C < 1 || M > kMost || C > kMost || !norm_inputs(args + 4, dev, M, C, &in)) Py_RETURN_NONE;
    const at::Tensor *r = tensor(args[1]), *rstd = tensor(args[2]), *dres;
    if (!matrix(r, at::kBFloat16, dev, M, C) || !matrix(rstd, at::kFloat, dev, 2, M) ||
        !optional(args[3], &dres, [&](const at::Tensor* t) { return matrix(t, at::kBFloat16, dev, M, C); }))
        Py_RETURN_NONE;
    at::Tensor dx = empty_like_type(*dn, {M, C}, at::kBFloat16), dpre = empty_like_type(*dn, {C}, at::kBFloat16);
    at::Tensor dy, dpost, dgate;
    if (in.y) dy = empty_like_type(*dn, {M, C}, at::kBFloat16);
    if (in.post) dpost = empty_like_type(*dn, {C}, at::kBFloat16);
    if (in.gate) dgate = empty_like_type(*dn, in.gate->sizes(), at::kBFloat16);
    const size_t bytes = api.norm_workspace(static_cast<int>(M), static_cast<int>(C));
    at::Tensor ws = empty_like_type(*dn, {static_cast<int64_t>(bytes)}, at::kByte);
    void *pdy = in.y ? dy.data_ptr() : nullptr, *pdpost = in.post ? dpost.data_ptr() : nullptr;
    void* pdgate = in.gate ? dgate.data_ptr() : nullptr;
    void* st_ = stream(dev);
    int st;
    Py_BEGIN_ALLOW_THREADS
    st = api.norm_backward(dn->data_ptr(), ptr(dres), r->data_ptr(), static_cast<const float*>(rstd->data_ptr()),
                           ptr(in.y), static_cast<int>(M), static_cast<int>(C), ptr(in.post), ptr(in.gate), in.gate_kind,
                           static_cast<float>(in.alpha), in.pre->data_ptr(), static_cast<float>(in.off), dx.data_ptr(),
                           pdy, dpre.data_ptr(), pdpost, pdgate, ws.data_ptr(), bytes, st_);
    Py_END_ALLOW_THREADS
    if (st != W4_OK) return PyLong_FromLong(st);
    return tuple({dx, dy, dpre, dpost, dgate}, block_norm_grad_type);
    END_HANDLE_TH_ERRORS
}

// The library's functions by address, in the order of Api, then the named
// tuples of the norm's results and of its gradients.
PyObject* bind(PyObject*, PyObject* const* args, Py_ssize_t n) {
    constexpr Py_ssize_t kFunctions = sizeof(Api) / sizeof(void*);
    void** f = reinterpret_cast<void**>(&api);
    if (n != kFunctions + 2) {
        PyErr_SetString(PyExc_TypeError, "bind: wrong number of arguments");
        return nullptr;
    }
    for (Py_ssize_t i = 0; i < kFunctions; ++i) {
        f[i] = PyLong_AsVoidPtr(args[i]);
        if (!f[i]) {
            if (!PyErr_Occurred()) PyErr_SetString(PyExc_ValueError, "bind: null function");
            return nullptr;
        }
    }
    for (Py_ssize_t i = kFunctions; i < n; ++i) {
        if (!PyType_Check(args[i]) || !PyType_IsSubtype(reinterpret_cast<PyTypeObject*>(args[i]), &PyTuple_Type)) {
            PyErr_SetString(PyExc_TypeError, "bind: a tuple type is needed");
            return nullptr;
        }
        Py_INCREF(args[i]);
        (i == kFunctions ? block_norm_type : block_norm_grad_type) = reinterpret_cast<PyTypeObject*>(args[i]);
    }
    Py_RETURN_NONE;
}

template <PyObject* (*F)(PyObject*, PyObject* const*, Py_ssize_t)>
PyMethodDef method(const char* name) {
    return {name, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(F)), METH_FASTCALL, nullptr};
}

PyMethodDef methods[] = {method<bind>("bind"),     method<quantize_rows>("quantize_rows"),
                         method<gemm>("gemm"),     method<linear>("linear"),
                         method<norm>("norm"),     method<norm_backward>("norm_backward"),
                         {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "w8_native", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit_w8_native(void) { return PyModule_Create(&module); }
