// ck_bind.cpp -- the fp4 calls from torch tensors without Python's share of the host time.
//
// Each function takes the tensors of the ck.py function of its name, in order.  Where they are what
// the call wants, it allocates its outputs and workspace (the products take given ones too), calls the
// library on torch's current stream and returns the result (or the library's status, an int, if that is
// not CK_OK).  Anything else, a wrong type or size, another current device, an allocation that fails, the
// quantizer's given codes or scales or rows of codes that are not whole 16 bytes, makes it return None with
// nothing done: ck.py then goes through its own checks, which say what is wrong or handle the case.
// A call costs about 2 us here that Python's checks and ctypes take 9 for.
#include <ATen/ATen.h>
#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAStream.h>
#include <dlfcn.h>
#include <algorithm>
#include <torch/csrc/Dtype.h>
#include <torch/csrc/autograd/python_variable.h>

#include "ck.h"

namespace {

decltype(&ck_fp4_scales_bytes) scales_bytes;
decltype(&ck_fp4_linear_workspace_bytes) workspace_bytes;
decltype(&ck_quant_fp4) quant_fp4;
decltype(&ck_dequant_fp4) dequant_fp4;
decltype(&ck_fp4_linear) fp4_linear;
decltype(&ck_fp4_expert_linear) fp4_expert_linear;

// A strided CUDA tensor whose memory holds its values (a negated view's holds their negatives).
bool in_memory(const at::Tensor& t) { return t.is_cuda() && t.layout() == at::kStrided && !t.is_neg(); }

// An argument that may be None.  `ok` turns false where it is neither None nor such a tensor on device
// `dev`.
struct Arg {
    const at::Tensor* t = nullptr;
    void* ptr() const { return t ? t->data_ptr() : nullptr; }
};
Arg optional(PyObject* o, int dev, bool& ok) {
    Arg a;
    if (o == Py_None) return a;
    if (!THPVariable_Check(o)) {
        ok = false;
        return a;
    }
    a.t = &THPVariable_Unpack(o);
    if (!in_memory(*a.t) || a.t->get_device() != dev) ok = false;
    return a;
}

// A CUDA tensor on the current device; nullptr otherwise.
const at::Tensor* on_current_device(PyObject* o, int& dev) {
    if (!THPVariable_Check(o)) return nullptr;
    const at::Tensor& t = THPVariable_Unpack(o);
    if (!in_memory(t)) return nullptr;
    dev = t.get_device();
    return dev == c10::cuda::current_device() ? &t : nullptr;
}

int float_code(at::ScalarType s) {
    return s == at::kFloat ? CK_F32 : s == at::kHalf ? CK_F16 : s == at::kBFloat16 ? CK_BF16 : -1;
}

bool format_of(PyObject* o, ck_fp4_format& f) {
    int beyond;
    const long v = PyLong_Check(o) ? PyLong_AsLongAndOverflow(o, &beyond) : -1;
    if (v != CK_MXFP4 && v != CK_NVFP4) return false;
    f = static_cast<ck_fp4_format>(v);
    return true;
}

bool bytes_of(const at::Tensor& t, size_t least) {
    return t.scalar_type() == at::kByte && t.is_contiguous() && (size_t)t.numel() >= least;
}

bool tensor_scale(const Arg& a, int64_t n, ck_fp4_format f) {
    return !a.t || (f == CK_NVFP4 && a.t->scalar_type() == at::kFloat && a.t->numel() == n && a.t->is_contiguous());
}

// Number of experts, 0 without offsets, -1 for anything else.
int64_t experts(const Arg& a) {
    if (!a.t) return 0;
    if (a.t->scalar_type() != at::kInt || a.t->dim() != 1 || !a.t->is_contiguous() || a.t->numel() < 2) return -1;
    return a.t->numel() - 1;
}

bool sizes(int64_t K, ck_fp4_format f) { return K > 0 && K % (f == CK_NVFP4 ? 16 : 32) == 0; }

PyObject* status(ck_status st) { return PyLong_FromLong(st); }

PyObject* none() { Py_RETURN_NONE; }

// (x, fmt, tensor_scale, offsets, codes, scales) -> (codes, scales)
PyObject* py_quant(PyObject*, PyObject* const* a, Py_ssize_t n) {
    if (n != 6 || !quant_fp4) return none();
    try {
        int dev;
        const at::Tensor* x = on_current_device(a[0], dev);
        ck_fp4_format f;
        if (!x || x->dim() != 2 || !format_of(a[1], f)) return none();
        bool ok = true;
        const Arg ts = optional(a[2], dev, ok), off = optional(a[3], dev, ok);
        const int64_t M = x->size(0), K = x->size(1), E = experts(off), half = K / 2;
        const int dt = float_code(x->scalar_type());
        if (!ok || dt < 0 || E < 0 || !sizes(K, f) || !tensor_scale(ts, 1, f)) return none();
        if (a[4] != Py_None || a[5] != Py_None || half % 16 != 0) return none();
        const auto bytes = x->options().dtype(at::kByte);
        at::Tensor codes = at::empty({M, half}, bytes);
        at::Tensor scales = at::empty({(int64_t)scales_bytes(M, K, f, (int)E)}, bytes);
        const ck_status st = quant_fp4(
            x->data_ptr(), (ck_dtype)dt, M, K, x->stride(0), x->stride(1), f, (const float*)ts.ptr(),
            (const int32_t*)off.ptr(), (int)E, (uint8_t*)codes.data_ptr(), half, (uint8_t*)scales.data_ptr(),
            c10::cuda::getCurrentCUDAStream(dev).stream());
        if (st != CK_OK) return status(st);
        PyObject* r = PyTuple_New(2);
        PyTuple_SET_ITEM(r, 0, THPVariable_Wrap(std::move(codes)));
        PyTuple_SET_ITEM(r, 1, THPVariable_Wrap(std::move(scales)));
        return r;
    } catch (...) {
        return none();
    }
}

// (codes, scales, fmt, tensor_scale, offsets, out_dtype) -> out
PyObject* py_dequant(PyObject*, PyObject* const* a, Py_ssize_t n) {
    if (n != 6 || !dequant_fp4) return none();
    try {
        int dev;
        const at::Tensor* c = on_current_device(a[0], dev);
        ck_fp4_format f;
        if (!c || c->dim() != 2 || !format_of(a[2], f) || !THPDtype_Check(a[5])) return none();
        bool ok = true;
        const Arg s = optional(a[1], dev, ok), ts = optional(a[3], dev, ok), off = optional(a[4], dev, ok);
        const int64_t M = c->size(0), half = c->size(1), K = 2 * half, E = experts(off);
        const at::ScalarType od = reinterpret_cast<THPDtype*>(a[5])->scalar_type;
        const int odt = float_code(od);
        if (!ok || !s.t || E < 0 || odt < 0 || !sizes(K, f) || !tensor_scale(ts, 1, f) ||
            c->scalar_type() != at::kByte || c->stride(1) != 1 || (M > 1 && c->stride(0) < half) ||
            !bytes_of(*s.t, scales_bytes(M, K, f, (int)E)))
            return none();
        at::Tensor out = at::empty({M, K}, c->options().dtype(od));
        const ck_status st = dequant_fp4(
            (const uint8_t*)c->data_ptr(), std::max(c->stride(0), half), (const uint8_t*)s.ptr(), M, K, f, (const float*)ts.ptr(),
            (const int32_t*)off.ptr(), (int)E, out.data_ptr(), (ck_dtype)odt, K,
            c10::cuda::getCurrentCUDAStream(dev).stream());
        if (st != CK_OK) return status(st);
        return THPVariable_Wrap(std::move(out));
    } catch (...) {
        return none();
    }
}

// (x, offsets, w, w_scales, fmt, bias, x_scales, x_tensor_scale, w_tensor_scale, out, out_dtype, workspace,
//  dev_status) -> out; offsets None for the plain linear
PyObject* py_product(PyObject*, PyObject* const* a, Py_ssize_t n) {
    if (n != 13 || !fp4_linear) return none();
    try {
        int dev;
        const at::Tensor* x = on_current_device(a[0], dev);
        ck_fp4_format f;
        if (!x || x->dim() != 2 || !format_of(a[4], f)) return none();
        bool ok = true;
        const Arg off = optional(a[1], dev, ok), w = optional(a[2], dev, ok), wsc = optional(a[3], dev, ok),
                  bias = optional(a[5], dev, ok), xsc = optional(a[6], dev, ok), xts = optional(a[7], dev, ok),
                  wts = optional(a[8], dev, ok), given = optional(a[9], dev, ok), work = optional(a[11], dev, ok),
                  dst = optional(a[12], dev, ok);
        const int64_t E = experts(off);
        if ((work.t && !work.t->is_contiguous()) || (dst.t && (dst.t->scalar_type() != at::kInt || dst.t->numel() < 1)))
            return none();
        if (!ok || E < 0 || !w.t || !wsc.t || w.t->dim() != (E ? 3 : 2)) return none();
        const bool codes_in = x->scalar_type() == at::kByte;
        const int dt = codes_in ? (int)CK_FP4 : float_code(x->scalar_type());
        const int64_t M = x->size(0), K = x->size(1) * (codes_in ? 2 : 1), half = K / 2;
        const int64_t d = E ? 1 : 0, N = w.t->size(d), W = E ? E : 1;
        if (dt < 0 || !sizes(K, f)) return none();
        // one row's (or channel's) pitch is never used, and need not be one that TMA could
        const int64_t pitch1 = (half + 15) / 16 * 16, w_ld = N > 1 ? w.t->stride(d) : pitch1;
        if (w.t->scalar_type() != at::kByte || w.t->size(d + 1) != half || w.t->stride(d + 1) != 1 || w_ld < half ||
            (E && w.t->size(0) != E))
            return none();
        const size_t per = scales_bytes(N, K, f, 0);
        if (!bytes_of(*wsc.t, (size_t)W * per) ||
            (E && (wsc.t->dim() != 2 || wsc.t->size(0) != E || (size_t)wsc.t->size(1) != per)))
            return none();
        if (!tensor_scale(xts, 1, f) || !tensor_scale(wts, W, f)) return none();
        int bdt = CK_F32;
        if (bias.t) {
            bdt = float_code(bias.t->scalar_type());
            if (bdt < 0 || bias.t->numel() != W * N || !bias.t->is_contiguous()) return none();
        }
        int64_t sm = x->stride(0), sk = x->stride(1);
        void* ws = nullptr;
        size_t wsb = 0;
        at::Tensor scratch;
        if (codes_in) {
            if (M == 1) sm = pitch1;
            if (sk != 1 || sm < half || !xsc.t || !bytes_of(*xsc.t, scales_bytes(M, K, f, (int)E))) return none();
        } else if (work.t) {
            wsb = work.t->nbytes();
            ws = work.t->data_ptr();
        } else if ((wsb = workspace_bytes(M, K, f, (int)E)) != 0) {
            scratch = at::empty({(int64_t)wsb}, x->options().dtype(at::kByte));
            ws = scratch.data_ptr();
        }
        at::ScalarType od = codes_in ? (bias.t ? bias.t->scalar_type() : at::kBFloat16) : x->scalar_type();
        if (a[10] != Py_None) {
            if (!THPDtype_Check(a[10])) return none();
            od = reinterpret_cast<THPDtype*>(a[10])->scalar_type;
        }
        at::Tensor out;
        if (given.t) {
            if (given.t->dim() != 2 || given.t->size(0) != M || given.t->size(1) != N || given.t->stride(1) != 1 ||
                (M > 1 && given.t->stride(0) < N))
                return none();
            out = *given.t;
            od = out.scalar_type();
        }
        const int odt = float_code(od);
        if (odt < 0) return none();
        if (!given.t) out = at::empty({M, N}, x->options().dtype(od));
        const int64_t ldo = std::max(out.stride(0), N);
        const cudaStream_t stream = c10::cuda::getCurrentCUDAStream(dev).stream();
        const auto* xs = codes_in ? (const uint8_t*)xsc.ptr() : nullptr;
        const ck_status st =
            E ? fp4_expert_linear(x->data_ptr(), (ck_dtype)dt, M, K, sm, sk, f, xs, (const float*)xts.ptr(),
                                  (const int32_t*)off.ptr(), (int)E, (const uint8_t*)w.ptr(), N, w_ld, w.t->stride(0),
                                  (const uint8_t*)wsc.ptr(), (const float*)wts.ptr(), bias.ptr(),
                                  (ck_dtype)bdt, out.data_ptr(), (ck_dtype)odt, ldo, ws, wsb,
                                  (int*)dst.ptr(), stream)
              : fp4_linear(x->data_ptr(), (ck_dtype)dt, M, K, sm, sk, f, xs, (const float*)xts.ptr(),
                           (const uint8_t*)w.ptr(), N, w_ld, (const uint8_t*)wsc.ptr(),
                           (const float*)wts.ptr(), bias.ptr(), (ck_dtype)bdt, out.data_ptr(), (ck_dtype)odt,
                           ldo, ws, wsb, (int*)dst.ptr(), stream);
        if (st != CK_OK) return status(st);
        return THPVariable_Wrap(std::move(out));
    } catch (...) {
        return none();
    }
}

// load(path): the library whose functions are called (the one that ck.py loaded).
PyObject* py_load(PyObject*, PyObject* arg) {
    const char* path = PyUnicode_AsUTF8(arg);
    if (!path) return nullptr;
    void* h = dlopen(path, RTLD_NOW | RTLD_LOCAL);
    if (!h) {
        PyErr_SetString(PyExc_ImportError, dlerror());
        return nullptr;
    }
    auto get = [h](auto& fn, const char* name) { fn = reinterpret_cast<std::decay_t<decltype(fn)>>(dlsym(h, name)); };
    get(scales_bytes, "ck_fp4_scales_bytes");
    get(workspace_bytes, "ck_fp4_linear_workspace_bytes");
    get(quant_fp4, "ck_quant_fp4");
    get(dequant_fp4, "ck_dequant_fp4");
    get(fp4_linear, "ck_fp4_linear");
    get(fp4_expert_linear, "ck_fp4_expert_linear");
    if (!scales_bytes || !workspace_bytes || !quant_fp4 || !dequant_fp4 || !fp4_linear || !fp4_expert_linear) {
        PyErr_SetString(PyExc_ImportError, "the library lacks an fp4 entry point");
        return nullptr;
    }
    Py_RETURN_NONE;
}

PyMethodDef methods[] = {
    {"load", py_load, METH_O, nullptr},
    {"quant", (PyCFunction)(void (*)())py_quant, METH_FASTCALL, nullptr},
    {"dequant", (PyCFunction)(void (*)())py_dequant, METH_FASTCALL, nullptr},
    {"product", (PyCFunction)(void (*)())py_product, METH_FASTCALL, nullptr},
    {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_ck_bind", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

// torch_version: what it was built against; ck.py uses it with no other.
PyMODINIT_FUNC PyInit__ck_bind() {
    PyObject* m = PyModule_Create(&module);
    if (m && PyModule_AddStringConstant(m, "torch_version", CK_TORCH_VERSION) != 0) {
        Py_DECREF(m);
        return nullptr;
    }
    return m;
}
