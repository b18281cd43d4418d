// torch_binding.cpp -- the operators around the experts as Python calls on
// torch tensors: argument checks, output tensors, the current stream, and one
// call into the library.  Small calls are bound by the host: the same steps in
// Python took 20 us for a norm of four rows and 13 us for a combine's gradient,
// of which the kernels need 2 and 4.
//
// A function returns its outputs, or the library's status code (an int) for
// the caller to raise; a tensor of the wrong type or shape is a ValueError
// raised here.
#include <Python.h>

#include <ATen/ATen.h>
#include <ATen/cuda/EmptyTensor.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include <initializer_list>
#include <sstream>
#include <string>

#include "moe_dispatch.h"

namespace {

using at::ScalarType;
using at::Tensor;
using Sizes = std::initializer_list<int64_t>;

constexpr ScalarType kBf16 = at::kBFloat16, kF32 = at::kFloat, kE4m3 = at::kFloat8_e4m3fn, kI32 = at::kInt;

const char* name_of(ScalarType t) {
    switch (t) {
        case at::kBFloat16: return "torch.bfloat16";
        case at::kHalf: return "torch.float16";
        case at::kFloat: return "torch.float32";
        case at::kDouble: return "torch.float64";
        case at::kFloat8_e4m3fn: return "torch.float8_e4m3fn";
        case at::kInt: return "torch.int32";
        case at::kLong: return "torch.int64";
        case at::kByte: return "torch.uint8";
        default: return at::toString(t);
    }
}

struct BadArgument {  // a Python exception is set
};

[[noreturn]] void refuse(const std::string& why) {
    PyErr_SetString(PyExc_ValueError, why.c_str());
    throw BadArgument();
}

template <typename List>
std::string text(const List& sizes) {
    std::ostringstream s;
    s << "(";
    int i = 0;
    for (const int64_t n : sizes) s << (i++ ? ", " : "") << n;
    s << (i == 1 ? ",)" : ")");
    return s.str();
}

// A tensor argument; undefined for None.
Tensor tensor(PyObject* o, const char* name) {
    if (o == Py_None) return Tensor();
    if (!THPVariable_Check(o)) {
        PyErr_Format(PyExc_TypeError, "%s must be a tensor", name);
        throw BadArgument();
    }
    return THPVariable_Unpack(o);
}

// The kernels run on the current device and reach only its memory.  A call asks
// for the device once (OnStream, which also looks at the tensors before it).
thread_local int call_device = -1;

bool fits(const Tensor& t, ScalarType type, Sizes sizes) {
    return t.defined() && t.scalar_type() == type && t.is_cuda() && (call_device < 0 || t.get_device() == call_device) &&
           t.is_contiguous() && t.sizes() == at::IntArrayRef(sizes.begin(), sizes.size());
}

void need(const Tensor& t, ScalarType type, Sizes sizes, const char* name) {
    if (fits(t, type, sizes)) return;
    std::ostringstream s;
    s << name << " must be a contiguous CUDA " << name_of(type) << " tensor of shape " << text(sizes)
      << " on the current device (got ";
    if (t.defined()) s << name_of(t.scalar_type()) << " " << text(t.sizes()) << " on " << t.device().str();
    else s << "None";
    refuse(s.str() + ")");
}

void need_float(const Tensor& t, const char* name) {  // bfloat16 or float32
    if (t.defined() && (t.scalar_type() == kBf16 || t.scalar_type() == kF32)) return;
    refuse(std::string(name) + " must be bfloat16 or float32 (got " + (t.defined() ? name_of(t.scalar_type()) : "None") +
           ")");
}

void need_dims(const Tensor& t, int64_t dims, const char* name) {
    if (!t.defined() || t.dim() != dims)
        refuse(std::string(name) + " must have " + std::to_string(dims) + " dimensions (got " +
               (t.defined() ? text(t.sizes()) : "None") + ")");
}

Tensor empty(Sizes sizes, ScalarType type, const Tensor& like) {
    return at::detail::empty_cuda(at::IntArrayRef(sizes.begin(), sizes.size()), type, like.device(), c10::nullopt);
}

// An output: the caller's tensor, checked, or a new one.
Tensor output(const Tensor& given, Sizes sizes, ScalarType type, const Tensor& like, const char* name) {
    if (!given.defined()) return empty(sizes, type, like);
    need(given, type, sizes, name);
    return given;
}

template <typename T = void>
T* ptr(const Tensor& t) {
    return t.defined() ? static_cast<T*>(t.data_ptr()) : nullptr;
}

int dtype_of(const Tensor& t) {
    return t.scalar_type() == kF32 ? MOE_DTYPE_F32 : t.scalar_type() == kE4m3 ? MOE_DTYPE_E4M3 : MOE_DTYPE_BF16;
}

// The stream that a call launches on: an integer handle, or None for the
// current one.  While it lives, the handle's stream is the current one, so that
// what the call allocates comes from the memory of the stream that uses it: a
// workspace that is released as the call returns can only go to later work of
// that stream, and no earlier work of another stream still writes to it.  Made
// once a CUDA tensor has been seen: without a GPU there is no stream to ask for.
class OnStream {
public:
    OnStream(PyObject* o, const Tensor& first, const char* name)
        : current_(c10::cuda::getCurrentCUDAStream()), handle_(current_.stream()) {
        call_device = current_.device_index();
        if (first.get_device() != call_device) {
            call_device = -1;
            refuse(std::string(name) + " must be on the current device (got " + first.device().str() + ")");
        }
        if (o == Py_None) return;
        void* p = PyLong_AsVoidPtr(o);
        if (p == nullptr && PyErr_Occurred()) {
            call_device = -1;
            throw BadArgument();
        }
        handle_ = static_cast<cudaStream_t>(p);
        if (handle_ == current_.stream()) return;
        const c10::DeviceIndex device = current_.device_index();
        guard_.reset_stream(p == nullptr ? c10::cuda::getDefaultCUDAStream(device)
                                         : c10::cuda::getStreamFromExternal(handle_, device));
        other_ = true;
    }
    ~OnStream() { call_device = -1; }
    OnStream(const OnStream&) = delete;
    cudaStream_t handle() const { return handle_; }
    // An output that the call allocated: the caller's current stream goes on to use it.
    void hand_over(const Tensor& out, PyObject* given) const {
        if (other_ && given == Py_None && out.defined()) out.record_stream(current_.unwrap());
    }

private:
    c10::cuda::CUDAStream current_;
    cudaStream_t handle_;
    c10::cuda::OptionalCUDAStreamGuard guard_;
    bool other_ = false;
};

int as_int(int64_t n, const char* name) {
    if (n > INT32_MAX) refuse(std::string(name) + " is too large");
    return static_cast<int>(n);
}

void groups_of(MoePlanOut* plan, PyObject* cu, PyObject* count, PyObject* status, int64_t E) {
    const Tensor c = tensor(cu, "cu_seqlens"), n = tensor(count, "tokens_per_expert"), s = tensor(status, "status");
    if (n.defined() && n.numel() != E)
        refuse("the plan has " + std::to_string(n.numel()) + " experts, w_gate_up " + std::to_string(E));
    need(c, kI32, {E + 1}, "cu_seqlens");
    need(n, kI32, {E}, "tokens_per_expert");
    need(s, kI32, {4}, "status");
    plan->cu_seqlens = ptr<int32_t>(c);
    plan->tokens_per_expert = ptr<int32_t>(n);
    plan->status = ptr<int32_t>(s);
}

PyObject* wrap(const Tensor& t) {
    if (t.defined()) return THPVariable_Wrap(t);
    Py_RETURN_NONE;
}

PyObject* wrap(std::initializer_list<Tensor> outs) {
    PyObject* r = PyTuple_New(static_cast<Py_ssize_t>(outs.size()));
    if (r == nullptr) return nullptr;
    Py_ssize_t i = 0;
    for (const Tensor& t : outs) PyTuple_SET_ITEM(r, i++, wrap(t));
    return r;
}

bool count_is(Py_ssize_t n, Py_ssize_t want) {
    if (n == want) return true;
    PyErr_Format(PyExc_TypeError, "%zd arguments expected (got %zd)", want, n);
    return false;
}

// residual_norm(x, weight, residual, eps, quantize, out, residual_out, q, q_scale, stream)
PyObject* residual_norm(PyObject*, PyObject* const* a, Py_ssize_t n) {
    HANDLE_TH_ERRORS
    if (!count_is(n, 10)) return nullptr;
    try {
        const Tensor x = tensor(a[0], "x"), weight = tensor(a[1], "weight"), residual = tensor(a[2], "residual");
        const double eps = PyFloat_AsDouble(a[3]);
        if (eps == -1.0 && PyErr_Occurred()) return nullptr;
        const bool quantize = a[4] == Py_True;
        Tensor residual_out = tensor(a[6], "residual_out"), q = tensor(a[7], "q"), q_scale = tensor(a[8], "q_scale");
        need_dims(x, 2, "x");
        const int64_t N = x.size(0), H = x.size(1);
        need(x, kBf16, {N, H}, "x");
        const OnStream stream(a[9], x, "x");
        need_float(weight, "weight");
        need(weight, weight.scalar_type(), {H}, "weight");
        if (residual.defined()) {
            need_float(residual, "residual");
            need(residual, residual.scalar_type(), {N, H}, "residual");
            residual_out = output(residual_out, {N, H}, residual.scalar_type(), x, "residual_out");
        } else if (residual_out.defined()) {
            refuse("residual_out needs a residual");
        }
        const Tensor y = output(tensor(a[5], "out"), {N, H}, kBf16, x, "out"), rstd = empty({N}, kF32, x);
        if (quantize) {
            q = output(q, {N, H}, kE4m3, x, "q");
            q_scale = output(q_scale, {N}, kF32, x, "q_scale");
        } else if (q.defined() || q_scale.defined()) {
            refuse("q and q_scale need quantize=True");
        }
        const int rc = moe_residual_norm(ptr<uint16_t>(x), ptr<>(residual), residual.defined() ? dtype_of(residual) : 0,
                                         ptr<>(weight), dtype_of(weight), as_int(N, "N"), as_int(H, "H"),
                                         static_cast<float>(eps), ptr<uint16_t>(y), ptr<>(residual_out), ptr<float>(rstd),
                                         ptr<uint8_t>(q), ptr<float>(q_scale), stream.handle());
        stream.hand_over(y, a[5]);
        stream.hand_over(residual_out, a[6]);
        stream.hand_over(rstd, Py_None);
        stream.hand_over(q, a[7]);
        stream.hand_over(q_scale, a[8]);
        return rc != MOE_OK ? PyLong_FromLong(rc) : wrap({y, residual_out, rstd, q, q_scale});
    } catch (const BadArgument&) {
        return nullptr;
    }
    END_HANDLE_TH_ERRORS
}

// residual_norm_backward(dy, s, weight, rstd, ds, stream)
PyObject* residual_norm_backward(PyObject*, PyObject* const* a, Py_ssize_t n) {
    HANDLE_TH_ERRORS
    if (!count_is(n, 6)) return nullptr;
    try {
        const Tensor dy = tensor(a[0], "dy"), s = tensor(a[1], "s"), weight = tensor(a[2], "weight"),
                     rstd = tensor(a[3], "rstd"), ds = tensor(a[4], "ds");
        need_dims(dy, 2, "dy");
        const int64_t N = dy.size(0), H = dy.size(1);
        need(dy, kBf16, {N, H}, "dy");
        const OnStream stream(a[5], dy, "dy");
        need_float(s, "s");
        need(s, s.scalar_type(), {N, H}, "s");
        need_float(weight, "weight");
        need(weight, weight.scalar_type(), {H}, "weight");
        need(rstd, kF32, {N}, "rstd");
        if (ds.defined()) need(ds, s.scalar_type(), {N, H}, "ds");
        const Tensor dx = empty({N, H}, kBf16, dy), dres = s.scalar_type() == kF32 ? empty({N, H}, kF32, dy) : Tensor(),
                     dweight = empty({H}, kF32, dy);
        const int64_t bytes =
            static_cast<int64_t>(moe_residual_norm_backward_workspace_size(as_int(N, "N"), as_int(H, "H")));
        const Tensor ws = empty({bytes}, at::kByte, dy);
        const int rc = moe_residual_norm_backward(ptr<uint16_t>(dy), ptr<>(s), dtype_of(s), ptr<>(weight),
                                                  dtype_of(weight), ptr<float>(rstd), ptr<>(ds), static_cast<int>(N),
                                                  static_cast<int>(H), ptr<uint16_t>(dx), ptr<float>(dres),
                                                  ptr<float>(dweight), ptr<>(ws), static_cast<size_t>(bytes),
                                                  stream.handle());
        for (const Tensor& t : {dx, dres, dweight}) stream.hand_over(t, Py_None);
        return rc != MOE_OK ? PyLong_FromLong(rc) : wrap({dx, dres, dweight});
    } catch (const BadArgument&) {
        return nullptr;
    }
    END_HANDLE_TH_ERRORS
}

// expert_ffn(x, w_gate_up, w_down, cu_seqlens, tokens_per_expert, status, x_scale, w_scale, h, preact, out, stream)
PyObject* expert_ffn(PyObject*, PyObject* const* a, Py_ssize_t n) {
    HANDLE_TH_ERRORS
    if (!count_is(n, 12)) return nullptr;
    try {
        const Tensor x = tensor(a[0], "x"), wgu = tensor(a[1], "w_gate_up"), wd = tensor(a[2], "w_down"),
                     x_scale = tensor(a[6], "x_scale"), w_scale = tensor(a[7], "w_scale"), preact = tensor(a[9], "preact");
        need_dims(x, 2, "x");
        need_dims(wgu, 4, "w_gate_up");
        const int64_t rows = x.size(0), H = x.size(1), E = wgu.size(0), I = wgu.size(2);
        const ScalarType type = x.scalar_type();
        if (type != kBf16 && type != kE4m3)
            refuse(std::string("x must be bfloat16 or float8_e4m3fn (got ") + name_of(type) + ")");
        need(x, type, {rows, H}, "x");
        const OnStream stream(a[11], x, "x");
        need(wgu, type, {E, 2, I, H}, "w_gate_up");
        need(wd, kBf16, {E, H, I}, "w_down");
        if (type == kE4m3) {
            if (!x_scale.defined() || !w_scale.defined()) refuse("8-bit rows and weights need x_scale and w_scale");
            need(x_scale, kF32, {rows}, "x_scale");
            need(w_scale, kF32, {E, 2, I}, "w_scale");
        } else if (x_scale.defined() || w_scale.defined()) {
            refuse("x_scale and w_scale go with 8-bit rows and weights");
        }
        MoePlanOut plan = {};
        groups_of(&plan, a[3], a[4], a[5], E);
        const Tensor h = output(tensor(a[8], "h"), {rows, I}, kBf16, x, "h");
        if (preact.defined()) need(preact, kF32, {rows, 2, I}, "preact");
        const Tensor y = output(tensor(a[10], "out"), {rows, H}, kBf16, x, "out");
        const int rc = moe_expert_ffn(ptr<>(x), ptr<float>(x_scale), ptr<>(wgu), ptr<float>(w_scale), ptr<uint16_t>(wd),
                                      rows, as_int(E, "E"), as_int(H, "H"), as_int(I, "I"), dtype_of(x), &plan,
                                      ptr<uint16_t>(h), ptr<float>(preact), ptr<uint16_t>(y), stream.handle());
        stream.hand_over(y, a[10]);
        return rc != MOE_OK ? PyLong_FromLong(rc) : wrap(y);
    } catch (const BadArgument&) {
        return nullptr;
    }
    END_HANDLE_TH_ERRORS
}

// expert_ffn_backward(dy, x, h, preact, w_gate_up, w_down, cu_seqlens, tokens_per_expert, status, dx, dgate_up, need_dx,
//                     need_dw, stream)
PyObject* expert_ffn_backward(PyObject*, PyObject* const* a, Py_ssize_t n) {
    HANDLE_TH_ERRORS
    if (!count_is(n, 14)) return nullptr;
    try {
        const Tensor dy = tensor(a[0], "dy"), x = tensor(a[1], "x"), h = tensor(a[2], "h"), preact = tensor(a[3], "preact"),
                     wgu = tensor(a[4], "w_gate_up"), wd = tensor(a[5], "w_down");
        Tensor dx = tensor(a[9], "dx");
        const bool need_dx = a[11] == Py_True, need_dw = a[12] == Py_True;
        need_dims(x, 2, "x");
        need_dims(wgu, 4, "w_gate_up");
        const int64_t rows = x.size(0), H = x.size(1), E = wgu.size(0), I = wgu.size(2);
        need(x, kBf16, {rows, H}, "x");
        const OnStream stream(a[13], x, "x");
        need(dy, kBf16, {rows, H}, "dy");
        need(h, kBf16, {rows, I}, "h");
        need(preact, kF32, {rows, 2, I}, "preact");
        need(wgu, kBf16, {E, 2, I, H}, "w_gate_up");
        need(wd, kBf16, {E, H, I}, "w_down");
        MoePlanOut plan = {};
        groups_of(&plan, a[6], a[7], a[8], E);
        const Tensor dgu = output(tensor(a[10], "dgate_up"), {rows, 2, I}, kBf16, x, "dgate_up");
        if (need_dx) dx = output(dx, {rows, H}, kBf16, x, "dx");
        else if (dx.defined()) refuse("dx is given but need_dx is False");
        const Tensor dwgu = need_dw ? empty({E, 2, I, H}, kBf16, x) : Tensor(),
                     dwd = need_dw ? empty({E, H, I}, kBf16, x) : Tensor();
        const int rc = moe_expert_ffn_backward(
            ptr<uint16_t>(dy), ptr<uint16_t>(x), ptr<uint16_t>(h), ptr<float>(preact), ptr<uint16_t>(wgu),
            ptr<uint16_t>(wd), rows, as_int(E, "E"), as_int(H, "H"), as_int(I, "I"), &plan, ptr<uint16_t>(dgu),
            ptr<uint16_t>(dx), ptr<uint16_t>(dwgu), ptr<uint16_t>(dwd), stream.handle());
        stream.hand_over(dx, a[9]);
        for (const Tensor& t : {dwgu, dwd}) stream.hand_over(t, Py_None);
        return rc != MOE_OK ? PyLong_FromLong(rc) : wrap({dx, dwgu, dwd});
    } catch (const BadArgument&) {
        return nullptr;
    }
    END_HANDLE_TH_ERRORS
}

// combine_backward(dout, y, topk_w, dst, zero_fill_ranges, status, dy, dw, stream)
PyObject* combine_backward(PyObject*, PyObject* const* a, Py_ssize_t n) {
    HANDLE_TH_ERRORS
    if (!count_is(n, 9)) return nullptr;
    try {
        const Tensor dout = tensor(a[0], "dout"), y = tensor(a[1], "y"), w = tensor(a[2], "topk_w"),
                     dst = tensor(a[3], "dst"), zfr = tensor(a[4], "zero_fill_ranges"), status = tensor(a[5], "status");
        need_dims(dout, 2, "dout");
        need_dims(y, 2, "y");
        need_dims(dst, 2, "dst");
        need_dims(zfr, 2, "zero_fill_ranges");
        const int64_t N = dout.size(0), H = dout.size(1), rows = y.size(0), K = dst.size(1), E = zfr.size(0);
        need(dout, kBf16, {N, H}, "dout");
        const OnStream stream(a[8], dout, "dout");
        need(y, kBf16, {rows, H}, "y");
        need(w, kF32, {N, K}, "topk_w");
        need(dst, kI32, {N, K}, "dst");
        need(zfr, kI32, {E, 2}, "zero_fill_ranges");
        need(status, kI32, {4}, "status");
        const Tensor dy = output(tensor(a[6], "dy"), {rows, H}, kBf16, y, "dy"),
                     dw = output(tensor(a[7], "dw"), {N, K}, kF32, y, "dw");
        MoePlanOut plan = {};
        plan.dst = ptr<int32_t>(dst);
        plan.zero_fill_ranges = ptr<int32_t>(zfr);
        plan.status = ptr<int32_t>(status);
        const int rc = moe_combine_backward(ptr<uint16_t>(dout), ptr<uint16_t>(y), ptr<float>(w), as_int(N, "N"),
                                            as_int(K, "K"), as_int(H, "H"), as_int(E, "E"), rows, &plan, ptr<uint16_t>(dy),
                                            ptr<float>(dw), stream.handle());
        stream.hand_over(dy, a[6]);
        stream.hand_over(dw, a[7]);
        return rc != MOE_OK ? PyLong_FromLong(rc) : wrap({dy, dw});
    } catch (const BadArgument&) {
        return nullptr;
    }
    END_HANDLE_TH_ERRORS
}

#define MOE_ENTRY(f) \
    { #f, reinterpret_cast<PyCFunction>(reinterpret_cast<void*>(f)), METH_FASTCALL, nullptr }

PyMethodDef methods[] = {MOE_ENTRY(residual_norm),       MOE_ENTRY(residual_norm_backward), MOE_ENTRY(expert_ffn),
                         MOE_ENTRY(expert_ffn_backward), MOE_ENTRY(combine_backward),       {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_torch_binding", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

extern "C" PyMODINIT_FUNC PyInit__torch_binding() { return PyModule_Create(&module); }
