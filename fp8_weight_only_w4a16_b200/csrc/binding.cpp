// binding.cpp -- the Python side of the calls for any number of tokens and of the
// draft verification: checks of the tensors, outputs, the device and its current
// stream, and one call of the C ABI.  A small call's GPU work is a few
// microseconds, as much as the same steps take in interpreted code, so they are
// made here.  The functions of libskinny are given by address (bind), so the
// module uses the very library that the package has loaded.
#define PY_SSIZE_T_CLEAN
#include <Python.h>

#include <ATen/ATen.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/DynamicTypes.h>
#include <torch/csrc/Dtype.h>
#include <torch/csrc/autograd/python_variable.h>

#include <stdexcept>
#include <string>

#include "../../include/skinny.h"

namespace {

decltype(&skinny_gemm_experts) f_gemm_experts;
decltype(&skinny_gemm_experts_silu_mul) f_gemm_experts_silu_mul;
decltype(&skinny_quantize_int8) f_quantize_int8;
decltype(&skinny_int8_gemm) f_int8_gemm;
decltype(&skinny_verify_draft) f_verify_draft;
decltype(&skinny_experts_packed_bytes) f_experts_packed_bytes;
PyObject* g_error;      // SkinnyError(status, what)

struct Refused : std::runtime_error {      // becomes a ValueError
    using std::runtime_error::runtime_error;
};

std::string shape_text(c10::IntArrayRef s)
{
    std::string t = "[";
    for (size_t i = 0; i < s.size(); ++i) t += (i ? ", " : "") + std::to_string(s[i]);
    return t + "]";
}

const at::Tensor& tensor(PyObject* o, const char* what)
{
    if (!THPVariable_Check(o)) throw Refused(std::string(what) + " must be a tensor");
    return THPVariable_Unpack(o);
}

void check(const at::Tensor& t, at::ScalarType type, c10::IntArrayRef shape, const char* what)
{
    if (t.scalar_type() != type || t.sizes() != shape || !t.is_contiguous())
        throw Refused(std::string(what) + " must be a contiguous " + c10::toString(type) + " " + shape_text(shape) +
                      " tensor");
}

// The same for a buffer of any shape.
void check_count(const at::Tensor& t, at::ScalarType type, int64_t count, const char* what)
{
    if (t.scalar_type() != type || t.numel() != count || !t.is_contiguous())
        throw Refused(std::string(what) + " must be a contiguous " + c10::toString(type) + " tensor of " +
                      std::to_string(count) + " elements");
}

// The device of a call: that of its first tensor; every other one has to be on it.
struct Device {
    c10::Device d;
    explicit Device(const at::Tensor& t) : d(t.device())
    {
        if (!d.is_cuda()) throw Refused("tensors on a CUDA device expected, got " + d.str());
    }
    void also(const at::Tensor& t) const
    {
        if (t.device() != d) throw Refused("tensors on one device expected: " + d.str() + " and " + t.device().str());
    }
};

// The call's device and stream (None: the device's current one), current while
// this lives.  Outputs are allocated under it: the allocator gives memory to a
// stream, and a block of another one's may still be read or written by what is
// pending there.
struct Current {
    c10::cuda::OptionalCUDAGuard device;
    c10::cuda::OptionalCUDAStreamGuard stream;      // (sets the device, too)
    void* handle;
    Current(PyObject* given, const Device& on)
    {
        if (given == Py_None) {
            device.set_device(on.d);
            handle = c10::cuda::getCurrentCUDAStream(on.d.index()).stream();
            return;
        }
        PyObject* v = PyObject_GetAttrString(given, "cuda_stream");
        if (!v) throw Refused("stream must be a torch.cuda.Stream");
        handle = PyLong_AsVoidPtr(v);
        Py_DECREF(v);
        if (PyErr_Occurred()) throw Refused("stream must be a torch.cuda.Stream");
        stream.reset_stream(c10::cuda::getStreamFromExternal(static_cast<cudaStream_t>(handle), on.d.index()));
    }
};

struct Workspace {
    void* ptr = nullptr;
    size_t bytes = 0;
    Workspace(PyObject* o, const Device& on)
    {
        if (o == Py_None) return;
        const at::Tensor& t = tensor(o, "workspace");
        on.also(t);
        // (its bytes are counted from the first one on)
        if (!t.is_contiguous()) throw Refused("workspace must be contiguous");
        ptr = t.data_ptr();
        bytes = t.nbytes();
    }
};

// y as given, or a new [rows, cols] tensor of out_dtype (None: float16).
at::Tensor output(PyObject* given, PyObject* out_dtype, const Device& on, int64_t rows, int64_t cols, int* code)
{
    at::Tensor y;
    if (given == Py_None) {
        at::ScalarType type = at::kHalf;
        if (out_dtype != Py_None) {
            if (!THPDtype_Check(out_dtype)) throw Refused("out_dtype must be a torch.dtype");
            type = reinterpret_cast<THPDtype*>(out_dtype)->scalar_type;
        }
        if (type == at::kHalf || type == at::kFloat)
            y = at::empty({rows, cols}, at::TensorOptions().dtype(type).device(on.d));
    } else {
        y = tensor(given, "y");
        on.also(y);
    }
    if (!y.defined() || y.dim() != 2 || y.size(0) != rows || y.size(1) != cols || !y.is_contiguous() ||
        (y.scalar_type() != at::kHalf && y.scalar_type() != at::kFloat))
        throw Refused("y must be a contiguous float16/float32 [" + std::to_string(rows) + ", " + std::to_string(cols) +
                      "] tensor");
    *code = y.scalar_type() == at::kFloat ? SKINNY_OUT_F32 : SKINNY_OUT_F16;
    return y;
}

struct Failed {      // becomes a SkinnyError
    int status;
    const char* what;
};

void status(int s, const char* what)
{
    if (s != SKINNY_OK) throw Failed{s, what};
}

template <typename F>
PyObject* guarded(Py_ssize_t have, Py_ssize_t want, F body)
{
    if (have != want) {
        PyErr_Format(PyExc_TypeError, "%zd arguments expected, got %zd", want, have);
        return nullptr;
    }
    try {
        return body();
    } catch (const Refused& e) {
        PyErr_Clear();
        PyErr_SetString(PyExc_ValueError, e.what());
    } catch (const Failed& e) {
        PyObject* x = PyObject_CallFunction(g_error, "is", e.status, e.what);
        if (x) {
            PyErr_SetObject(g_error, x);
            Py_DECREF(x);
        }
    } catch (const std::exception& e) {
        PyErr_SetString(PyExc_RuntimeError, e.what());
    }
    return nullptr;
}

PyObject* pair(const at::Tensor& a, const at::Tensor& b)
{
    return Py_BuildValue("(NN)", THPVariable_Wrap(a), THPVariable_Wrap(b));
}

// (silu, y, x, fmt, E, N, K, data, scale, offsets, out_dtype, workspace, stream) -> y
PyObject* gemm_experts(PyObject*, PyObject* const* a, Py_ssize_t n)
{
    return guarded(n, 13, [&] {
        const bool silu = a[0] == Py_True;
        const at::Tensor& x = tensor(a[2], "x");
        const long fmt = PyLong_AsLong(a[3]);
        const int64_t E = PyLong_AsLongLong(a[4]), N = PyLong_AsLongLong(a[5]), K = PyLong_AsLongLong(a[6]);
        const at::Tensor &data = tensor(a[7], "data"), &scale = tensor(a[8], "scale"), &off = tensor(a[9], "offsets");
        if (x.scalar_type() != at::kHalf || x.dim() != 2 || x.size(1) != K || !x.is_contiguous())
            throw Refused("x must be a contiguous float16 [T, " + std::to_string(K) + "] tensor");
        check(off, at::kInt, {E + 1}, "offsets");
        // the kernel reads the packed experts and their scales by E, N and K
        const size_t packed = f_experts_packed_bytes((int)fmt, E, N, K, silu);
        if (packed == 0) throw Failed{SKINNY_ERR_INVALID_ARG, "packed experts' shape"};
        check_count(data, at::kByte, (int64_t)packed, "data");
        check_count(scale, at::kFloat, fmt == SKINNY_FMT_NVFP4 ? E : E * N, "scale");
        const int64_t T = x.size(0), outputs = silu ? N / 2 : N;
        const Device on(x);
        for (const at::Tensor* t : {&data, &scale, &off}) on.also(*t);
        const Workspace ws(a[11], on);
        const Current now(a[12], on);
        int code;
        const at::Tensor y = output(a[1], a[10], on, T, outputs, &code);
        status((silu ? f_gemm_experts_silu_mul : f_gemm_experts)(
                   (int)fmt, x.data_ptr(), T, K, static_cast<const int32_t*>(off.data_ptr()), E, data.data_ptr(),
                   static_cast<const float*>(scale.data_ptr()), outputs, y.data_ptr(), code, ws.ptr, ws.bytes,
                   now.handle),
               silu ? "skinny_gemm_experts_silu_mul" : "skinny_gemm_experts");
        return THPVariable_Wrap(y);
    });
}

// (q, row_scale, x, stream) -> (q, row_scale)
PyObject* quantize_int8(PyObject*, PyObject* const* a, Py_ssize_t n)
{
    return guarded(n, 4, [&] {
        const at::Tensor& x = tensor(a[2], "x");
        if ((x.scalar_type() != at::kHalf && x.scalar_type() != at::kFloat) || x.dim() != 2 || !x.is_contiguous())
            throw Refused("x must be a contiguous float16/float32 [M, K] tensor");
        const int64_t M = x.size(0), K = x.size(1);
        at::Tensor q, s;
        if (a[0] != Py_None) {
            q = tensor(a[0], "q");
            s = tensor(a[1], "row_scale");
            check(q, at::kChar, {M, K}, "q");
            check(s, at::kFloat, {M}, "row_scale");
        }
        const Device on(x);
        const Current now(a[3], on);
        if (q.defined()) {
            on.also(q);
            on.also(s);
        } else {
            q = at::empty({M, K}, at::TensorOptions().dtype(at::kChar).device(on.d));
            s = at::empty({M}, at::TensorOptions().dtype(at::kFloat).device(on.d));
        }
        status(f_quantize_int8(x.data_ptr(), x.scalar_type() == at::kFloat ? SKINNY_OUT_F32 : SKINNY_OUT_F16, M, K,
                               q.data_ptr(), static_cast<float*>(s.data_ptr()), now.handle),
               "skinny_quantize_int8");
        return pair(q, s);
    });
}

// (y, q, row_scale, codes, channel_scale, out_dtype, workspace, stream) -> y
PyObject* gemm_int8(PyObject*, PyObject* const* a, Py_ssize_t n)
{
    return guarded(n, 8, [&] {
        const at::Tensor &q = tensor(a[1], "q"), &rs = tensor(a[2], "row_scale"), &c = tensor(a[3], "codes"),
                         &cs = tensor(a[4], "channel_scale");
        if (c.dim() != 2) throw Refused("codes must be a contiguous int8 [N, K] tensor");
        const int64_t N = c.size(0), K = c.size(1);
        check(c, at::kChar, {N, K}, "codes");
        check(cs, at::kFloat, {N}, "channel_scale");
        if (q.scalar_type() != at::kChar || q.dim() != 2 || q.size(1) != K || !q.is_contiguous())
            throw Refused("q must be a contiguous int8 [M, " + std::to_string(K) + "] tensor");
        const int64_t M = q.size(0);
        check(rs, at::kFloat, {M}, "row_scale");
        const Device on(q);
        for (const at::Tensor* t : {&rs, &c, &cs}) on.also(*t);
        const Workspace ws(a[6], on);
        const Current now(a[7], on);
        int code;
        const at::Tensor y = output(a[0], a[5], on, M, N, &code);
        status(f_int8_gemm(q.data_ptr(), static_cast<const float*>(rs.data_ptr()), M, K, c.data_ptr(),
                           static_cast<const float*>(cs.data_ptr()), N, y.data_ptr(), code, ws.ptr, ws.bytes,
                           now.handle),
               "skinny_int8_gemm");
        return THPVariable_Wrap(y);
    });
}

// (tokens, accepted, target, draft, draft_tokens, uniform, num_drafts, stream) -> (tokens, accepted)
PyObject* verify_draft(PyObject*, PyObject* const* a, Py_ssize_t n)
{
    return guarded(n, 8, [&] {
        const at::Tensor &p = tensor(a[2], "target"), &d = tensor(a[4], "draft_tokens"), &u = tensor(a[5], "uniform");
        const at::ScalarType type = p.scalar_type();
        const int kind = type == at::kFloat ? SKINNY_PROB_F32 : type == at::kHalf ? SKINNY_PROB_F16
                         : type == at::kBFloat16 ? SKINNY_PROB_BF16 : -1;
        if (kind < 0 || p.dim() != 3 || p.size(1) < 1 || p.size(2) < 1)
            throw Refused("target must be a float32/float16/bfloat16 [B, S+1, V] tensor");
        const int64_t B = p.size(0), S = p.size(1) - 1, V = p.size(2);
        if (V > 1 && p.stride(2) != 1) throw Refused("target must have unit stride along V");
        check(d, at::kInt, {B, S}, "draft_tokens");
        check(u, at::kFloat, {B, S + 1}, "uniform");
        const bool has_draft = a[3] != Py_None, has_count = a[6] != Py_None;
        at::Tensor q, count, tokens, accepted;
        if (has_draft) {
            q = tensor(a[3], "draft");
            if (q.scalar_type() != type || q.sizes() != c10::IntArrayRef({B, S, V}))
                throw Refused("draft must be a " + shape_text({B, S, V}) + " tensor of target's dtype");
            if (V > 1 && q.stride(2) != 1) throw Refused("draft must have unit stride along V");
        }
        if (has_count) {
            count = tensor(a[6], "num_drafts");
            check(count, at::kInt, {B}, "num_drafts");
        }
        if (a[0] != Py_None) {
            tokens = tensor(a[0], "tokens");
            accepted = tensor(a[1], "accepted");
            check(tokens, at::kInt, {B, S + 1}, "tokens");
            check(accepted, at::kInt, {B}, "accepted");
        }
        const Device on(p);
        for (const at::Tensor* t : std::initializer_list<const at::Tensor*>{&d, &u, &q, &count, &tokens, &accepted})
            if (t->defined()) on.also(*t);
        const Current now(a[7], on);
        if (!tokens.defined()) {
            const auto ints = at::TensorOptions().dtype(at::kInt).device(on.d);
            tokens = at::empty({B, S + 1}, ints);
            accepted = at::empty({B}, ints);
        }
        const bool drawn = has_draft && S > 0;
        status(f_verify_draft(p.data_ptr(), p.stride(0), p.stride(1), drawn ? q.data_ptr() : nullptr,
                              drawn ? q.stride(0) : 0, drawn ? q.stride(1) : 0, kind,
                              S > 0 ? static_cast<const int32_t*>(d.data_ptr()) : nullptr,
                              static_cast<const float*>(u.data_ptr()),
                              has_count ? static_cast<const int32_t*>(count.data_ptr()) : nullptr, B, S, V,
                              static_cast<int32_t*>(tokens.data_ptr()), static_cast<int32_t*>(accepted.data_ptr()),
                              now.handle),
               "skinny_verify_draft");
        return pair(tokens, accepted);
    });
}

// (SkinnyError, addresses of the functions: those above, then skinny_experts_packed_bytes)
PyObject* bind(PyObject*, PyObject* const* a, Py_ssize_t n)
{
    return guarded(n, 7, [&] {
        void* f[6];
        for (int i = 0; i < 6; ++i) f[i] = PyLong_AsVoidPtr(a[i + 1]);
        f_gemm_experts = reinterpret_cast<decltype(f_gemm_experts)>(f[0]);
        f_gemm_experts_silu_mul = reinterpret_cast<decltype(f_gemm_experts_silu_mul)>(f[1]);
        f_quantize_int8 = reinterpret_cast<decltype(f_quantize_int8)>(f[2]);
        f_int8_gemm = reinterpret_cast<decltype(f_int8_gemm)>(f[3]);
        f_verify_draft = reinterpret_cast<decltype(f_verify_draft)>(f[4]);
        f_experts_packed_bytes = reinterpret_cast<decltype(f_experts_packed_bytes)>(f[5]);
        Py_INCREF(a[0]);
        Py_XDECREF(g_error);
        g_error = a[0];
        Py_RETURN_NONE;
    });
}

#define METHOD(name) {#name, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(name)), METH_FASTCALL, nullptr}
PyMethodDef g_methods[] = {METHOD(bind), METHOD(gemm_experts), METHOD(quantize_int8), METHOD(gemm_int8),
                           METHOD(verify_draft), {nullptr, nullptr, 0, nullptr}};
PyModuleDef g_module = {PyModuleDef_HEAD_INIT, "_binding", nullptr, -1, g_methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__binding() { return PyModule_Create(&g_module); }
