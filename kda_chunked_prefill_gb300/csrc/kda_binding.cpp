// The plain calls of the binding as one native call each: arguments checked, outputs allocated and the C entry point called on the current
// stream without returning to Python in between. On the GB300's host, calls back to back, as Python and ctypes and as this: the gated norm of
// 7 tokens 15 and 5.5 us (its kernel takes 2), 3 x 4 steps 20 and 5.9 (5), a product of 256 rows 16 and 10 (9), 256 tokens in chunks 24 and
// 21 (20). Tensors are taken and made without torch's dispatcher; the C entry points and their checks are the same.
//
// A call returns None where it is not plain: an argument that the checks here do not accept, a device other than the current one, a tensor
// of a class of its own. The caller then takes its general path, which has the checks' messages and the other cases. An int is the C
// entry point's error code.
#include <Python.h>

#include <ATen/cuda/EmptyTensor.h>
#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/autograd/python_variable.h>

#include <cmath>
#include <cstdint>

#include "kda.h"

namespace {

using at::ScalarType;
constexpr ScalarType BF16 = ScalarType::BFloat16, F32 = ScalarType::Float, F8 = ScalarType::Float8_e4m3fn, I32 = ScalarType::Int,
                     U8 = ScalarType::Byte;

// The entry points' addresses, as the caller has loaded them.
struct {
    decltype(&kda_gated_rms_norm) norm;
    decltype(&kda_scaled_matmul) product;
    decltype(&kda_gated_delta_decode_fwd) decode;
    decltype(&kda_gated_delta_chunk_fwd) chunk;
    decltype(&kda_gated_delta_chunk_fwd_workspace_size) workspace;
} entry;

struct Not {};  // not a plain call

const at::Tensor &tensor(PyObject *o, ScalarType type) {
    if (!THPVariable_CheckExact(o)) throw Not{};
    const at::Tensor &t = THPVariable_Unpack(o);
    if (t.scalar_type() != type || !t.is_cuda()) throw Not{};
    return t;
}
void need(const at::Tensor &t, at::IntArrayRef shape, int device) {
    if (t.sizes() != shape || t.get_device() != device || !t.is_contiguous()) throw Not{};
}
// [T, heads, 128] with tokens that may be strided: their distance
int64_t heads_view(const at::Tensor &t, int64_t tokens, int device) {
    if (t.dim() != 3 || t.size(0) != tokens || t.get_device() != device) throw Not{};
    const int64_t width = t.size(1) * t.size(2);
    if (tokens == 0 || t.is_contiguous()) return width;
    if (t.stride(2) != 1 || (t.stride(1) != t.size(2) && t.size(1) > 1)) throw Not{};
    if (tokens == 1) return width;
    if (t.stride(0) < width || t.stride(0) % 8) throw Not{};
    return t.stride(0);
}
int current(const at::Tensor &t) {
    const int device = t.get_device();
    if (device != c10::cuda::current_device()) throw Not{};
    return device;
}
at::Tensor empty(at::IntArrayRef shape, ScalarType type, int device) {
    return at::Tensor(at::detail::empty_cuda(shape, type, at::Device(at::kCUDA, static_cast<c10::DeviceIndex>(device)), std::nullopt));
}
double number(PyObject *o) {
    const double x = PyFloat_AsDouble(o);
    if (x == -1.0 && PyErr_Occurred()) {
        PyErr_Clear();
        throw Not{};
    }
    return x;
}
int64_t integer(PyObject *o) {
    const long long x = PyLong_AsLongLong(o);
    if (x == -1 && PyErr_Occurred()) {
        PyErr_Clear();
        throw Not{};
    }
    return x;
}
const void *at_of(const at::Tensor &t) { return t.const_data_ptr(); }
template <typename F>
int without_gil(F &&f) {
    int rc;
    Py_BEGIN_ALLOW_THREADS;
    rc = f();
    Py_END_ALLOW_THREADS;
    return rc;
}
PyObject *pair(const at::Tensor &a, const at::Tensor &b) {
    PyObject *x = THPVariable_Wrap(a), *y = b.defined() ? THPVariable_Wrap(b) : Py_NewRef(Py_None);
    PyObject *r = x && y ? PyTuple_Pack(2, x, y) : nullptr;
    Py_XDECREF(x);
    Py_XDECREF(y);
    return r;
}
// f(args) with what it throws in Python's terms
template <typename F>
PyObject *guarded(Py_ssize_t n, Py_ssize_t count, F &&f) {
    if (n != count) {
        PyErr_SetString(PyExc_TypeError, "wrong number of arguments");
        return nullptr;
    }
    try {
        return f();
    } catch (const Not &) {
        Py_RETURN_NONE;
    } catch (...) {  // (no memory: the general path says so)
        Py_RETURN_NONE;
    }
}

PyObject *gated_rms_norm(PyObject *, PyObject *const *a, Py_ssize_t n) {  // x, gate, weight, eps, silu
    return guarded(n, 5, [&]() -> PyObject * {
        if (!THPVariable_CheckExact(a[0])) throw Not{};
        const ScalarType kind = THPVariable_Unpack(a[0]).scalar_type();
        if (kind != BF16 && kind != F32) throw Not{};
        const at::Tensor &x = tensor(a[0], kind), &gate = tensor(a[1], BF16), &weight = tensor(a[2], F32);
        const int device = current(x);
        if (x.dim() != 3 || !x.is_contiguous()) throw Not{};
        const int64_t T = x.size(0), H = x.size(1), D = x.size(2), stride = heads_view(gate, T, device);
        if (gate.sizes() != x.sizes() || H > INT32_MAX || D > INT32_MAX) throw Not{};
        need(weight, {D}, device);
        const float eps = static_cast<float>(number(a[3]));
        const int silu = static_cast<int>(integer(a[4]));
        const at::Tensor y = empty({T, H * D}, F8, device), scale = empty({T, H}, F32, device);
        const auto s = c10::cuda::getCurrentCUDAStream(static_cast<c10::DeviceIndex>(device)).stream();
        const int rc = without_gil([&] {
            return entry.norm(at_of(x), at_of(gate), stride, static_cast<const float *>(at_of(weight)), T, static_cast<int32_t>(H),
                              static_cast<int32_t>(D), eps, kind == F32, silu, y.mutable_data_ptr(),
                              static_cast<float *>(scale.mutable_data_ptr()), reinterpret_cast<kda_stream_t>(s));
        });
        return rc == KDA_OK ? pair(y, scale) : PyLong_FromLong(rc);
    });
}

PyObject *scaled_matmul(PyObject *, PyObject *const *a, Py_ssize_t n) {  // x, x_scale, weight, weight_scale
    return guarded(n, 4, [&]() -> PyObject * {
        const at::Tensor &x = tensor(a[0], F8), &xs = tensor(a[1], F32), &w = tensor(a[2], F8), &ws = tensor(a[3], F32);
        const int device = current(x);
        if (x.dim() < 1 || w.dim() != 2 || !x.is_contiguous()) throw Not{};
        const int64_t N = w.size(0), K = w.size(1), blocks = (K + 127) / 128;
        if (x.size(-1) != K || N > INT32_MAX || K > INT32_MAX) throw Not{};
        c10::SmallVector<int64_t, 5> shape(x.sizes().begin(), x.sizes().end());
        const bool per_block = xs.dim() == x.dim();
        int64_t rows = 1;
        for (int64_t i = 0; i + 1 < x.dim(); ++i) rows *= x.size(i);
        shape.back() = blocks;
        need(xs, per_block ? at::IntArrayRef(shape) : at::IntArrayRef(shape.data(), shape.size() - 1), device);
        need(w, {N, K}, device);
        need(ws, {(N + 127) / 128, blocks}, device);
        shape.back() = N;
        const at::Tensor y = empty(shape, BF16, device);
        const auto s = c10::cuda::getCurrentCUDAStream(static_cast<c10::DeviceIndex>(device)).stream();
        const int rc = without_gil([&] {
            return entry.product(at_of(x), static_cast<const float *>(at_of(xs)), per_block, at_of(w), static_cast<const float *>(at_of(ws)),
                                 rows, static_cast<int32_t>(K), static_cast<int32_t>(N), y.mutable_data_ptr(), nullptr,
                                 reinterpret_cast<kda_stream_t>(s));
        });
        return rc == KDA_OK ? THPVariable_Wrap(y) : PyLong_FromLong(rc);
    });
}

struct Delta {
    const at::Tensor &q, &k, &v, &g, &beta;
    int device;
    int64_t T, Hk, H, D, V, qs, ks, vs;
    const float *state = nullptr;
    Delta(PyObject *const *a, PyObject *s, int64_t num_seqs)
        : q(tensor(a[0], BF16)), k(tensor(a[1], BF16)), v(tensor(a[2], BF16)), g(tensor(a[3], F32)), beta(tensor(a[4], F32)),
          device(current(q)) {
        if (q.dim() != 3 || v.dim() != 3) throw Not{};
        T = q.size(0), Hk = q.size(1), D = q.size(2), H = v.size(1), V = v.size(2);
        qs = heads_view(q, T, device), ks = heads_view(k, T, device), vs = heads_view(v, T, device);
        if (k.sizes() != q.sizes() || Hk < 1 || H % Hk || H > INT32_MAX || D > INT32_MAX || V > INT32_MAX) throw Not{};
        need(g, {T, H}, device);
        need(beta, {T, H}, device);
        if (s != Py_None) {
            const at::Tensor &t = tensor(s, F32);
            need(t, {num_seqs, H, D, V}, device);
            state = static_cast<const float *>(at_of(t));
        }
    }
    float scale(PyObject *s) const { return static_cast<float>(s == Py_None ? std::pow(static_cast<double>(D), -0.5) : number(s)); }
    const float *f(const at::Tensor &t) const { return static_cast<const float *>(at_of(t)); }
};

PyObject *gated_delta_decode(PyObject *, PyObject *const *a, Py_ssize_t n) {  // q, k, v, g, beta, num_seqs, state, scale, in_place
    return guarded(n, 9, [&]() -> PyObject * {
        const int64_t N = integer(a[5]);
        const Delta d(a, a[6], N);
        if (N < 1 || N > INT32_MAX || d.T % N || d.T / N > INT32_MAX) throw Not{};
        const bool in_place = a[8] == Py_True;
        if (in_place && !d.state) throw Not{};
        const float scale = d.scale(a[7]);
        const at::Tensor o = empty({d.T, d.H, d.V}, BF16, d.device);
        const at::Tensor last = in_place ? THPVariable_Unpack(a[6]) : empty({N, d.H, d.D, d.V}, F32, d.device);
        const auto s = c10::cuda::getCurrentCUDAStream(static_cast<c10::DeviceIndex>(d.device)).stream();
        const int rc = without_gil([&] {
            return entry.decode(at_of(d.q), at_of(d.k), at_of(d.v), d.f(d.g), d.f(d.beta), static_cast<int32_t>(N),
                                static_cast<int32_t>(d.T / N), static_cast<int32_t>(d.H), static_cast<int32_t>(d.Hk),
                                static_cast<int32_t>(d.D), static_cast<int32_t>(d.V), d.qs, d.ks, d.vs, d.state, scale,
                                o.mutable_data_ptr(), static_cast<float *>(last.mutable_data_ptr()), nullptr,
                                reinterpret_cast<kda_stream_t>(s));
        });
        return rc == KDA_OK ? pair(o, last) : PyLong_FromLong(rc);
    });
}

PyObject *gated_delta_chunk(PyObject *, PyObject *const *a, Py_ssize_t n) {  // q, k, v, g, beta, cu_seqlens, state, scale, final state
    return guarded(n, 9, [&]() -> PyObject * {
        const at::Tensor &cu = tensor(a[5], I32);
        if (cu.dim() != 1 || cu.size(0) < 1 || cu.size(0) > INT32_MAX) throw Not{};
        const int64_t N = cu.size(0) - 1;
        const Delta d(a, a[6], N);
        need(cu, {N + 1}, d.device);
        const float scale = d.scale(a[7]);
        const at::Tensor o = empty({d.T, d.H, d.V}, BF16, d.device);
        at::Tensor last, workspace;
        if (a[8] == Py_True) last = empty({N, d.H, d.D, d.V}, F32, d.device);
        const size_t bytes = entry.workspace(static_cast<int32_t>(N), d.T, static_cast<int32_t>(d.H));
        if (bytes) workspace = empty({static_cast<int64_t>(bytes)}, U8, d.device);
        const auto s = c10::cuda::getCurrentCUDAStream(static_cast<c10::DeviceIndex>(d.device)).stream();
        const int rc = without_gil([&] {
            return entry.chunk(at_of(d.q), at_of(d.k), at_of(d.v), d.f(d.g), d.f(d.beta), static_cast<const int32_t *>(at_of(cu)),
                               static_cast<int32_t>(N), d.T, static_cast<int32_t>(d.H), static_cast<int32_t>(d.Hk),
                               static_cast<int32_t>(d.D), static_cast<int32_t>(d.V), d.qs, d.ks, d.vs, d.state, scale,
                               o.mutable_data_ptr(), last.defined() ? static_cast<float *>(last.mutable_data_ptr()) : nullptr, nullptr,
                               bytes ? workspace.mutable_data_ptr() : nullptr, bytes, reinterpret_cast<kda_stream_t>(s));
        });
        return rc == KDA_OK ? pair(o, last) : PyLong_FromLong(rc);
    });
}

PyObject *set_entry(PyObject *, PyObject *const *a, Py_ssize_t n) {  // addresses, in the order of `entry`
    void *p[5];
    if (n != 5) {
        PyErr_SetString(PyExc_TypeError, "five addresses");
        return nullptr;
    }
    for (int i = 0; i < 5; ++i) {
        p[i] = PyLong_AsVoidPtr(a[i]);
        if (PyErr_Occurred()) return nullptr;
    }
    entry = {reinterpret_cast<decltype(entry.norm)>(p[0]), reinterpret_cast<decltype(entry.product)>(p[1]),
             reinterpret_cast<decltype(entry.decode)>(p[2]), reinterpret_cast<decltype(entry.chunk)>(p[3]),
             reinterpret_cast<decltype(entry.workspace)>(p[4])};
    Py_RETURN_NONE;
}

#define FAST(f) reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(f)), METH_FASTCALL
PyMethodDef methods[] = {{"set_entry", FAST(set_entry), nullptr},
                         {"gated_rms_norm", FAST(gated_rms_norm), nullptr},
                         {"scaled_matmul", FAST(scaled_matmul), nullptr},
                         {"gated_delta_decode", FAST(gated_delta_decode), nullptr},
                         {"gated_delta_chunk", FAST(gated_delta_chunk), nullptr},
                         {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_native", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

// torch_version: of the torch whose headers this was compiled against. Tensors are read by their layout there, which another version need not
// have, and the loader would not notice.
PyMODINIT_FUNC PyInit__native() {
    PyObject *m = PyModule_Create(&module);
    if (m && PyModule_AddStringConstant(m, "torch_version", KDA_TORCH_VERSION) < 0) {
        Py_DECREF(m);
        return nullptr;
    }
    return m;
}
