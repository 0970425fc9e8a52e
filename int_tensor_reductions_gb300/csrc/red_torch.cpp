// red_torch.cpp -- Python entry of the losses over rows of logits: torch
// tensors to the C calls of red.h.
//
// One training step on a few rows, or the scoring of one token, takes the GPU
// 2 to 10 us; checking and unpacking a dozen tensors and allocating the
// results in interpreted Python takes 20 (measured on the GB300's host).  Here
// that is about 5.  The functions below do what the wrappers of the other
// calls do in Python (dtype, device, size and layout checks that raise
// ValueError, allocation, the current stream) and return the results, or the
// status as an int when the C call refuses.
#define PY_SSIZE_T_CLEAN
#include <Python.h>

#include <array>

#include <ATen/core/Tensor.h>
#include <ATen/ops/empty.h>
#include <ATen/ops/empty_strided.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include "red.h"

namespace {

struct Refused {};  // a Python exception is set

template <typename... A>
[[noreturn]] void refuse(const char *fmt, A... a)
{
    PyErr_Format(PyExc_ValueError, fmt, a...);
    throw Refused();
}

const at::Tensor &tensor(PyObject *o, const char *name)
{
    if (!THPVariable_Check(o)) {
        PyErr_Format(PyExc_TypeError, "%s must be a tensor", name);
        throw Refused();
    }
    return THPVariable_Unpack(o);
}

double number(PyObject *o)
{
    const double v = PyFloat_AsDouble(o);
    if (v == -1.0 && PyErr_Occurred())
        throw Refused();
    return v;
}

int integer(PyObject *o, const char *name)
{
    const long long v = PyLong_AsLongLong(o);
    if (v == -1 && PyErr_Occurred())
        throw Refused();
    if (v != static_cast<int>(v))
        refuse("%s = %lld is out of range", name, v);
    return static_cast<int>(v);
}

int dtype_code(at::ScalarType t, const char *name)
{
    switch (t) {
    case at::kFloat: return RED_F32;
    case at::kHalf: return RED_F16;
    case at::kBFloat16: return RED_BF16;
    default: refuse("%s must be float32, float16 or bfloat16", name);
    }
}

// The logits: a 2-D CUDA tensor of contiguous rows.
struct Logits {
    const at::Tensor &x;
    int dtype;
    int64_t rows, len, ld;
    int device;

    explicit Logits(PyObject *o) : x(tensor(o, "x"))
    {
        dtype = dtype_code(x.scalar_type(), "x");
        if (!x.is_cuda())
            refuse("x must be a CUDA tensor");
        if (x.dim() != 2)
            refuse("x must be 2-D (rows, vocab)");
        rows = x.size(0);
        len = x.size(1);
        ld = stride(x, "x");
        device = x.get_device();
    }
    static int64_t stride(const at::Tensor &t, const char *name)
    {
        const int64_t rows = t.size(0), len = t.size(1);
        if (rows > 0 && len > 1 && t.stride(1) != 1)
            refuse("%s's rows must be contiguous (stride 1 along the vocabulary)", name);
        const int64_t ld = rows > 1 ? t.stride(0) : len;
        if (ld < len)
            refuse("%s's row stride is smaller than its number of columns", name);
        return ld;
    }
    // A contiguous vector of n elements beside x; NULL for None.
    template <class T>
    const T *vector(PyObject *o, const char *name, int64_t n) const
    {
        if (o == Py_None)
            return nullptr;
        const at::Tensor &t = tensor(o, name);
        const bool ids = std::is_same<T, int64_t>::value;
        if (t.scalar_type() != (ids ? at::kLong : at::kFloat))
            refuse("%s must have dtype %s", name, ids ? "int64" : "float32");
        if (!t.is_cuda() || t.get_device() != device)
            refuse("%s must be on x's device", name);
        if (t.numel() != n)
            refuse("%s must hold %lld element(s), has %lld", name, (long long)n, (long long)t.numel());
        if (!t.is_contiguous())
            refuse("%s must be contiguous", name);
        return static_cast<const T *>(t.data_ptr());
    }
    at::Tensor floats(int64_t n) const { return at::empty({n}, x.options().dtype(at::kFloat)); }
};

// Vectors of floats in one allocation, each from a 16-byte boundary on: an
// allocation is a microsecond of the host's time.
template <size_t N>
std::array<at::Tensor, N> float_vectors(const Logits &l, const int64_t (&sizes)[N])
{
    int64_t total = 0;
    for (const int64_t n : sizes)
        total += (n + 3) / 4 * 4;
    const at::Tensor whole = l.floats(total);
    std::array<at::Tensor, N> parts;
    int64_t begin = 0;
    for (size_t i = 0; i < N; ++i) {
        auto part = c10::make_intrusive<c10::TensorImpl>(c10::TensorImpl::VIEW, c10::Storage(whole.storage()),
                                                         whole.key_set(), whole.dtype());
        part->set_storage_offset(begin);
        part->set_sizes_contiguous(sizes[i]);
        parts[i] = at::Tensor(std::move(part));
        begin += (sizes[i] + 3) / 4 * 4;
    }
    return parts;
}

float *data(const at::Tensor &t) { return static_cast<float *>(t.data_ptr()); }

// The gradient: None for a new tensor of x's row stride, False for none, or a
// tensor of x's shape to write (x itself for in place).
struct Gradient {
    at::Tensor t;
    void *ptr = nullptr;
    int64_t ld = 0;

    Gradient(PyObject *o, const Logits &l, const char *name)
    {
        if (o == Py_False)
            return;
        if (o == Py_None) {
            t = l.ld == l.len ? at::empty({l.rows, l.len}, l.x.options())
                              : at::empty_strided({l.rows, l.len}, {l.ld, 1}, l.x.options());
            ld = l.ld;
        } else {
            t = tensor(o, name);
            if (t.scalar_type() != l.x.scalar_type() || !t.is_cuda() || t.get_device() != l.device ||
                t.sizes() != l.x.sizes())
                refuse("%s must have x's dtype, device and shape", name);
            ld = Logits::stride(t, name);
        }
        ptr = t.data_ptr();
    }
};

PyObject *wrap(const at::Tensor &t)
{
    if (!t.defined())
        Py_RETURN_NONE;
    return THPVariable_Wrap(t);
}

template <typename... T>
PyObject *results(const T &...t)
{
    PyObject *r = PyTuple_New(sizeof...(t));
    if (!r)
        throw Refused();
    Py_ssize_t i = 0;
    bool ok = true;
    for (PyObject *o : {wrap(t)...}) {
        ok = ok && o;
        PyTuple_SET_ITEM(r, i++, o);
    }
    if (!ok) {
        Py_DECREF(r);
        throw Refused();
    }
    return r;
}

// The stream of a call: an address, or the device's current one for None.  It is
// the current one while this lives, so that what the call allocates is memory of
// that stream: a block of the caller's own stream may still be in use there.
struct OnStream {
    c10::cuda::OptionalCUDAGuard device;
    c10::cuda::OptionalCUDAStreamGuard given;
    red_stream_t stream;

    OnStream(PyObject *o, const Logits &l)
    {
        if (o == Py_None) {
            device.set_index(l.device);
            stream = reinterpret_cast<red_stream_t>(c10::cuda::getCurrentCUDAStream(l.device).stream());
            return;
        }
        const unsigned long long address = PyLong_AsUnsignedLongLong(o);
        if (PyErr_Occurred())
            throw Refused();
        stream = reinterpret_cast<red_stream_t>(static_cast<uintptr_t>(address));
        given.reset_stream(c10::cuda::getStreamFromExternal(reinterpret_cast<cudaStream_t>(stream),
                                                            static_cast<c10::DeviceIndex>(l.device)));
    }
};

template <class F>
PyObject *guarded(const char *name, Py_ssize_t given, Py_ssize_t wanted, F f)
{
    if (given != wanted) {
        PyErr_Format(PyExc_TypeError, "%s takes %zd arguments", name, wanted);
        return nullptr;
    }
    HANDLE_TH_ERRORS  // torch's exceptions as Python's
    try {
        return f();
    } catch (const Refused &) {
        return nullptr;
    }
    END_HANDLE_TH_ERRORS
}

#define RETURN_IF_REFUSED(status) \
    if ((status) != RED_OK)       \
        return PyLong_FromLong(status)

// (x, target, scale, out, lse, stream)
PyObject *logprob(PyObject *, PyObject *const *a, Py_ssize_t n)
{
    return guarded("logprob", n, 6, [&] {
        const Logits l(a[0]);
        const OnStream on(a[5], l);
        const int64_t *target = l.vector<int64_t>(a[1], "target", l.rows);
        const float *given = l.vector<float>(a[3], "out", l.rows), *given_lse = l.vector<float>(a[4], "lse", l.rows);
        at::Tensor out, lse;
        if (!given && !given_lse) {
            auto made = float_vectors(l, {l.rows, l.rows});
            out = std::move(made[0]);
            lse = std::move(made[1]);
        } else {
            out = given ? tensor(a[3], "out") : l.floats(l.rows);
            lse = given_lse ? tensor(a[4], "lse") : l.floats(l.rows);
        }
        RETURN_IF_REFUSED(red_logprob(l.dtype, l.x.data_ptr(), l.rows, l.len, l.ld, (float)number(a[2]), target,
                                      data(out), data(lse), on.stream));
        return results(out, lse);
    });
}

// (x, target, lse, dlogp, scale, out, stream)
PyObject *logprob_grad(PyObject *, PyObject *const *a, Py_ssize_t n)
{
    return guarded("logprob_grad", n, 7, [&] {
        const Logits l(a[0]);
        const OnStream on(a[6], l);
        if (a[5] == Py_False)
            refuse("out must be a tensor or None");
        const int64_t *target = l.vector<int64_t>(a[1], "target", l.rows);
        const float *lse = l.vector<float>(a[2], "lse", l.rows), *dlogp = l.vector<float>(a[3], "dlogp", l.rows);
        const Gradient g(a[5], l, "out");
        RETURN_IF_REFUSED(red_logprob_grad(l.dtype, l.x.data_ptr(), l.rows, l.len, l.ld, (float)number(a[4]), target,
                                           lse, dlogp, g.ptr, g.ld, on.stream));
        return wrap(g.t);
    });
}

// (x, ids, vals, lse, weight, scale, grad_scale, grad, stream)
PyObject *distill(PyObject *, PyObject *const *a, Py_ssize_t n)
{
    return guarded("distill", n, 9, [&] {
        const Logits l(a[0]);
        const OnStream on(a[8], l);
        const at::Tensor &ids = tensor(a[1], "ids"), &vals = tensor(a[2], "vals");
        if (ids.dim() != 2 || vals.sizes() != ids.sizes() || ids.size(0) != l.rows)
            refuse("ids and vals must be (rows, k)");
        const int64_t k = ids.size(1);
        const int vcode = dtype_code(vals.scalar_type(), "vals");
        if (!vals.is_cuda() || vals.get_device() != l.device || !vals.is_contiguous())
            refuse("vals must be contiguous and on x's device");
        const int64_t *id = l.vector<int64_t>(a[1], "ids", l.rows * k);
        const float *lse = l.vector<float>(a[3], "lse", l.rows), *weight = l.vector<float>(a[4], "weight", l.rows);
        const Gradient g(a[7], l, "grad");
        const auto [loss, stats] = float_vectors(l, {l.rows, 2});
        RETURN_IF_REFUSED(red_distill(l.dtype, l.x.data_ptr(), l.rows, l.len, l.ld, (float)number(a[5]), k, id, vcode,
                                      vals.data_ptr(), lse, weight, (float)number(a[6]), data(loss), data(stats),
                                      g.ptr, g.ld, on.stream));
        return results(loss, stats, g.t);
    });
}

// (x, target, old_logp, adv, ref_logp, weight, clip_low, clip_high, kl_coef, scale, grad_scale, grad, stream)
PyObject *policy(PyObject *, PyObject *const *a, Py_ssize_t n)
{
    return guarded("policy", n, 13, [&] {
        const Logits l(a[0]);
        const OnStream on(a[12], l);
        const int64_t *target = l.vector<int64_t>(a[1], "target", l.rows);
        const float *old_logp = l.vector<float>(a[2], "old_logp", l.rows), *adv = l.vector<float>(a[3], "adv", l.rows);
        const float *ref = l.vector<float>(a[4], "ref_logp", l.rows), *weight = l.vector<float>(a[5], "weight", l.rows);
        const Gradient g(a[11], l, "grad");
        const auto [loss, logp, stats] = float_vectors(l, {l.rows, l.rows, 4});
        RETURN_IF_REFUSED(red_policy(l.dtype, l.x.data_ptr(), l.rows, l.len, l.ld, (float)number(a[9]), target,
                                     old_logp, ref, adv, weight, (float)number(a[6]), (float)number(a[7]),
                                     (float)number(a[8]), (float)number(a[10]), data(loss), data(logp), data(stats),
                                     g.ptr, g.ld, on.stream));
        return results(loss, logp, stats, g.t);
    });
}

// (x, target, offsets, ref_logp, weight, kind, beta, margin, smoothing, average, scale, grad_scale, grad, stream)
PyObject *preference(PyObject *, PyObject *const *a, Py_ssize_t n)
{
    return guarded("preference", n, 14, [&] {
        const Logits l(a[0]);
        const OnStream on(a[13], l);
        const int64_t entries = tensor(a[2], "offsets").numel();
        if (entries % 2 != 1)
            refuse("offsets needs 2 * pairs + 1 entries");
        const int64_t pairs = entries / 2;
        const int64_t *target = l.vector<int64_t>(a[1], "target", l.rows);
        const int64_t *offsets = l.vector<int64_t>(a[2], "offsets", entries);
        const float *ref = l.vector<float>(a[3], "ref_logp", 2 * pairs), *weight = l.vector<float>(a[4], "weight", pairs);
        const Gradient g(a[12], l, "grad");
        const auto [loss, seq, stats] = float_vectors(l, {pairs, 2 * pairs, 4});
        // (freed on return: the allocator keeps it for this stream's later work)
        const at::Tensor work = l.floats(3 * l.rows + pairs);
        const int average = PyObject_IsTrue(a[9]);
        if (average < 0)
            throw Refused();
        RETURN_IF_REFUSED(red_preference(l.dtype, l.x.data_ptr(), l.rows, l.len, l.ld, (float)number(a[10]), target,
                                         offsets, pairs, ref, weight, integer(a[5], "kind"), (float)number(a[6]),
                                         (float)number(a[7]), (float)number(a[8]), average, (float)number(a[11]),
                                         data(loss), data(seq), data(stats), data(work), g.ptr, g.ld,
                                         on.stream));
        return results(loss, seq, stats, g.t);
    });
}

#define FAST(name) {#name, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(name)), METH_FASTCALL, nullptr}
PyMethodDef methods[] = {FAST(logprob), FAST(logprob_grad), FAST(distill), FAST(policy), FAST(preference),
                         {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_red_torch", "Losses of libred.so on torch tensors.", -1, methods,
                      nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__red_torch() { return PyModule_Create(&module); }
