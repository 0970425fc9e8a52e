// red_torch.cpp -- Python entry of the losses, of the root-mean-square norm and of
// the balance loss: torch tensors to the C calls of red.h.
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

    explicit Logits(PyObject *o, const char *name = "x") : x(tensor(o, name))
    {
        dtype = dtype_code(x.scalar_type(), name);
        if (!x.is_cuda())
            refuse("%s must be a CUDA tensor", name);
        if (x.dim() != 2)
            refuse("%s must be 2-D (rows, columns)", name);
        rows = x.size(0);
        len = x.size(1);
        ld = stride(x, name);
        device = x.get_device();
    }
    static int64_t stride(const at::Tensor &t, const char *name)
    {
        const int64_t rows = t.size(0), len = t.size(1);
        if (rows > 0 && len > 1 && t.stride(1) != 1)
            refuse("%s's rows must be contiguous (stride 1 along the columns)", name);
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

// ------------------------------------- log-probabilities without the logits

// Hidden states (rows, dim) and the vocabulary's weights (vocab, dim) beside
// them.  Both need what the C call's tensor maps need: rows from 16-byte
// boundaries on.
struct Linear {
    Logits h;
    const at::Tensor &w;
    int64_t vocab, ldw;

    Linear(PyObject *hidden, PyObject *weight) : h(hidden, "hidden"), w(tensor(weight, "weight"))
    {
        if (h.dtype == RED_F32)
            refuse("hidden must be float16 or bfloat16");
        if (w.scalar_type() != h.x.scalar_type() || !w.is_cuda() || w.get_device() != h.device || w.dim() != 2 ||
            w.size(1) != h.len)
            refuse("weight must be (vocab, dim) of hidden's dtype, dim and device");
        vocab = w.size(0);
        ldw = Logits::stride(w, "weight");
    }
    // Scratch of a call (freed on return: the allocator keeps it for this stream's later work).
    at::Tensor work(bool grad, int64_t *bytes) const
    {
        *bytes = red_linear_work_bytes(h.rows, h.len, vocab, grad);
        return at::empty({*bytes < 0 ? 0 : *bytes}, h.x.options().dtype(at::kByte));
    }
    // A gradient: None for a new matrix (rows on 16-byte boundaries), False for none, or one to write.
    struct Out {
        at::Tensor t;
        void *ptr = nullptr;
        int64_t ld = 0;
    };
    Out out(PyObject *o, const at::Tensor &like, const char *name) const
    {
        Out g;
        if (o == Py_False)
            return g;
        if (o == Py_None) {
            const int64_t ld = (h.len + 7) / 8 * 8;
            g.t = ld == h.len ? at::empty(like.sizes(), like.options())
                              : at::empty_strided(like.sizes(), {ld, 1}, like.options());
        } else {
            g.t = tensor(o, name);
            if (g.t.scalar_type() != like.scalar_type() || !g.t.is_cuda() || g.t.get_device() != h.device ||
                g.t.sizes() != like.sizes())
                refuse("%s must have the dtype, device and shape of what it is the gradient of", name);
        }
        g.ld = Logits::stride(g.t, name);
        g.ptr = g.t.data_ptr();
        return g;
    }
};

// (hidden, weight, target, scale, stream)
PyObject *linear_logprob(PyObject *, PyObject *const *a, Py_ssize_t n)
{
    return guarded("linear_logprob", n, 5, [&] {
        const Linear l(a[0], a[1]);
        const OnStream on(a[4], l.h);
        const int64_t *target = l.h.vector<int64_t>(a[2], "target", l.h.rows);
        const auto [logp, lse] = float_vectors(l.h, {l.h.rows, l.h.rows});
        int64_t bytes;
        const at::Tensor work = l.work(false, &bytes);
        RETURN_IF_REFUSED(red_linear_logprob(l.h.dtype, l.h.x.data_ptr(), l.h.rows, l.h.len, l.h.ld, l.w.data_ptr(),
                                             l.vocab, l.ldw, (float)number(a[3]), target, data(logp), data(lse),
                                             work.data_ptr(), bytes, on.stream));
        return results(logp, lse);
    });
}

// (hidden, weight, target, lse, dlogp, dlse, scale, grad_hidden, grad_weight, stream)
PyObject *linear_logprob_grad(PyObject *, PyObject *const *a, Py_ssize_t n)
{
    return guarded("linear_logprob_grad", n, 10, [&] {
        const Linear l(a[0], a[1]);
        const OnStream on(a[9], l.h);
        const int64_t rows = l.h.rows;
        const int64_t *target = l.h.vector<int64_t>(a[2], "target", rows);
        const float *lse = l.h.vector<float>(a[3], "lse", rows), *dlogp = l.h.vector<float>(a[4], "dlogp", rows);
        const float *dlse = l.h.vector<float>(a[5], "dlse", rows);
        const auto gh = l.out(a[7], l.h.x, "grad_hidden"), gw = l.out(a[8], l.w, "grad_weight");
        int64_t bytes;
        const at::Tensor work = l.work(true, &bytes);
        RETURN_IF_REFUSED(red_linear_logprob_grad(l.h.dtype, l.h.x.data_ptr(), rows, l.h.len, l.h.ld, l.w.data_ptr(),
                                                  l.vocab, l.ldw, (float)number(a[6]), target, lse, dlogp, dlse, gh.ptr,
                                                  gh.ld, gw.ptr, gw.ld, work.data_ptr(), bytes, on.stream));
        return results(gh.t, gw.t);
    });
}

// ------------------------------------------------- root-mean-square norm

// New results of a call.  Small ones share an allocation: each is a microsecond of the
// host's time, and that of a norm of one row is 2 us on the GPU.  Large ones do not, so
// that one that is kept keeps no other's memory.
class Results {
    static constexpr int64_t SMALL = 1 << 20, ALIGN = 128;
    const Logits &l;
    const bool merged;
    at::Tensor whole;
    int64_t used = 0;

public:
    // `bytes`: of all of them, `count` in number.
    Results(const Logits &like, int64_t bytes, int count) : l(like), merged(bytes <= SMALL)
    {
        if (merged)
            whole = at::empty({bytes + count * ALIGN}, l.x.options().dtype(at::kByte));
    }
    at::Tensor rows(int64_t n, int64_t cols, int64_t ld, at::ScalarType type)
    {
        if (!merged)
            return ld == cols ? at::empty({n, cols}, l.x.options().dtype(type))
                              : at::empty_strided({n, cols}, {ld, 1}, l.x.options().dtype(type));
        return part({n, cols}, {ld, 1}, n * ld, type);
    }
    at::Tensor vector(int64_t n, at::ScalarType type)
    {
        return merged ? part({n}, {1}, n, type) : at::empty({n}, l.x.options().dtype(type));
    }

private:
    at::Tensor part(c10::IntArrayRef sizes, c10::IntArrayRef strides, int64_t elements, at::ScalarType type)
    {
        auto impl = c10::make_intrusive<c10::TensorImpl>(c10::TensorImpl::VIEW, c10::Storage(whole.storage()),
                                                         whole.key_set(), c10::scalarTypeToTypeMeta(type));
        const int64_t size = (int64_t)c10::elementSize(type);
        impl->set_storage_offset(used / size);
        impl->set_sizes_and_strides(sizes, strides);
        used += (elements * size + ALIGN - 1) / ALIGN * ALIGN;
        return at::Tensor(std::move(impl));
    }
};

// Row stride of a new matrix like x: x's where that is a padding, else (rows out of a
// larger tensor: every row would take as much memory as in that) to the next 16 bytes.
int64_t new_ld(const Logits &l)
{
    const int64_t unit = 16 / (int64_t)l.x.element_size();
    return l.ld - l.len <= 128 ? l.ld : (l.len + unit - 1) / unit * unit;
}

// A matrix like x: dtype, device and shape; its row stride through *ld.
const at::Tensor &beside(const Logits &l, PyObject *o, const char *name, int64_t *ld)
{
    const at::Tensor &t = tensor(o, name);
    if (t.scalar_type() != l.x.scalar_type() || !t.is_cuda() || t.get_device() != l.device || t.sizes() != l.x.sizes())
        refuse("%s must have x's dtype, device and shape", name);
    *ld = Logits::stride(t, name);
    return t;
}
// The weight (len values of x's type or fp32; None: 1) and its type.
const void *norm_weight(const Logits &l, PyObject *o, int *wtype)
{
    *wtype = l.dtype;
    if (o == Py_None)
        return nullptr;
    const at::Tensor &t = tensor(o, "weight");
    *wtype = dtype_code(t.scalar_type(), "weight");
    if (!t.is_cuda() || t.get_device() != l.device || t.numel() != l.len || !t.is_contiguous())
        refuse("weight must be a contiguous vector of x's columns on x's device");
    return t.data_ptr();
}

struct NormInputs {
    Logits l;
    const void *residual = nullptr, *weight;
    int64_t ldr = 0, ldt = 0;
    int wtype;
    bool with_residual;  // (a matrix without rows has no address)
    at::Tensor total, rstd;

    NormInputs(PyObject *x, PyObject *w, PyObject *res) : l(x)
    {
        weight = norm_weight(l, w, &wtype);
        with_residual = res != Py_None;
        if (with_residual)
            residual = beside(l, res, "residual", &ldr).data_ptr();
    }
    // After the stream is set: what the call allocates is that stream's.
    void results(Results &made, PyObject *given_total)
    {
        if (with_residual) {
            total = given_total == Py_None ? made.rows(l.rows, l.len, new_ld(l), l.x.scalar_type())
                                           : beside(l, given_total, "total", &ldt);
            ldt = Logits::stride(total, "total");
        } else if (given_total != Py_None) {
            refuse("total comes with a residual");
        }
        rstd = made.vector(l.rows, at::kFloat);
    }
    // Bytes of y (or 8-bit values and scales), total and rstd, at most.
    int64_t bytes() const { return l.rows * (2 * new_ld(l) * (int64_t)l.x.element_size() + 4 * (l.len / 32 + 2)); }
    void *total_ptr() const { return total.defined() ? total.data_ptr() : nullptr; }
};

// (x, weight, residual, eps, out, total, stream)
PyObject *rmsnorm(PyObject *, PyObject *const *a, Py_ssize_t n)
{
    return guarded("rmsnorm", n, 7, [&] {
        NormInputs in(a[0], a[1], a[2]);
        const OnStream on(a[6], in.l);
        int64_t ldy = new_ld(in.l);
        Results made(in.l, in.bytes(), 3);
        const at::Tensor y = a[4] == Py_None ? made.rows(in.l.rows, in.l.len, ldy, in.l.x.scalar_type())
                                             : beside(in.l, a[4], "out", &ldy);
        in.results(made, a[5]);
        RETURN_IF_REFUSED(red_rmsnorm(in.l.dtype, in.l.x.data_ptr(), in.l.rows, in.l.len, in.l.ld, in.residual, in.ldr,
                                      in.wtype, in.weight, (float)number(a[3]), y.data_ptr(), ldy, in.total_ptr(),
                                      in.ldt, data(in.rstd), on.stream));
        return results(y, in.total, in.rstd);
    });
}

// (x, weight, residual, eps, kind, block, out, total, stream)
PyObject *rmsnorm_quant(PyObject *, PyObject *const *a, Py_ssize_t n)
{
    return guarded("rmsnorm_quant", n, 9, [&] {
        NormInputs in(a[0], a[1], a[2]);
        const OnStream on(a[8], in.l);
        const int kind = integer(a[4], "kind"), block = integer(a[5], "block");
        const at::ScalarType type = kind == RED_QUANT_I8 ? at::kChar : at::kFloat8_e4m3fn;
        Results made(in.l, in.bytes(), 4);
        at::Tensor q;
        if (a[6] == Py_None) {
            q = made.rows(in.l.rows, in.l.len, in.l.len, type);
        } else {
            q = tensor(a[6], "out");
            if (q.scalar_type() != type || !q.is_cuda() || q.get_device() != in.l.device || q.sizes() != in.l.x.sizes())
                refuse("out must be of the 8-bit type, on x's device and of x's shape");
        }
        // (a block that the call refuses has no scales)
        const int64_t blocks = block > 0 ? (in.l.len + block - 1) / block : 1;
        const at::Tensor scales = made.rows(block < 32 ? in.l.rows * (block == 0) : in.l.rows, blocks, blocks, at::kFloat);
        in.results(made, a[7]);
        RETURN_IF_REFUSED(red_rmsnorm_quant(in.l.dtype, in.l.x.data_ptr(), in.l.rows, in.l.len, in.l.ld, in.residual,
                                            in.ldr, in.wtype, in.weight, (float)number(a[3]), kind, block, q.data_ptr(),
                                            Logits::stride(q, "out"), data(scales), in.total_ptr(), in.ldt,
                                            data(in.rstd), on.stream));
        return results(q, scales, in.total, in.rstd);
    });
}

// (dy, x, rstd, weight, dtotal, grad, grad_weight, stream)
PyObject *rmsnorm_grad(PyObject *, PyObject *const *a, Py_ssize_t n)
{
    return guarded("rmsnorm_grad", n, 8, [&] {
        const Logits l(a[1]);
        const OnStream on(a[7], l);
        int64_t lddy, ldt = 0, ldd = new_ld(l);
        const at::Tensor &dy = beside(l, a[0], "dy", &lddy);
        const float *rstd = l.vector<float>(a[2], "rstd", l.rows);
        int wtype;
        const void *weight = norm_weight(l, a[3], &wtype);
        const void *dtotal = a[4] == Py_None ? nullptr : beside(l, a[4], "dtotal", &ldt).data_ptr();
        Results made(l, l.rows * ldd * (int64_t)l.x.element_size() + 4 * l.len, 2);
        const at::Tensor dx = a[5] == Py_None ? made.rows(l.rows, l.len, ldd, l.x.scalar_type())
                                              : beside(l, a[5], "grad", &ldd);
        at::Tensor dw;
        if (a[6] == Py_None) {
            if (weight)
                dw = made.vector(l.len, tensor(a[3], "weight").scalar_type());
        } else if (a[6] != Py_False) {
            dw = tensor(a[6], "grad_weight");
            if (dw.scalar_type() != (weight ? tensor(a[3], "weight") : l.x).scalar_type() || !dw.is_cuda() ||
                dw.get_device() != l.device || dw.numel() != l.len || !dw.is_contiguous())
                refuse("grad_weight must be a contiguous vector of weight's dtype, size and device");
        }
        RETURN_IF_REFUSED(red_rmsnorm_grad(l.dtype, dy.data_ptr(), lddy, l.x.data_ptr(), l.rows, l.len, l.ld, rstd, wtype,
                                           weight, dtotal, ldt, dx.data_ptr(), ldd,
                                           dw.defined() ? dw.data_ptr() : nullptr, on.stream));
        return results(dx, dw);
    });
}

// ------------------------------------------------------------ balance loss

// (x, ids, live, coef, z_coef, kind, grad_scale, grad, stream)
PyObject *balance(PyObject *, PyObject *const *a, Py_ssize_t n)
{
    return guarded("balance", n, 9, [&] {
        const Logits l(a[0]);
        const OnStream on(a[8], l);
        const at::Tensor &ids = tensor(a[1], "ids");
        if (ids.dim() != 2 || ids.size(0) != l.rows)
            refuse("ids must be (rows, k)");
        const int64_t k = ids.size(1);
        const int64_t *id = l.vector<int64_t>(a[1], "ids", l.rows * k);
        const uint8_t *live = nullptr;
        if (a[2] != Py_None) {
            const at::Tensor &t = tensor(a[2], "live");
            if ((t.scalar_type() != at::kBool && t.scalar_type() != at::kByte) || !t.is_cuda() ||
                t.get_device() != l.device || t.numel() != l.rows || !t.is_contiguous())
                refuse("live must be a contiguous vector of one bool or uint8 per row on x's device");
            live = static_cast<const uint8_t *>(t.data_ptr());
        }
        int64_t ldd = new_ld(l);
        Results made(l, l.rows * ldd * (int64_t)l.x.element_size() + 12 * l.len + 16, 4);
        at::Tensor dx;
        if (a[7] == Py_None)
            dx = made.rows(l.rows, l.len, ldd, l.x.scalar_type());
        else if (a[7] != Py_False)
            dx = beside(l, a[7], "grad", &ldd);
        const at::Tensor counts = made.vector(l.len, at::kLong), prob = made.vector(l.len, at::kFloat),
                         stats = made.vector(4, at::kFloat);
        RETURN_IF_REFUSED(red_balance(l.dtype, l.x.data_ptr(), l.rows, l.len, l.ld, id, k, live,
                                      integer(a[5], "kind"), (float)number(a[3]), (float)number(a[4]),
                                      (float)number(a[6]), static_cast<int64_t *>(counts.data_ptr()), data(prob),
                                      data(stats), dx.defined() ? dx.data_ptr() : nullptr, ldd, on.stream));
        return results(counts, prob, stats, dx);
    });
}

#define FAST(name) {#name, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(name)), METH_FASTCALL, nullptr}
PyMethodDef methods[] = {FAST(logprob), FAST(logprob_grad), FAST(distill), FAST(policy), FAST(preference),
                         FAST(linear_logprob), FAST(linear_logprob_grad), FAST(rmsnorm),
                         FAST(rmsnorm_quant), FAST(rmsnorm_grad), FAST(balance),
                         {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_red_torch", "Losses and norms of libred.so on torch tensors.", -1, methods,
                      nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__red_torch() { return PyModule_Create(&module); }
