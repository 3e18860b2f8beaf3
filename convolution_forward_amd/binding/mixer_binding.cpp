// Python binding of the token-mixer calls (include/convfwd.h), for their host
// time: a single token's kernel takes a few microseconds, and marshalling the
// same arguments in Python took longer than it (12.7 us a call against 5 us
// of kernel). Argument marshalling only, as in the rest of the binding: the
// checks here are those that need tensors (type, shape, layout, device), the
// library makes the others.
//
// Each function takes exactly the positional arguments that mixer.py passes,
// raises ValueError for a tensor that does not fit, and returns its outputs,
// or the library's status as an int where that is not CONV_OK.
#include <Python.h>

#include <ATen/ATen.h>
#include <c10/core/DeviceGuard.h>
#include <c10/hip/HIPStream.h>
#include <torch/csrc/Dtype.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include <sstream>
#include <string>

#include "convfwd.h"

namespace {

struct ValueError {
    std::string what;
};

template <class... A>
[[noreturn]] void refuse(const A &...parts)
{
    std::ostringstream s;
    (s << ... << parts);
    throw ValueError{s.str()};
}

using Tensor = at::Tensor;

const Tensor *maybe(PyObject *o, const char *what)
{
    if (o == Py_None)
        return nullptr;
    if (!THPVariable_Check(o))
        refuse(what, " must be a tensor");
    return &THPVariable_Unpack(o);
}

const Tensor &tensor(PyObject *o, const char *what)
{
    const Tensor *t = maybe(o, what);
    if (!t)
        refuse(what, " must be a tensor");
    return *t;
}

long long integer(PyObject *o)
{
    const long long v = PyLong_AsLongLong(o);
    if (v == -1 && PyErr_Occurred())
        throw python_error();
    return v;
}

double number(PyObject *o)
{
    const double v = PyFloat_AsDouble(o);
    if (v == -1.0 && PyErr_Occurred())
        throw python_error();
    return v;
}

at::ScalarType dtype_of(PyObject *o, const char *what)
{
    if (!THPDtype_Check(o))
        refuse(what, " must be a torch.dtype");
    return reinterpret_cast<THPDtype *>(o)->scalar_type;
}

conv_dtype float_code(at::ScalarType t, const char *what)
{
    if (t == at::kFloat)
        return CONV_F32;
    if (t != at::kBFloat16)
        refuse(what, ": unsupported dtype ", t, "; use float32 or bfloat16");
    return CONV_BF16;
}

conv_dtype eight_code(at::ScalarType t, const char *what)
{
    if (t == at::kChar)
        return CONV_I8;
    if (t != at::kFloat8_e4m3fn)
        refuse(what, ": unsupported dtype ", t, "; use int8 or float8_e4m3fn");
    return CONV_E4M3;
}

void *ptr(const Tensor *t) { return t ? t->data_ptr() : nullptr; }
void *ptr(const Tensor &t) { return t.data_ptr(); }

// All on the first one's GPU.
template <class... T>
void same_gpu(const Tensor &first, const T *...others)
{
    if (!first.is_cuda())
        refuse("tensors must live on the GPU (no CPU path exists)");
    const auto gpu = first.device();
    auto check = [&](const Tensor *t) {
        if (t && t->device() != gpu)
            refuse("tensors on ", gpu, " and ", t->device(), ": all must be on one GPU");
    };
    (check(others), ...);
}

void *stream_of(const Tensor &t) { return c10::hip::getCurrentHIPStream(t.device().index()).stream(); }

Tensor fresh(const Tensor &like, at::IntArrayRef sizes, at::ScalarType t)
{
    return at::empty(sizes, like.options().dtype(t));
}

void *vector(const Tensor *t, int64_t n, at::ScalarType type, const char *what)
{
    if (!t)
        return nullptr;
    if (t->scalar_type() != type || t->numel() != n || !t->is_contiguous())
        refuse(what, " must be a contiguous ", type, " tensor of ", n, " values");
    return t->data_ptr();
}

// Row stride of a [..., width] tensor whose channels are adjacent and whose rows are evenly spaced.
int64_t row_stride(const Tensor &t, const char *what, int64_t width, int64_t rows, at::ScalarType type)
{
    const int64_t dim = t.dim();
    if (dim >= 1 && t.size(-1) == width && t.scalar_type() == type && (width == 0 || t.numel() / width == rows)) {
        if (t.is_contiguous())
            return width;
        if (t.stride(-1) == 1 || width == 1) {
            int64_t step = 0, count = 0;        // from the innermost axis of more than one row outwards
            bool even = true;
            for (int64_t d = dim - 2; d >= 0 && even; --d) {
                if (t.size(d) == 1)
                    continue;
                if (count)
                    even = t.stride(d) == step * count;
                else
                    step = t.stride(d);
                count = (count ? count : 1) * t.size(d);
            }
            if (even)
                return count ? step : width;
        }
    }
    refuse(what, " must hold ", rows, " evenly spaced rows of ", width, " adjacent ", type, " values, got ", t.sizes(), " ",
           t.scalar_type(), " with strides ", t.strides());
}

int small(int64_t v, const char *what)
{
    if (v > INT32_MAX)
        refuse(what, " of ", v, " is too large");
    return (int)v;
}

// (tokens, sequences) of a tensor [batch, length, ...] or [tokens, ...] whose last `tail` axes are not tokens.
struct Seqs {
    int64_t tokens;
    int count;
};

Seqs sequences(const Tensor &t, int64_t tail, const Tensor *offsets)
{
    const int64_t dim = t.dim() - tail;
    if (dim == 2) {
        if (offsets)
            refuse("seq_offsets go with [tokens, ...] tensors");
        return {t.size(0) * t.size(1), small(t.size(0), "a count of sequences")};
    }
    if (dim != 1)
        refuse("expected [batch, length, ...] or [tokens, ...], got ", t.sizes());
    if (!offsets)
        return {t.size(0), 1};
    if (offsets->scalar_type() != at::kInt || offsets->dim() != 1 || offsets->numel() < 2 || !offsets->is_contiguous())
        refuse("seq_offsets must be a contiguous int32 tensor of num_seqs + 1 values");
    return {t.size(0), small(offsets->numel() - 1, "a count of sequences")};
}

// Slots of a state tensor [slots, *shape]; `slots`, if any, is what another has.
int64_t state(const Tensor *t, at::IntArrayRef shape, at::ScalarType type, int64_t slots)
{
    if (!t)
        return slots;
    if (t->scalar_type() != type || t->dim() != (int64_t)shape.size() + 1 || t->sizes().slice(1) != shape ||
        !t->is_contiguous())
        refuse("states must be contiguous ", type, " tensors [slots, ", shape, "], got ", t->sizes(), " ", t->scalar_type());
    if (slots && t->size(0) != slots)
        refuse("initial_state and final_state must have as many slots");
    return t->size(0);
}

// (token, head) strides of [tokens, heads, width], tokens possibly over two axes.
void head_strides(const Tensor &t, int64_t tokens, const char *what, int64_t heads, int64_t width, at::ScalarType type,
                  int64_t (&out)[2])
{
    const int64_t dim = t.dim();
    bool ok = (dim == 3 || dim == 4) && t.scalar_type() == type && t.size(-2) == heads && t.size(-1) == width &&
              (t.stride(-1) == 1 || width == 1);
    if (ok && dim == 4) {
        const int64_t b = t.size(0), n = t.size(1);
        ok = b * n == tokens && (b <= 1 || n <= 1 || t.stride(0) == n * t.stride(1));
        out[0] = n > 1 ? t.stride(1) : t.stride(0);
    } else if (ok) {
        ok = t.size(0) == tokens;
        out[0] = t.stride(0);
    }
    if (!ok)
        refuse(what, ": shape ", t.sizes(), ", strides ", t.strides(), ", ", t.scalar_type(),
               " do not fit the other tensors");
    out[1] = t.stride(-2);
}

PyObject *status(conv_status st) { return PyLong_FromLong(st); }

PyObject *wrap(Tensor t) { return THPVariable_Wrap(std::move(t)); }

// x, weight, residual, eps, out_dtype, out, scale, sum_out -> (q, scale, h)
PyObject *rms_norm_q8(PyObject *const *a)
{
    const Tensor &x = tensor(a[0], "x"), &weight = tensor(a[1], "weight");
    const Tensor *residual = maybe(a[2], "residual"), *out = maybe(a[5], "out"), *scale = maybe(a[6], "scale"),
                 *sum = maybe(a[7], "sum_out");
    same_gpu(x, &weight, residual, out, scale, sum);
    const at::ScalarType type = x.scalar_type();
    const conv_dtype dt = float_code(type, "x");
    if (x.dim() < 1)
        refuse("x must have channels");
    const int64_t width = x.size(-1);
    if (width == 0)
        refuse("x must have channels");
    const int64_t rows = x.numel() / width;
    const int64_t xs = row_stride(x, "x", width, rows, type);
    const void *wp = vector(&weight, width, type, "weight");
    if (sum && !residual)
        refuse("sum_out without a residual");
    const at::ScalarType qtype = out ? out->scalar_type() : dtype_of(a[4], "out_dtype");
    const conv_dtype qdt = eight_code(qtype, "out_dtype");
    int64_t rs = 0, hs = 0, qs = width;
    if (residual)
        rs = row_stride(*residual, "residual", width, rows, type);
    if (sum)
        hs = row_stride(*sum, "sum_out", width, rows, type);
    if (out)
        qs = row_stride(*out, "out", width, rows, qtype);
    if (scale)
        vector(scale, rows, at::kFloat, "scale");
    const c10::DeviceGuard guard(x.device());
    Tensor h = sum ? *sum : Tensor();
    if (residual && !sum) {
        h = fresh(x, x.sizes(), type);
        hs = width;
    }
    Tensor q = out ? *out : fresh(x, x.sizes(), qtype);
    Tensor s = scale ? *scale : fresh(x, x.sizes().slice(0, x.dim() - 1), at::kFloat);
    const conv_status st = conv_rms_norm_q8_fwd(ptr(x), xs, ptr(residual), rs, wp, h.defined() ? h.data_ptr() : nullptr, hs,
                                                ptr(q), qs, static_cast<float *>(ptr(s)), rows, small(width, "a width"),
                                                (float)number(a[3]), dt, qdt, stream_of(x));
    if (st != CONV_OK)
        return status(st);
    PyObject *r = PyTuple_New(3);
    if (!r)
        throw python_error();
    PyTuple_SET_ITEM(r, 0, wrap(std::move(q)));
    PyTuple_SET_ITEM(r, 1, wrap(std::move(s)));
    if (h.defined()) {
        PyTuple_SET_ITEM(r, 2, wrap(std::move(h)));
    } else {
        Py_INCREF(Py_None);
        PyTuple_SET_ITEM(r, 2, Py_None);
    }
    return r;
}

// x, x_scale, w, w_scale, bias, out_dtype, out, variant -> y
PyObject *matmul_q8(PyObject *const *a)
{
    const Tensor &x = tensor(a[0], "x"), &xscale = tensor(a[1], "x_scale"), &w = tensor(a[2], "w"),
                 &wscale = tensor(a[3], "w_scale");
    const Tensor *bias = maybe(a[4], "bias"), *out = maybe(a[6], "out");
    same_gpu(x, &xscale, &w, &wscale, bias, out);
    const at::ScalarType type = x.scalar_type();
    const conv_dtype qdt = eight_code(type, "x");
    if (x.dim() < 1 || w.dim() != 2 || x.size(-1) == 0)
        refuse("expected x [..., K] and w [N, K], got ", x.sizes(), " and ", w.sizes());
    const int64_t K = x.size(-1), M = x.numel() / K, N = w.size(0);
    const int64_t xs = row_stride(x, "x", K, M, type), ws = row_stride(w, "w", K, N, type);
    const auto *sx = static_cast<const float *>(vector(&xscale, M, at::kFloat, "x_scale"));
    const auto *sw = static_cast<const float *>(vector(&wscale, N, at::kFloat, "w_scale"));
    const auto *b = static_cast<const float *>(vector(bias, N, at::kFloat, "bias"));
    const at::ScalarType ytype = out ? out->scalar_type() : dtype_of(a[5], "out_dtype");
    const conv_dtype ydt = float_code(ytype, "out_dtype");
    int64_t ys = N;
    if (out)
        ys = row_stride(*out, "out", N, M, ytype);
    const c10::DeviceGuard guard(x.device());
    Tensor y;
    if (out) {
        y = *out;
    } else {
        c10::SmallVector<int64_t, 5> sizes(x.sizes().begin(), x.sizes().end());
        sizes.back() = N;
        y = fresh(x, sizes, ytype);
    }
    const conv_status st = conv_matmul_q8_fwd(ptr(x), xs, sx, ptr(w), ws, sw, b, ptr(y), ys, M, small(N, "a channel count"),
                                              small(K, "a K"), qdt, ydt, (int)integer(a[7]), stream_of(x));
    return st != CONV_OK ? status(st) : wrap(std::move(y));
}

// x, w, bias, silu, seq_offsets, initial_state, final_state, slots, out -> y
PyObject *causal_conv1d(PyObject *const *a)
{
    const Tensor &x = tensor(a[0], "x"), &w = tensor(a[1], "w");
    const Tensor *bias = maybe(a[2], "bias"), *offsets = maybe(a[4], "seq_offsets"), *si = maybe(a[5], "initial_state"),
                 *so = maybe(a[6], "final_state"), *slots = maybe(a[7], "slots"), *out = maybe(a[8], "out");
    same_gpu(x, &w, bias, offsets, si, so, slots, out);
    const at::ScalarType type = x.scalar_type();
    const conv_dtype dt = float_code(type, "x");
    const Seqs seq = sequences(x, 1, offsets);
    const int64_t channels = x.size(-1);
    if (w.dim() != 2 || w.size(0) != channels || w.scalar_type() != type || !w.is_contiguous())
        refuse("w must be a contiguous [", channels, ", taps] tensor of ", type);
    const int64_t taps = w.size(1);
    const auto *b = static_cast<const float *>(vector(bias, channels, at::kFloat, "bias"));
    const int64_t shape[2] = {taps - 1, channels};
    const int64_t num = state(so, shape, type, state(si, shape, type, 0));
    const auto *sl = static_cast<const int32_t *>(vector(slots, seq.count, at::kInt, "slots"));
    const int64_t xs = row_stride(x, "x", channels, seq.tokens, type);
    const int64_t ys = out ? row_stride(*out, "out", channels, seq.tokens, type) : channels;
    const c10::DeviceGuard guard(x.device());
    Tensor y = out ? *out : fresh(x, x.sizes(), type);
    const conv_status st = conv_causal1d_fwd(ptr(x), xs, ptr(w), b, ptr(y), ys, static_cast<const int32_t *>(ptr(offsets)),
                                             ptr(si), ptr(so), sl, small(num, "a slot count"), seq.tokens, seq.count,
                                             small(channels, "a channel count"), small(taps, "a tap count"),
                                             (int)integer(a[3]), dt, stream_of(x));
    return st != CONV_OK ? status(st) : wrap(std::move(y));
}

// q, k, v, g, beta, scale, normalize, seq_offsets, initial_state, final_state, slots, out, workspace, variant -> o
PyObject *gated_delta_rule(PyObject *const *a)
{
    const Tensor &q = tensor(a[0], "q"), &k = tensor(a[1], "k"), &v = tensor(a[2], "v"), &g = tensor(a[3], "g"),
                 &beta = tensor(a[4], "beta");
    const Tensor *offsets = maybe(a[7], "seq_offsets"), *si = maybe(a[8], "initial_state"), *so = maybe(a[9], "final_state"),
                 *slots = maybe(a[10], "slots"), *out = maybe(a[11], "out"), *work = maybe(a[12], "workspace");
    same_gpu(q, &k, &v, &g, &beta, offsets, si, so, slots, out, work);
    const at::ScalarType type = q.scalar_type();
    const conv_dtype dt = float_code(type, "q");
    const Seqs seq = sequences(q, 2, offsets);
    if (v.dim() < 3)
        refuse("v must be [..., heads, channels], got ", v.sizes());
    const int64_t Hk = q.size(-2), Dk = q.size(-1), Hv = v.size(-2), Dv = v.size(-1);
    int64_t sq[2], sk[2], sv[2], st_o[2];
    head_strides(q, seq.tokens, "q", Hk, Dk, type, sq);
    head_strides(k, seq.tokens, "k", Hk, Dk, type, sk);
    head_strides(v, seq.tokens, "v", Hv, Dv, type, sv);
    const auto *gp = static_cast<const float *>(vector(&g, seq.tokens * Hv, at::kFloat, "g"));
    const auto *bp = static_cast<const float *>(vector(&beta, seq.tokens * Hv, at::kFloat, "beta"));
    const int64_t shape[3] = {Hv, Dk, Dv};
    const int64_t num = state(so, shape, at::kFloat, state(si, shape, at::kFloat, 0));
    const auto *sl = static_cast<const int32_t *>(vector(slots, seq.count, at::kInt, "slots"));
    if (out)
        head_strides(*out, seq.tokens, "out", Hv, Dv, type, st_o);
    const int hk = small(Hk, "a head count"), hv = small(Hv, "a head count"), dk = small(Dk, "a head's width"),
              dv = small(Dv, "a head's width"), variant = (int)integer(a[13]);
    const double scale = a[5] == Py_None ? 1.0 / std::sqrt((double)Dk) : number(a[5]);
    const c10::DeviceGuard guard(q.device());
    Tensor o = out ? *out : fresh(v, v.sizes(), type);
    Tensor space;
    int64_t bytes = 0;
    if (work) {
        bytes = work->numel();
        vector(work, bytes, at::kByte, "workspace");
    } else {
        bytes = conv_delta_rule_workspace(seq.tokens, seq.count, hk, hv, dk, dv, dt, variant);
        if (bytes > 0)
            space = fresh(q, {bytes}, at::kByte);
    }
    void *wp = work ? work->data_ptr() : (space.defined() ? space.data_ptr() : nullptr);
    const conv_status st = conv_delta_rule_fwd(
        ptr(q), sq, ptr(k), sk, ptr(v), sv, gp, bp, static_cast<const int32_t *>(ptr(offsets)),
        static_cast<const float *>(ptr(si)), static_cast<float *>(ptr(so)), sl, small(num, "a slot count"), ptr(o),
        out ? st_o : nullptr, wp, bytes, seq.tokens, seq.count, hk, hv, dk, dv, (float)scale, PyObject_IsTrue(a[6]), dt,
        variant, stream_of(q));
    return st != CONV_OK ? status(st) : wrap(std::move(o));
}

template <PyObject *(*F)(PyObject *const *), int N>
PyObject *entry(PyObject *, PyObject *const *args, Py_ssize_t n)
{
    HANDLE_TH_ERRORS
    if (n != N) {
        PyErr_Format(PyExc_TypeError, "expected %d arguments, got %zd", N, n);
        return nullptr;
    }
    try {
        return F(args);
    } catch (const ValueError &e) {
        PyErr_SetString(PyExc_ValueError, e.what.c_str());
        return nullptr;
    }
    END_HANDLE_TH_ERRORS
}

template <PyObject *(*F)(PyObject *const *), int N>
PyMethodDef method(const char *name)
{
    return {name, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(entry<F, N>)), METH_FASTCALL, nullptr};
}

PyMethodDef methods[] = {
    method<rms_norm_q8, 8>("rms_norm_q8"),
    method<matmul_q8, 8>("matmul_q8"),
    method<causal_conv1d, 9>("causal_conv1d"),
    method<gated_delta_rule, 14>("gated_delta_rule"),
    {nullptr, nullptr, 0, nullptr},
};

PyModuleDef module = {PyModuleDef_HEAD_INIT, "_mixer", "Token-mixer calls of libconvfwd on torch tensors.", -1, methods,
                      nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__mixer(void) { return PyModule_Create(&module); }
