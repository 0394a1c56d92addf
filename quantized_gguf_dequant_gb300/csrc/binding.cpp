// binding.cpp -- the Python calls of the decode-step operators.
//
// A decode step makes several calls of a few microseconds each, so what the
// host spends on one counts.  This module takes torch tensors apart, checks
// them, allocates what is to be returned and calls the C ABI (whose addresses
// the package hands over at load time); through ctypes and Python the same
// checks and allocations took twice as long.  It computes nothing.
#include <Python.h>

#include <ATen/core/Tensor.h>
#include <ATen/ops/empty.h>
#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/Dtype.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include "qmm.h"

namespace {

decltype(&qmm_kv_append) g_append;
decltype(&qmm_kv_read) g_read;
decltype(&qmm_attn_decode) g_attn;
decltype(&qmm_logits_adjust) g_logits;
decltype(&qmm_last_error) g_last_error;
PyObject *g_error;  // the package's QmmError

struct Cache {
    qmm_kv_t handle;
    int device;
    int64_t heads, D;
};

const char *const kCapsule = "qmm.cache";

#define FAIL(...)                                                                                 \
    do {                                                                                          \
        PyErr_Format(PyExc_ValueError, __VA_ARGS__);                                              \
        return false;                                                                             \
    } while (0)

std::string shape_of(at::IntArrayRef s)
{
    std::string out = "(";
    for (size_t i = 0; i < s.size(); ++i)
        out += (i ? ", " : "") + std::to_string(s[i]);
    return out + ")";
}

bool tensor(PyObject *o, const char *name, const at::Tensor *&t)
{
    if (!THPVariable_Check(o))
        FAIL("%s must be a tensor", name);
    t = &THPVariable_Unpack(o);
    return true;
}

// A plain type's id.
bool type_id(at::ScalarType s, int &id)
{
    switch (s) {
    case at::kFloat: id = QMM_F32; return true;
    case at::kHalf: id = QMM_F16; return true;
    case at::kBFloat16: id = QMM_BF16; return true;
    default:
        FAIL("%s is not supported (float32, float16 and bfloat16 are)", c10::toString(s));
    }
}

bool on_device(const at::Tensor &t, const char *name, int device)
{
    if (!t.is_cuda())
        FAIL("%s must live on the CUDA device", name);
    if (t.device().index() != device)
        FAIL("%s lives on device %d, the call is for device %d", name, int(t.device().index()),
             device);
    return true;
}

// A contiguous device tensor of a type and (n >= 0) of n elements; None gives null.
bool flat(PyObject *o, const char *name, at::ScalarType type, int64_t n, int device, void *&p)
{
    p = nullptr;
    if (o == Py_None)
        return true;
    const at::Tensor *t;
    if (!tensor(o, name, t))
        return false;
    if (t->scalar_type() != type)
        FAIL("%s must be %s, not %s", name, c10::toString(type), c10::toString(t->scalar_type()));
    if (!on_device(*t, name, device))
        return false;
    if (!t->is_contiguous())
        FAIL("%s must be contiguous", name);
    if (n >= 0 && t->numel() != n)
        FAIL("%s has %lld elements; %lld are needed", name, (long long)t->numel(), (long long)n);
    p = t->data_ptr();
    return true;
}

// Elements between the tokens of a [T, heads, D] tensor whose tokens may lie
// apart, such as a slice of a fused projection's output.
bool tokens(PyObject *o, const char *name, int64_t T, int64_t heads, int64_t D,
            at::ScalarType type, int device, void *&p, int64_t &ld)
{
    const at::Tensor *t;
    if (!tensor(o, name, t))
        return false;
    const at::IntArrayRef s = t->sizes();
    if (s.size() != 3 || s[0] != T || s[1] != heads || s[2] != D)
        FAIL("%s has shape %s; (%lld, %lld, %lld) is needed", name, shape_of(s).c_str(),
             (long long)T, (long long)heads, (long long)D);
    if (t->scalar_type() != type)
        FAIL("%s is %s; %s is needed", name, c10::toString(t->scalar_type()), c10::toString(type));
    if (!on_device(*t, name, device))
        return false;
    const at::IntArrayRef st = t->strides();
    if (st[2] != 1 || (heads > 1 && st[1] != D))
        FAIL("%s: the heads of a token must be contiguous", name);
    p = t->data_ptr();
    ld = T > 1 ? st[0] : heads * D;
    return true;
}

// None (the device's current stream), a stream object, or a raw handle.
bool stream_of(PyObject *o, int device, void *&s)
{
    if (o == Py_None) {
        s = c10::cuda::getCurrentCUDAStream(c10::DeviceIndex(device)).stream();
        return true;
    }
    PyObject *raw = o;
    if (PyLong_Check(o))
        Py_INCREF(raw);
    else if (!(raw = PyObject_GetAttrString(o, "cuda_stream")))
        return false;
    s = PyLong_AsVoidPtr(raw);
    Py_DECREF(raw);
    return !PyErr_Occurred();
}

// A new output.  For work on a stream that is not the current one its memory
// is that stream's (what the current stream still does with memory given back
// is no concern of it), and is not given out again before the current stream,
// which is likely to read it, has passed the point where it is dropped.
PyObject *output(at::IntArrayRef shape, at::ScalarType type, int device, void *stream, void *&p)
{
    const auto options =
        at::TensorOptions().dtype(type).device(at::Device(at::kCUDA, c10::DeviceIndex(device)));
    const c10::cuda::CUDAStream current =
        c10::cuda::getCurrentCUDAStream(c10::DeviceIndex(device));
    at::Tensor t;
    if (current.stream() == stream) {
        t = at::empty(shape, options);
    } else {
        c10::cuda::CUDAStreamGuard on(c10::cuda::getStreamFromExternal(
            static_cast<cudaStream_t>(stream), c10::DeviceIndex(device)));
        t = at::empty(shape, options);
        t.record_stream(current.unwrap());
    }
    p = t.data_ptr();
    return THPVariable_Wrap(std::move(t));
}

// What a call on a stream that is not the current one reads or writes: memory
// that the caller drops is not given out again before that stream is done.
// named: the call's stream argument.
void used_on(PyObject *named, void *stream, int device, std::initializer_list<PyObject *> given)
{
    if (named == Py_None ||
        c10::cuda::getCurrentCUDAStream(c10::DeviceIndex(device)).stream() == stream)
        return;
    const c10::Stream on = c10::cuda::getStreamFromExternal(static_cast<cudaStream_t>(stream),
                                                            c10::DeviceIndex(device))
                               .unwrap();
    for (PyObject *o : given)
        if (o && THPVariable_Check(o) && THPVariable_Unpack(o).numel() > 0)
            THPVariable_Unpack(o).record_stream(on);
}

bool ok(qmm_status rc)
{
    if (rc == QMM_OK)
        return true;
    if (PyObject *e = PyObject_CallFunction(g_error, "is", int(rc), g_last_error())) {
        PyErr_SetObject(g_error, e);
        Py_DECREF(e);
    }
    return false;
}

Cache *cache_of(PyObject *o) { return static_cast<Cache *>(PyCapsule_GetPointer(o, kCapsule)); }

bool count(Py_ssize_t n, Py_ssize_t want)
{
    if (n != want)
        FAIL("%zd arguments; %zd are needed", n, want);
    return true;
}

// A reference that is given up unless it is returned.
struct Held {
    PyObject *o = nullptr;
    ~Held() { Py_XDECREF(o); }
    PyObject *release()
    {
        PyObject *r = o;
        o = nullptr;
        return r;
    }
    // the caller's object, or the new one
    void borrow(PyObject *other)
    {
        Py_INCREF(other);
        o = other;
    }
};

// (cache, k, v, slots, q, pos, rope, q_out, stream) -> rotated q or None
PyObject *append(PyObject *, PyObject *const *a, Py_ssize_t n)
{
    HANDLE_TH_ERRORS
    if (!count(n, 9))
        return nullptr;
    Cache *c = cache_of(a[0]);
    const at::Tensor *k;
    if (!c || !tensor(a[1], "k", k))
        return nullptr;
    const at::ScalarType type = k->scalar_type();
    const int64_t T = k->dim() ? k->size(0) : 0;
    int id;
    void *kp, *vp, *sp, *qp = nullptr, *op = nullptr, *pp = nullptr, *stream;
    int64_t ldk, ldv, ldq = 0, ldo = 0, heads = 0;
    if (!type_id(type, id) || !tokens(a[1], "k", T, c->heads, c->D, type, c->device, kp, ldk) ||
        !tokens(a[2], "v", T, c->heads, c->D, type, c->device, vp, ldv) ||
        !flat(a[3], "slots", at::kLong, T, c->device, sp) || !stream_of(a[8], c->device, stream))
        return nullptr;
    Held out;
    if (a[4] != Py_None) {
        const at::Tensor *q;
        if (!tensor(a[4], "q", q))
            return nullptr;
        heads = q->dim() > 1 ? q->size(1) : 0;
        if (!tokens(a[4], "q", T, heads, c->D, type, c->device, qp, ldq))
            return nullptr;
        if (a[7] != Py_None) {
            if (!tokens(a[7], "q_out", T, heads, c->D, type, c->device, op, ldo))
                return nullptr;
            out.borrow(a[7]);
        } else {
            if (!(out.o = output({T, heads, c->D}, type, c->device, stream, op)))
                return nullptr;
            ldo = heads * c->D;
        }
    }
    const qmm_rope *rope = nullptr;
    Held inv_freq;
    if (a[6] != Py_None) {
        PyObject *at = PyObject_GetAttrString(a[6], "address");
        if (!at)
            return nullptr;
        rope = static_cast<const qmm_rope *>(PyLong_AsVoidPtr(at));
        Py_DECREF(at);
        if (!rope || !(at = PyObject_GetAttrString(a[6], "device")))
            return nullptr;
        const long device = PyLong_AsLong(at);
        Py_DECREF(at);
        if (PyErr_Occurred())
            return nullptr;
        if (device != c->device) {
            PyErr_Format(PyExc_ValueError, "rope's inv_freq lives on device %ld, the call is for "
                         "device %d", device, c->device);
            return nullptr;
        }
        if (a[8] != Py_None && !(inv_freq.o = PyObject_GetAttrString(a[6], "inv_freq")))
            return nullptr;
        if (!flat(a[5], "pos", at::kInt, rope->n_axes * T, c->device, pp))
            return nullptr;
        // [T, axes] has as many elements and would turn tokens by others' positions
        if (pp && rope->n_axes > 1) {
            const at::IntArrayRef s = THPVariable_Unpack(a[5]).sizes();
            if (s.size() != 2 || s[0] != rope->n_axes || s[1] != T) {
                PyErr_Format(PyExc_ValueError, "pos has shape %s; (%d, %lld) is needed",
                             shape_of(s).c_str(), int(rope->n_axes), (long long)T);
                return nullptr;
            }
        }
    }
    qmm_status rc;
    Py_BEGIN_ALLOW_THREADS
    rc = g_append(c->handle, id, T, kp, ldk, vp, ldv, static_cast<const int64_t *>(sp), qp, ldq,
                  int32_t(heads), op, ldo, static_cast<const int32_t *>(pp), rope, stream);
    Py_END_ALLOW_THREADS
    if (!ok(rc))
        return nullptr;
    used_on(a[8], stream, c->device, {a[1], a[2], a[3], a[4], a[5], a[7], inv_freq.o});
    if (out.o)
        return out.release();
    Py_RETURN_NONE;
    END_HANDLE_TH_ERRORS
}

// (cache, q, page_table, lens, scale, softcap, window, alibi, out, lse, return_lse, stream)
// -> out, or (out, lse)
PyObject *attend(PyObject *, PyObject *const *a, Py_ssize_t n)
{
    HANDLE_TH_ERRORS
    if (!count(n, 12))
        return nullptr;
    Cache *c = cache_of(a[0]);
    const at::Tensor *q, *table;
    if (!c || !tensor(a[1], "q", q) || !tensor(a[2], "page_table", table))
        return nullptr;
    const at::ScalarType type = q->scalar_type();
    const int64_t B = q->dim() ? q->size(0) : 0, heads = q->dim() > 1 ? q->size(1) : 0;
    int id;
    void *qp, *op, *lp = nullptr, *np, *ap, *stream;
    int64_t ldq, ldo = heads * c->D;
    if (!type_id(type, id) || !tokens(a[1], "q", B, heads, c->D, type, c->device, qp, ldq) ||
        !flat(a[3], "lens", at::kInt, B, c->device, np) ||
        !flat(a[7], "alibi", at::kFloat, heads, c->device, ap) ||
        !stream_of(a[11], c->device, stream))
        return nullptr;
    if (table->dim() != 2 || table->size(0) != B || table->scalar_type() != at::kInt ||
        !table->is_contiguous()) {
        PyErr_Format(PyExc_ValueError, "page_table must be a contiguous int32 tensor of [%lld, pages]",
                     (long long)B);
        return nullptr;
    }
    if (!on_device(*table, "page_table", c->device))
        return nullptr;
    qmm_attn o;
    o.scale = a[4] == Py_None ? float(1.0 / std::sqrt(double(c->D))) : float(PyFloat_AsDouble(a[4]));
    o.softcap = float(PyFloat_AsDouble(a[5]));
    const long window = PyLong_AsLong(a[6]);
    if (PyErr_Occurred())
        return nullptr;
    o.window = int32_t(std::max(-1l, std::min(window, 0x7fffffffl)));
    o.alibi = static_cast<const float *>(ap);
    const int want = PyObject_IsTrue(a[10]);
    if (want < 0)
        return nullptr;
    Held out, lse;
    if (a[8] != Py_None) {
        if (!tokens(a[8], "out", B, heads, c->D, type, c->device, op, ldo))
            return nullptr;
        out.borrow(a[8]);
    } else if (!(out.o = output({B, heads, c->D}, type, c->device, stream, op))) {
        return nullptr;
    }
    if (a[9] != Py_None) {
        if (!flat(a[9], "lse", at::kFloat, B * heads, c->device, lp))
            return nullptr;
        lse.borrow(a[9]);
    } else if (want && !(lse.o = output({B, heads}, at::kFloat, c->device, stream, lp))) {
        return nullptr;
    }
    const int64_t ld_table = table->size(1);
    const int32_t *tp = static_cast<const int32_t *>(table->data_ptr());
    qmm_status rc;
    Py_BEGIN_ALLOW_THREADS
    rc = g_attn(c->handle, id, B, int32_t(std::min<int64_t>(heads, 0x7fffffff)), qp, ldq, tp,
                ld_table, static_cast<const int32_t *>(np), &o, op, ldo, static_cast<float *>(lp),
                stream);
    Py_END_ALLOW_THREADS
    if (!ok(rc))
        return nullptr;
    used_on(a[11], stream, c->device, {a[1], a[2], a[3], a[7], a[8], a[9]});
    return want ? PyTuple_Pack(2, out.o, lse.o) : out.release();
    END_HANDLE_TH_ERRORS
}

// (cache, slots, dtype, k_out, v_out, stream) -> (k, v)
PyObject *read(PyObject *, PyObject *const *a, Py_ssize_t n)
{
    HANDLE_TH_ERRORS
    if (!count(n, 6))
        return nullptr;
    Cache *c = cache_of(a[0]);
    const at::Tensor *slots;
    if (!c || !tensor(a[1], "slots", slots))
        return nullptr;
    at::ScalarType type = at::kFloat;
    if (a[2] != Py_None) {
        if (!THPDtype_Check(a[2])) {
            PyErr_SetString(PyExc_ValueError, "dtype must be a torch dtype");
            return nullptr;
        }
        type = reinterpret_cast<THPDtype *>(a[2])->scalar_type;
    } else if (THPVariable_Check(a[3])) {
        type = THPVariable_Unpack(a[3]).scalar_type();
    } else if (THPVariable_Check(a[4])) {
        type = THPVariable_Unpack(a[4]).scalar_type();
    }
    const int64_t T = slots->numel();
    int id;
    void *sp, *p[2], *stream;
    int64_t ld[2];
    if (!type_id(type, id) || !flat(a[1], "slots", at::kLong, -1, c->device, sp) ||
        !stream_of(a[5], c->device, stream))
        return nullptr;
    Held out[2];
    for (int w = 0; w < 2; ++w) {
        if (a[3 + w] != Py_None) {
            if (!tokens(a[3 + w], w ? "v_out" : "k_out", T, c->heads, c->D, type, c->device, p[w],
                        ld[w]))
                return nullptr;
            out[w].borrow(a[3 + w]);
        } else {
            if (!(out[w].o = output({T, c->heads, c->D}, type, c->device, stream, p[w])))
                return nullptr;
            ld[w] = c->heads * c->D;
        }
    }
    qmm_status rc;
    Py_BEGIN_ALLOW_THREADS
    rc = g_read(c->handle, id, T, static_cast<const int64_t *>(sp), p[0], ld[0], p[1], ld[1],
                stream);
    Py_END_ALLOW_THREADS
    if (!ok(rc))
        return nullptr;
    used_on(a[5], stream, c->device, {a[1], a[3], a[4]});
    return PyTuple_Pack(2, out[0].o, out[1].o);
    END_HANDLE_TH_ERRORS
}

// (logits, out, history, history_offsets, repeat, presence, frequency, bias_ids, bias_values,
//  bias_offsets, mask, stream) -> out
PyObject *logits(PyObject *, PyObject *const *a, Py_ssize_t n)
{
    HANDLE_TH_ERRORS
    if (!count(n, 12))
        return nullptr;
    const at::Tensor *z;
    if (!tensor(a[0], "logits", z))
        return nullptr;
    const at::ScalarType type = z->scalar_type();
    const at::IntArrayRef shape = z->sizes();
    int id;
    if (!type_id(type, id))
        return nullptr;
    if ((shape.size() != 1 && shape.size() != 2) || !z->is_cuda() ||
        (shape.back() > 1 && z->strides().back() != 1)) {
        PyErr_SetString(PyExc_ValueError, "logits must be [rows, vocabulary] or [vocabulary] on the "
                                          "CUDA device, each row contiguous");
        return nullptr;
    }
    const int device = z->device().index();
    // The C entry launches on the current device, whatever the pointers say.
    // (A cache's calls are held to its device by the entry.)
    c10::DeviceIndex current = -1;
    if (c10::cuda::GetDevice(&current) != cudaSuccess || device != current) {
        PyErr_Format(PyExc_ValueError, "logits live on device %d, but device %d is current", device,
                     int(current));
        return nullptr;
    }
    const int64_t B = shape.size() == 2 ? shape[0] : 1, V = shape.back();
    int64_t ld = V, ldo = V;
    if (B > 1)
        ld = z->stride(0);
    void *stream, *op;
    if (!stream_of(a[11], device, stream))
        return nullptr;
    Held out;
    if (a[1] != Py_None) {
        const at::Tensor *o;
        if (!tensor(a[1], "out", o))
            return nullptr;
        if (o->sizes() != shape || o->scalar_type() != type || !o->is_cuda() ||
            o->device().index() != device || (V > 1 && o->strides().back() != 1)) {
            PyErr_SetString(PyExc_ValueError, "out must be like logits");
            return nullptr;
        }
        if (B > 1)
            ldo = o->stride(0);
        op = o->data_ptr();
        out.borrow(a[1]);
    } else if (!(out.o = output(shape, type, device, stream, op))) {
        return nullptr;
    }
    qmm_logit_rules r = {};
    void *p[9];
    const at::Tensor *list;
    if (a[2] != Py_None) {
        if (!tensor(a[2], "history", list))
            return nullptr;
        r.n_history = list->numel();
    }
    if (a[7] != Py_None) {
        if (!tensor(a[7], "bias_ids", list))
            return nullptr;
        r.n_biases = list->numel();
    }
    const int64_t rows = r.n_history ? B + 1 : -1, brows = r.n_biases ? B + 1 : -1;
    if (!flat(a[2], "history", at::kInt, -1, device, p[0]) ||
        !flat(a[3], "history_offsets", at::kLong, rows, device, p[1]) ||
        !flat(a[4], "repeat", at::kFloat, B, device, p[2]) ||
        !flat(a[5], "presence", at::kFloat, B, device, p[3]) ||
        !flat(a[6], "frequency", at::kFloat, B, device, p[4]) ||
        !flat(a[7], "bias_ids", at::kInt, -1, device, p[5]) ||
        !flat(a[8], "bias_values", at::kFloat, r.n_biases ? r.n_biases : -1, device, p[6]) ||
        !flat(a[9], "bias_offsets", at::kLong, brows, device, p[7]) ||
        !flat(a[10], "mask", at::kInt, -1, device, p[8]))
        return nullptr;
    if (a[10] != Py_None) {
        const at::Tensor &m = THPVariable_Unpack(a[10]);
        const int64_t words = m.dim() ? m.sizes().back() : 0;
        if (words * 32 < V || (m.numel() != words && m.numel() != B * words)) {
            PyErr_Format(PyExc_ValueError, "mask of shape %s does not hold %lld or 1 rows of %lld "
                         "bits", shape_of(m.sizes()).c_str(), (long long)B, (long long)V);
            return nullptr;
        }
        r.ld_mask = m.numel() == B * words ? words : 0;
    }
    r.history = static_cast<const int32_t *>(p[0]);
    r.history_offsets = static_cast<const int64_t *>(p[1]);
    r.repeat = static_cast<const float *>(p[2]);
    r.presence = static_cast<const float *>(p[3]);
    r.frequency = static_cast<const float *>(p[4]);
    r.bias_ids = static_cast<const int32_t *>(p[5]);
    r.bias_values = static_cast<const float *>(p[6]);
    r.bias_offsets = static_cast<const int64_t *>(p[7]);
    r.mask = static_cast<const uint32_t *>(p[8]);
    const void *zp = z->data_ptr();
    qmm_status rc;
    Py_BEGIN_ALLOW_THREADS
    rc = g_logits(id, B, V, zp, ld, &r, op, ldo, stream);
    Py_END_ALLOW_THREADS
    if (!ok(rc))
        return nullptr;
    used_on(a[11], stream, device, {a[0], a[1], a[2], a[3], a[4], a[5], a[6], a[7], a[8], a[9], a[10]});
    return out.release();
    END_HANDLE_TH_ERRORS
}

// (handle, device, heads, head_dim) -> what the other calls take as the cache
PyObject *cache(PyObject *, PyObject *args)
{
    unsigned long long h;
    int device;
    long long heads, D;
    if (!PyArg_ParseTuple(args, "KiLL", &h, &device, &heads, &D))
        return nullptr;
    Cache *c = new (std::nothrow) Cache{reinterpret_cast<qmm_kv_t>(h), device, heads, D};
    if (!c)
        return PyErr_NoMemory();
    return PyCapsule_New(c, kCapsule, [](PyObject *o) {
        delete static_cast<Cache *>(PyCapsule_GetPointer(o, kCapsule));
    });
}

// (QmmError, addresses of qmm_kv_append, qmm_kv_read, qmm_attn_decode, qmm_logits_adjust,
//  qmm_last_error)
PyObject *init(PyObject *, PyObject *args)
{
    PyObject *error;
    unsigned long long f[5];
    if (!PyArg_ParseTuple(args, "OKKKKK", &error, f, f + 1, f + 2, f + 3, f + 4))
        return nullptr;
    Py_INCREF(error);
    Py_XSETREF(g_error, error);
    g_append = reinterpret_cast<decltype(g_append)>(f[0]);
    g_read = reinterpret_cast<decltype(g_read)>(f[1]);
    g_attn = reinterpret_cast<decltype(g_attn)>(f[2]);
    g_logits = reinterpret_cast<decltype(g_logits)>(f[3]);
    g_last_error = reinterpret_cast<decltype(g_last_error)>(f[4]);
    Py_RETURN_NONE;
}

template <typename F>
PyCFunction fast(F f)
{
    return reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(f));
}

PyMethodDef methods[] = {{"init", init, METH_VARARGS, nullptr},
                         {"cache", cache, METH_VARARGS, nullptr},
                         {"append", fast(append), METH_FASTCALL, nullptr},
                         {"attend", fast(attend), METH_FASTCALL, nullptr},
                         {"read", fast(read), METH_FASTCALL, nullptr},
                         {"logits", fast(logits), METH_FASTCALL, nullptr},
                         {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_native", nullptr, -1, methods};

} // namespace

extern "C" __attribute__((visibility("default"))) PyObject *PyInit__native(void)
{
    return PyModule_Create(&module);
}
