// binding.cpp -- the Python calls of the operators around the GEMVs of a decode
// step: tensors are checked here and become the structs of include/mq.h.  In C++
// because a call names up to 14 tensors: with few rows the call is what an eager
// step waits for.  Back to back, one row: rotation and append 9.4 us with the
// checks in Python, 2.9 so, of which 2.7 are the C call with its launch; attention
// 7.3 and 4.1.
// The module is used by __init__.py alone, which has the documented functions.
#include <torch/csrc/autograd/python_variable.h>

#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAStream.h>

#include <climits>

#include "mq.h"

namespace {

// Set by setup(): the library's entry points (of the libmq.so that ctypes has loaded), MQError, and
// the function that raises for a tensor that does not fit.
struct {
    decltype(&mq_rope_append) rope_append;
    decltype(&mq_attn_decode) attn_decode;
    decltype(&mq_sample) sample;
    decltype(&mq_q8_bytes) q8_bytes;
    decltype(&mq_add_rmsnorm_quant_q8) add_rmsnorm;
    decltype(&mq_kv_assign) kv_assign;
    decltype(&mq_verify) verify;
    PyObject *error, *bad_tensor;
} g;

constexpr at::ScalarType kF32 = at::kFloat, kI32 = at::kInt, kI64 = at::kLong, kU8 = at::kByte;

bool fail(int status, const char *where)
{
    if (PyObject *args = Py_BuildValue("(is)", status, where)) {
        PyErr_SetObject(g.error, args);
        Py_DECREF(args);
    }
    return false;
}

bool bad_tensor(PyObject *t, const char *what, at::ScalarType type, int device, bool shape, const char *expected,
                long long a, long long b = 0)
{
    char text[96];
    snprintf(text, sizeof text, expected, a, b);
    const char *name = type == kF32 ? "float32" : type == kI32 ? "int32" : type == kI64 ? "int64" : "uint8";
    PyObject *r = PyObject_CallFunction(g.bad_tensor, "Ossisi", t, text, name, device, what, shape ? 1 : 0);
    Py_XDECREF(r);
    if (!PyErr_Occurred()) PyErr_SetString(PyExc_TypeError, what);
    return false;
}

// The tensor of an object on cuda:device; null, with an exception, if it is none of that type.
const at::Tensor *tensor(PyObject *o, const char *what, at::ScalarType type, int device)
{
    if (!THPVariable_Check(o)) {
        PyErr_Format(PyExc_TypeError, "%s: expected a tensor, got %s", what, Py_TYPE(o)->tp_name);
        return nullptr;
    }
    const at::Tensor &t = THPVariable_Unpack(o);
    if (t.scalar_type() != type || !t.is_cuda() || t.get_device() != device || t.layout() != at::kStrided) {
        bad_tensor(o, what, type, device, false, "", 0);
        return nullptr;
    }
    return &t;
}

// An f32 [nt, cols] tensor whose rows are contiguous: its address and row stride.
template <class P>
bool rows(PyObject *o, const char *what, long long nt, long long cols, int device, P **ptr, long long *stride)
{
    const at::Tensor *t = tensor(o, what, kF32, device);
    if (!t) return false;
    const bool shape = t->dim() == 2 && t->size(0) == nt && t->size(1) == cols;
    const bool dense = shape && t->is_contiguous();
    if (!shape || (!dense && cols > 1 && t->stride(1) != 1))
        return bad_tensor(o, what, kF32, device, true, "[%lld, %lld] with contiguous rows", nt, cols);
    *ptr = static_cast<P *>(t->data_ptr());
    *stride = dense ? cols : t->stride(0);
    return true;
}

// A contiguous tensor of n values (n < 0: of any number); null for None.
template <class P>
bool vec(PyObject *o, const char *what, at::ScalarType type, long long n, int device, P **ptr,
         long long *numel = nullptr)
{
    *ptr = nullptr;
    if (numel) *numel = 0;
    if (o == Py_None) return true;
    const at::Tensor *t = tensor(o, what, type, device);
    if (!t) return false;
    if ((n >= 0 && t->numel() != n) || !t->is_contiguous())
        return n >= 0 ? bad_tensor(o, what, type, device, true, "%lld contiguous values", n)
                      : bad_tensor(o, what, type, device, true, "contiguous values", 0);
    *ptr = static_cast<P *>(t->data_ptr());
    if (numel) *numel = t->numel();
    return true;
}

// The page tables of nt rows.
bool page_table(PyObject *o, PyObject *seq, long long nt, int device, const int **ptr, int *n_seqs, int *per_seq)
{
    const at::Tensor *t = tensor(o, "pages", kI32, device);
    if (!t) return false;
    if (t->dim() != 2 || !t->is_contiguous() || t->size(0) > INT_MAX || t->size(1) > INT_MAX)
        return bad_tensor(o, "pages", kI32, device, true, "contiguous [sequences, pages per sequence]", 0);
    if (seq == Py_None && t->size(0) < nt) {
        PyErr_Format(PyExc_ValueError, "pages: %lld rows but %lld sequences", nt, (long long)t->size(0));
        return false;
    }
    *ptr = static_cast<const int *>(t->data_ptr());
    *n_seqs = (int)t->size(0), *per_seq = (int)t->size(1);
    return true;
}

// Rows and columns of the tensor that a call's shapes follow.
bool shape_of(PyObject *o, const char *what, const char *where, int *nt, long long *cols)
{
    if (!THPVariable_Check(o) || THPVariable_Unpack(o).dim() != 2) {
        PyErr_Format(PyExc_TypeError, "%s: expected a tensor of two dimensions", what);
        return false;
    }
    const at::Tensor &t = THPVariable_Unpack(o);
    if (t.size(0) > INT_MAX || t.size(1) > INT_MAX) return fail(MQ_ERR_SHAPE, where);
    *nt = (int)t.size(0), *cols = t.size(1);
    return true;
}

// Query heads of a row of `cols` values.
bool heads_of(long long cols, int head_dim, int *heads)
{
    if (cols % head_dim != 0) {
        PyErr_Format(PyExc_ValueError, "q: %lld columns are no whole heads of %d", cols, head_dim);
        return false;
    }
    *heads = (int)(cols / head_dim);
    return true;
}

// The stream of a launch on cuda:device, which must be the current device: a handle, or None for the
// current stream.
bool launch_stream(PyObject *s, int device, void **stream)
{
    if (c10::cuda::current_device() != device) {
        PyErr_Format(PyExc_ValueError, "the tensors are on cuda:%d, which is not the current device", device);
        return false;
    }
    *stream = s == Py_None ? c10::cuda::getCurrentCUDAStream((c10::DeviceIndex)device).stream() : PyLong_AsVoidPtr(s);
    return !PyErr_Occurred();
}

// A Python integer as a C one; beyond it: MQ_ERR_SHAPE.
bool integer(PyObject *o, const char *where, int *v)
{
    int over = 0;
    const long long x = PyLong_AsLongLongAndOverflow(o, &over);
    if (PyErr_Occurred()) return false;
    if (over || x > INT_MAX || x < INT_MIN) return fail(MQ_ERR_SHAPE, where);
    *v = (int)x;
    return true;
}

bool number(PyObject *o, float *v)
{
    *v = (float)PyFloat_AsDouble(o);
    return !PyErr_Occurred();
}

// The call without the interpreter's lock, and its error.
template <class F>
PyObject *launch(const char *where, PyObject *result, F &&call)
{
    int st;
    Py_BEGIN_ALLOW_THREADS
    st = call();
    Py_END_ALLOW_THREADS
    if (st != MQ_OK) {
        fail(st, where);
        return nullptr;
    }
    return Py_NewRef(result);
}

bool count_ok(const char *where, Py_ssize_t n, Py_ssize_t want)
{
    if (n == want) return true;
    PyErr_Format(PyExc_TypeError, "%s: %zd arguments, not %zd", where, n, want);
    return false;
}

// kv, device, q, k, v, positions, pages, q_out, rope, style, q_bias, k_bias, v_bias, q_gain, k_gain, eps,
// seq, status, stream
PyObject *rope_append(PyObject *const *a, Py_ssize_t n)
{
    static const char *where = "mq_rope_append";
    if (!count_ok(where, n, 19)) return nullptr;
    const auto *kv = static_cast<const mq_kv_cache *>(PyLong_AsVoidPtr(a[0]));
    int dev;
    if (!kv || !integer(a[1], where, &dev)) return nullptr;
    const int D = kv->head_dim;
    const long long nk = (long long)kv->n_kv_heads * D;
    mq_rope_append_args r = {};
    void *stream;
    long long nq, half;
    if (!launch_stream(a[18], dev, &stream) || !shape_of(a[2], "q", where, &r.nt, &nq) ||
        !page_table(a[6], a[16], r.nt, dev, &r.pages, &r.n_seqs, &r.pages_stride) || !heads_of(nq, D, &r.n_heads) ||
        !rows(a[2], "q", r.nt, nq, dev, &r.q, &r.q_stride) || !rows(a[3], "k", r.nt, nk, dev, &r.k, &r.k_stride) ||
        !rows(a[4], "v", r.nt, nk, dev, &r.v, &r.v_stride) ||
        !rows(a[7], "q_out", r.nt, nq, dev, &r.q_out, &r.q_out_stride) ||
        !vec(a[5], "positions", kI32, r.nt, dev, &r.positions) ||
        !vec(a[8], "rope", kI64, -1, dev, &r.rope_table, &half) || !integer(a[9], where, &r.rope_style) ||
        !vec(a[10], "q_bias", kF32, nq, dev, &r.q_bias) || !vec(a[11], "k_bias", kF32, nk, dev, &r.k_bias) ||
        !vec(a[12], "v_bias", kF32, nk, dev, &r.v_bias) || !vec(a[13], "q_gain", kF32, D, dev, &r.q_gain) ||
        !vec(a[14], "k_gain", kF32, D, dev, &r.k_gain) || !number(a[15], &r.eps) ||
        !vec(a[16], "seq", kI32, r.nt, dev, &r.seq) || !vec(a[17], "status", kI32, 1, dev, &r.status))
        return nullptr;
    r.rope_dims = (int)(half > D ? D + 1 : 2 * half);  // more than a head has: refused as one too many
    return launch(where, a[7], [&] { return g.rope_append(kv, &r, stream); });
}

// kv, device, q, lens, pages, scale, out, q8, ws, softcap, window, max_len, seq, status, stream
PyObject *attn_decode(PyObject *const *a, Py_ssize_t n)
{
    static const char *where = "mq_attn_decode";
    if (!count_ok(where, n, 15)) return nullptr;
    const auto *kv = static_cast<const mq_kv_cache *>(PyLong_AsVoidPtr(a[0]));
    int dev;
    if (!kv || !integer(a[1], where, &dev)) return nullptr;
    mq_attn_args r = {};
    void *stream;
    long long nq, q8_n, ws_n;
    uint8_t *q8, *ws;
    if (!launch_stream(a[14], dev, &stream) || !shape_of(a[2], "q", where, &r.nt, &nq) ||
        !page_table(a[4], a[12], r.nt, dev, &r.pages, &r.n_seqs, &r.pages_stride) ||
        !heads_of(nq, kv->head_dim, &r.n_heads) || !rows(a[2], "q", r.nt, nq, dev, &r.q, &r.q_stride) ||
        !vec(a[3], "lens", kI32, r.nt, dev, &r.lens) || !number(a[5], &r.scale) ||
        !rows(a[6], "out", r.nt, nq, dev, &r.out, &r.out_stride) ||
        !vec(a[7], "q8", kU8, -1, dev, &q8, &q8_n) || !vec(a[8], "ws", kU8, -1, dev, &ws, &ws_n) ||
        !number(a[9], &r.softcap) || !integer(a[10], where, &r.window) ||
        !vec(a[12], "seq", kI32, r.nt, dev, &r.seq) || !vec(a[13], "status", kI32, 1, dev, &r.status))
        return nullptr;
    if (a[11] == Py_None) {
        const long long all = (long long)r.pages_stride * kv->page_size;
        if (all > MQ_ATTN_MAX_LEN) {
            fail(MQ_ERR_SHAPE, where);
            return nullptr;
        }
        r.max_len = (int)all;
    } else if (!integer(a[11], where, &r.max_len)) {
        return nullptr;
    }
    if (a[7] != Py_None && q8_n < r.nt * (long long)g.q8_bytes((int)nq)) {
        PyErr_Format(PyExc_ValueError, "q8: smaller than %d planes of %lld values", r.nt, nq);
        return nullptr;
    }
    r.q8 = q8, r.ws = ws, r.ws_bytes = (size_t)ws_n;
    return launch(where, a[6], [&] { return g.attn_decode(kv, &r, stream); });
}

// logits, u, temperature, top_k, top_p, min_p, token, prob, stream
PyObject *sample(PyObject *const *a, Py_ssize_t n)
{
    static const char *where = "mq_sample";
    if (!count_ok(where, n, 9)) return nullptr;
    mq_sample_args r = {};
    void *stream;
    long long vocab;
    if (!shape_of(a[0], "logits", where, &r.nt, &vocab)) return nullptr;
    const at::Tensor &logits = THPVariable_Unpack(a[0]);
    if (!logits.is_cuda()) {
        PyErr_SetString(PyExc_TypeError, "logits: expected a CUDA tensor (the library has no CPU path)");
        return nullptr;
    }
    const int dev = (int)logits.get_device();
    r.vocab = (int)vocab;
    if (!launch_stream(a[8], dev, &stream) || !rows(a[0], "logits", r.nt, vocab, dev, &r.logits, &r.stride) ||
        !vec(a[1], "u", kF32, r.nt, dev, &r.u) || !vec(a[2], "temperature", kF32, r.nt, dev, &r.temperature) ||
        !vec(a[3], "top_k", kI32, r.nt, dev, &r.top_k) || !vec(a[4], "top_p", kF32, r.nt, dev, &r.top_p) ||
        !vec(a[5], "min_p", kF32, r.nt, dev, &r.min_p) || !vec(a[6], "token", kI32, r.nt, dev, &r.token) ||
        !vec(a[7], "prob", kF32, r.nt, dev, &r.prob))
        return nullptr;
    return launch(where, a[6], [&] { return g.sample(&r, stream); });
}

// A contiguous f32 tensor of nt rows of n values (one row: of one dimension too).
template <class P>
bool dense(PyObject *o, const char *what, long long nt, long long n, int device, P **ptr)
{
    const at::Tensor *t = tensor(o, what, kF32, device);
    if (!t) return false;
    const bool shape = t->dim() == 2 ? t->size(0) == nt && t->size(1) == n : t->dim() == 1 && nt == 1 && t->size(0) == n;
    if (!shape || !t->is_contiguous()) return bad_tensor(o, what, kF32, device, true, "contiguous [%lld, %lld]", nt, n);
    *ptr = static_cast<P *>(t->data_ptr());
    return true;
}

// The device of the tensor that a call's other tensors follow.
bool device_of(PyObject *o, const char *what, int *device)
{
    if (!THPVariable_Check(o) || !THPVariable_Unpack(o).is_cuda()) {
        PyErr_Format(PyExc_TypeError, "%s: expected a CUDA tensor (the library has no CPU path)", what);
        return false;
    }
    *device = (int)THPVariable_Unpack(o).get_device();
    return true;
}

// x, y, gain, eps, post_gain, gate, scale, x_out, z, q8, stream
PyObject *add_rmsnorm(PyObject *const *a, Py_ssize_t n)
{
    static const char *where = "mq_add_rmsnorm_quant_q8";
    int dev;
    if (!count_ok(where, n, 11) || !device_of(a[0], "x", &dev)) return nullptr;
    const at::Tensor &x = THPVariable_Unpack(a[0]);
    const long long nt = x.dim() == 2 ? x.size(0) : 1, cols = x.dim() > 0 ? x.size(x.dim() - 1) : 0;
    if (nt > INT_MAX || cols > INT_MAX) {
        fail(MQ_ERR_SHAPE, where);
        return nullptr;
    }
    mq_add_rmsnorm_args r = {};
    void *stream;
    long long q8_n;
    uint8_t *q8;
    r.nt = (int)nt, r.n = (int)cols;
    if (!launch_stream(a[10], dev, &stream) || !dense(a[0], "x", nt, cols, dev, &r.x) ||
        !dense(a[1], "y", nt, cols, dev, &r.y) || !dense(a[7], "x_out", nt, cols, dev, &r.x_out) ||
        (a[8] != Py_None && !dense(a[8], "z", nt, cols, dev, &r.z)) || !vec(a[2], "gain", kF32, cols, dev, &r.gain) ||
        !vec(a[4], "post_gain", kF32, cols, dev, &r.post_gain) || !vec(a[9], "q8", kU8, -1, dev, &q8, &q8_n) ||
        !number(a[3], &r.eps) || !number(a[6], &r.scale))
        return nullptr;
    if (a[5] != Py_None) {  // one gate for all rows: [n] or [1, n]
        const at::Tensor *gate = tensor(a[5], "gate", kF32, dev);
        if (!gate) return nullptr;
        if (gate->numel() == cols) {
            if (!vec(a[5], "gate", kF32, cols, dev, &r.gate)) return nullptr;
        } else if (!rows(a[5], "gate", nt, cols, dev, &r.gate, &r.gate_stride)) {
            return nullptr;
        }
    }
    if (a[9] != Py_None && cols > 0 && q8_n < nt * (long long)g.q8_bytes((int)cols)) {
        PyErr_Format(PyExc_ValueError, "q8: smaller than %lld planes of %lld values", nt, cols);
        return nullptr;
    }
    r.q8 = q8;
    return launch(where, Py_None, [&] { return g.add_rmsnorm(&r, stream); });
}

// cached, want, held, pages, free, n_free, page_size, starts, positions, seq, lens, held_out, n_free_out, status, stream
PyObject *kv_assign(PyObject *const *a, Py_ssize_t n)
{
    static const char *where = "mq_kv_assign";
    int dev;
    if (!count_ok(where, n, 15) || !device_of(a[0], "cached", &dev)) return nullptr;
    mq_kv_assign_args r = {};
    void *stream;
    long long seqs, list, nt;
    const int *pages;
    if (!launch_stream(a[14], dev, &stream) || !vec(a[0], "cached", kI32, -1, dev, &r.cached, &seqs) ||
        !vec(a[1], "want", kI32, seqs, dev, &r.want) || !vec(a[2], "held", kI32, seqs, dev, &r.held) ||
        !page_table(a[3], a[0], seqs, dev, &pages, &r.n_seqs, &r.pages_stride) ||
        !vec(a[4], "free", kI32, -1, dev, &r.free_pages, &list) || !vec(a[5], "n_free", kI32, 1, dev, &r.n_free) ||
        !integer(a[6], where, &r.page_size) || !vec(a[7], "starts", kI32, seqs + 1, dev, &r.starts) ||
        !vec(a[8], "positions", kI32, -1, dev, &r.positions, &nt) || !vec(a[9], "seq", kI32, nt, dev, &r.seq) ||
        !vec(a[10], "lens", kI32, nt, dev, &r.lens) || !vec(a[11], "held_out", kI32, seqs, dev, &r.held_out) ||
        !vec(a[12], "n_free_out", kI32, 1, dev, &r.n_free_out) || !vec(a[13], "status", kI32, 1, dev, &r.status))
        return nullptr;
    if (r.n_seqs != seqs) {
        PyErr_Format(PyExc_ValueError, "pages: %d sequences, not %lld", r.n_seqs, seqs);
        return nullptr;
    }
    if (list > INT_MAX || nt > INT_MAX) {
        fail(MQ_ERR_SHAPE, where);
        return nullptr;
    }
    r.pages = const_cast<int *>(pages), r.n_list = (int)list, r.nt = (int)nt;
    return launch(where, Py_None, [&] { return g.kv_assign(&r, stream); });
}

// logits, drafts, starts, u, u_draw, draft_probs, temperature, top_k, top_p, min_p, tokens, counts, ws, status, stream
PyObject *verify(PyObject *const *a, Py_ssize_t n)
{
    static const char *where = "mq_verify";
    mq_verify_args r = {};
    int dev;
    void *stream;
    long long vocab, seqs, ws_n;
    uint8_t *ws;
    if (!count_ok(where, n, 15) || !shape_of(a[0], "logits", where, &r.nt, &vocab) || !device_of(a[0], "logits", &dev))
        return nullptr;
    r.vocab = (int)vocab;
    if (!launch_stream(a[14], dev, &stream) || !rows(a[0], "logits", r.nt, vocab, dev, &r.logits, &r.stride) ||
        !vec(a[1], "drafts", kI32, r.nt, dev, &r.drafts) || !vec(a[2], "starts", kI32, -1, dev, &r.starts, &seqs))
        return nullptr;
    if (--seqs < 0 || seqs > INT_MAX) {
        fail(MQ_ERR_SHAPE, where);
        return nullptr;
    }
    r.n_seqs = (int)seqs;
    if (!vec(a[3], "u", kF32, r.nt, dev, &r.u) || !vec(a[4], "u_draw", kF32, seqs, dev, &r.u_draw) ||
        (a[5] != Py_None && !rows(a[5], "draft_probs", r.nt, vocab, dev, &r.draft_probs, &r.draft_stride)) ||
        !vec(a[6], "temperature", kF32, seqs, dev, &r.temperature) || !vec(a[7], "top_k", kI32, seqs, dev, &r.top_k) ||
        !vec(a[8], "top_p", kF32, seqs, dev, &r.top_p) || !vec(a[9], "min_p", kF32, seqs, dev, &r.min_p) ||
        !vec(a[10], "tokens", kI32, r.nt, dev, &r.tokens) || !vec(a[11], "counts", kI32, seqs, dev, &r.counts) ||
        !vec(a[12], "ws", kU8, -1, dev, &ws, &ws_n) || !vec(a[13], "status", kI32, 1, dev, &r.status))
        return nullptr;
    r.ws = ws, r.ws_bytes = (size_t)ws_n;
    return launch(where, Py_None, [&] { return g.verify(&r, stream); });
}

// The addresses of mq_rope_append, mq_attn_decode, mq_sample and mq_q8_bytes, MQError, the raising function; and of
// mq_add_rmsnorm_quant_q8, mq_kv_assign and mq_verify.
PyObject *setup(PyObject *const *a, Py_ssize_t n)
{
    if (!count_ok("setup", n, 9)) return nullptr;
    g.rope_append = (decltype(g.rope_append))PyLong_AsVoidPtr(a[0]);
    g.attn_decode = (decltype(g.attn_decode))PyLong_AsVoidPtr(a[1]);
    g.sample = (decltype(g.sample))PyLong_AsVoidPtr(a[2]);
    g.q8_bytes = (decltype(g.q8_bytes))PyLong_AsVoidPtr(a[3]);
    g.add_rmsnorm = (decltype(g.add_rmsnorm))PyLong_AsVoidPtr(a[6]);
    g.kv_assign = (decltype(g.kv_assign))PyLong_AsVoidPtr(a[7]);
    g.verify = (decltype(g.verify))PyLong_AsVoidPtr(a[8]);
    if (PyErr_Occurred()) return nullptr;
    Py_XSETREF(g.error, Py_NewRef(a[4]));
    Py_XSETREF(g.bad_tensor, Py_NewRef(a[5]));
    Py_RETURN_NONE;
}

// No C++ exception leaves the module (a tensor without storage raises one, an unusable device too).
template <PyObject *(*F)(PyObject *const *, Py_ssize_t)>
PyObject *guarded(PyObject *, PyObject *const *a, Py_ssize_t n)
{
    try {
        return F(a, n);
    } catch (const std::exception &e) {
        if (!PyErr_Occurred()) PyErr_SetString(PyExc_RuntimeError, e.what());
        return nullptr;
    }
}

#define METHOD(f) {#f, (PyCFunction)(void (*)())guarded<f>, METH_FASTCALL, nullptr}
PyMethodDef methods[] = {METHOD(rope_append), METHOD(attn_decode), METHOD(sample), METHOD(add_rmsnorm),
                         METHOD(kv_assign), METHOD(verify), METHOD(setup), {}};

PyModuleDef module = {PyModuleDef_HEAD_INIT, "mq_binding", nullptr, -1, methods};

}  // namespace

PyMODINIT_FUNC PyInit_mq_binding() { return PyModule_Create(&module); }
