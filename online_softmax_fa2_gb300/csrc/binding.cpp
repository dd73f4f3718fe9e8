// binding.cpp -- the quick way from Python to the entry points of the paged cache: a call on ordinary arguments in one
// step, without the binding's Python code (paged.py), which takes as long as the kernels of a small call (one token of 300
// keys over a cache in 8 bits: 22 us from Python, the kernel 7).
//
// Every function checks what paged.py checks.  It returns None for a call that it does not take (another device than the
// current one, anything that a check would refuse): paged.py then takes it, and raises what there is to raise.  It returns
// a status, an int, where the library refused the call, and otherwise what the call returns.
#include <torch/csrc/autograd/python_variable.h>
#include <ATen/ops/empty.h>

#include <cmath>
#include <dlfcn.h>

#include "../../include/attn.h"

namespace {

#define ENTRY(name) decltype(&name) name##_;
struct Library {
    ENTRY(attn_paged_append)
    ENTRY(attn_paged_append_q8)
    ENTRY(attn_paged_read_q8)
    ENTRY(attn_paged_fwd)
    ENTRY(attn_paged_fwd_workspace_bytes)
    ENTRY(attn_paged_fwd_q8)
    ENTRY(attn_paged_fwd_q8_workspace_bytes)
    ENTRY(attn_paged_prefix_fwd)
    ENTRY(attn_paged_prefix_fwd_workspace_bytes)
} lib;
#undef ENTRY

// Thrown where a call is left to paged.py.
struct NotTaken {};
void need(bool ok) {
    if (!ok) throw NotTaken{};
}

const at::Tensor &tensor(PyObject *o, int dev) {
    need(THPVariable_Check(o));
    const at::Tensor &t = THPVariable_Unpack(o);
    need(t.layout() == at::kStrided && t.is_cuda() && t.get_device() == dev);
    return t;
}
// Of that type and shape, with its last dimension contiguous.
const at::Tensor &tensor(PyObject *o, int dev, at::ScalarType dt, at::IntArrayRef shape) {
    const at::Tensor &t = tensor(o, dev);
    need(t.scalar_type() == dt && t.sizes() == shape && (shape.back() <= 1 || t.strides().back() == 1));
    return t;
}
bool given(PyObject *o) { return o != Py_None; }
int64_t whole(PyObject *o) {
    const long long v = PyLong_AsLongLong(o);
    if (v == -1 && PyErr_Occurred()) throw NotTaken{};
    return v;
}
float real(PyObject *o) {
    const double v = PyFloat_AsDouble(o);
    if (v == -1.0 && PyErr_Occurred()) throw NotTaken{};
    return (float)v;
}
int32_t truth(PyObject *o) {
    const int v = PyObject_IsTrue(o);
    need(v >= 0);
    return v;
}
template <size_t N>
void strides(int64_t (&to)[N], const at::Tensor &t) {
    for (size_t i = 0; i < N; ++i) to[i] = t.stride((int64_t)i);
}
const void *vector(PyObject *o, int dev, at::ScalarType dt, int64_t n) {
    return given(o) ? tensor(o, dev, dt, {n}).data_ptr() : nullptr;
}
int32_t type_of(const at::Tensor &t) {
    need(t.scalar_type() == at::kFloat || t.scalar_type() == at::kBFloat16);
    return t.scalar_type() == at::kBFloat16 ? ATTN_DTYPE_BF16 : ATTN_DTYPE_F32;
}
at::ScalarType byte_type(const at::Tensor &t, at::ScalarType named) {
    need(t.scalar_type() == named || t.scalar_type() == at::kByte);
    return t.scalar_type();
}

// The cache of a call: k_pages, v_pages, block_table, kv_lens, cu.
void fill_cache(attn_paged_cache_t &c, int dev, at::ScalarType dt, bool q8, int64_t T, int64_t d, PyObject *k, PyObject *v, PyObject *table,
                PyObject *lens, PyObject *cu) {
    const at::Tensor &kp = tensor(k, dev), &vp = tensor(v, dev), &bt = tensor(table, dev);
    need(kp.dim() == 4 && kp.size(3) == d && bt.dim() == 2);
    tensor(k, dev, q8 ? byte_type(kp, at::kFloat8_e4m3fn) : dt, kp.sizes());
    tensor(v, dev, q8 ? byte_type(vp, at::kFloat8_e4m3fn) : dt, kp.sizes());
    tensor(table, dev, at::kInt, bt.sizes());
    c.dtype = dt == at::kBFloat16 ? ATTN_DTYPE_BF16 : ATTN_DTYPE_F32;
    need(kp.size(1) <= INT32_MAX);
    c.page_size = (int32_t)kp.size(1);
    c.B = bt.size(0);
    c.T = T;
    c.Hkv = kp.size(2);
    c.d = d;
    c.k_pages = kp.data_ptr();
    c.v_pages = vp.data_ptr();
    strides(c.k_stride, kp);
    strides(c.v_stride, vp);
    c.num_pages = kp.size(0);
    c.block_table = static_cast<const int32_t *>(bt.data_ptr());
    c.table_width = bt.size(1);
    c.table_stride = bt.stride(0);
    c.kv_lens = static_cast<const int32_t *>(tensor(lens, dev, at::kInt, {c.B}).data_ptr());
    c.cu_q = static_cast<const int32_t *>(vector(cu, dev, at::kInt, c.B + 1));
}

void fill_scales(attn_paged_scales_t &s, const attn_paged_cache_t &c, int dev, PyObject *k, PyObject *v) {
    const at::Tensor &ks = tensor(k, dev), &vs = tensor(v, dev);
    const int64_t shape[3] = {c.num_pages, c.Hkv, c.page_size};
    tensor(k, dev, byte_type(ks, at::kFloat8_e8m0fnu), shape);
    tensor(v, dev, byte_type(vs, at::kFloat8_e8m0fnu), shape);
    s.k = ks.data_ptr();
    s.v = vs.data_ptr();
    strides(s.k_stride, ks);
    strides(s.v_stride, vs);
}

// f() without the interpreter's lock, as a call by ctypes has it: a launch may wait for room in the stream's queue, behind work that
// waits for a Python thread, and an allocation for the driver.
template <class F>
auto unlocked(F f) {
    struct Unlock {
        PyThreadState *state = PyEval_SaveThread();
        ~Unlock() { PyEval_RestoreThread(state); }
    } unlock;
    return f();
}

// A tensor to write: the given one, or a new one.
at::Tensor output(PyObject *o, int dev, at::ScalarType dt, at::IntArrayRef shape, const at::Tensor &like) {
    if (given(o)) return tensor(o, dev, dt, shape);
    return unlocked([&] { return at::empty(shape, like.options().dtype(dt)); });
}

PyObject *result(attn_status_t st, const at::Tensor &a) { return st ? PyLong_FromLong(st) : THPVariable_Wrap(a); }
PyObject *result(attn_status_t st, const at::Tensor &a, const at::Tensor &b) {
    if (st) return PyLong_FromLong(st);
    PyObject *x = THPVariable_Wrap(a), *y = THPVariable_Wrap(b), *r = x && y ? PyTuple_Pack(2, x, y) : nullptr;
    Py_XDECREF(x);
    Py_XDECREF(y);
    return r;
}

// body(device number, stream, arguments) with anything thrown as "not taken".  The first two arguments are the current
// device and its current stream.
template <class Body>
PyObject *call(PyObject *const *a, Py_ssize_t n, Py_ssize_t want, Body body) {
    try {
        need(n == want);
        const int64_t dev = whole(a[0]);
        void *stream = PyLong_AsVoidPtr(a[1]);
        need(!PyErr_Occurred());
        return body((int)dev, static_cast<attn_stream_t>(stream), a + 2);
    } catch (...) {
        PyErr_Clear();
        Py_RETURN_NONE;
    }
}

// q, k, v, k_pages, v_pages, k_scales, v_scales (None: not in 8 bits), block_table, kv_lens, cu_q, wq, wk, cos_sin, positions,
// eps, interleaved, q_out
PyObject *append(PyObject *, PyObject *const *args, Py_ssize_t n) {
    return call(args, n, 19, [](int dev, attn_stream_t stream, PyObject *const *a) {
        attn_paged_append_q8_params_t p{};
        attn_paged_append_params_t &x = p.append;
        const bool q8 = given(a[5]);
        const at::Tensor &q = tensor(a[0], dev);
        need(q.dim() == 3);
        type_of(q);
        const at::ScalarType dt = q.scalar_type();
        const int64_t T = q.size(0), d = q.size(2);
        fill_cache(x.cache, dev, dt, q8, T, d, a[3], a[4], a[7], a[8], a[9]);
        if (q8) fill_scales(p.scales, x.cache, dev, a[5], a[6]);
        const int64_t kv[3] = {T, x.cache.Hkv, d};
        const at::Tensor &k = tensor(a[1], dev, dt, kv), &v = tensor(a[2], dev, dt, kv);
        tensor(a[0], dev, dt, q.sizes());
        x.Hq = q.size(1);
        x.q = q.data_ptr();
        x.k = k.data_ptr();
        x.v = v.data_ptr();
        strides(x.q_stride, q);
        strides(x.k_stride, k);
        strides(x.v_stride, v);
        x.wq = vector(a[10], dev, dt, d);
        x.wk = vector(a[11], dev, dt, d);
        if (given(a[12])) {
            const at::Tensor &cs = tensor(a[12], dev);
            need(cs.dim() == 2);
            tensor(a[12], dev, at::kFloat, cs.sizes());
            x.cos_sin = static_cast<const float *>(cs.data_ptr());
            x.cos_sin_rows = cs.size(0);
            x.cos_sin_stride = cs.stride(0);
            x.rot = cs.size(1);
        }
        x.positions = static_cast<const int32_t *>(vector(a[13], dev, at::kInt, T));
        x.eps = real(a[14]);
        x.interleaved = truth(a[15]);
        const at::Tensor o = output(a[16], dev, dt, q.sizes(), q);
        x.q_out = o.data_ptr();
        strides(x.q_out_stride, o);
        return result(unlocked([&] { return q8 ? lib.attn_paged_append_q8_(&p, stream) : lib.attn_paged_append_(&x, stream); }), o);
    });
}

// k_pages, v_pages, k_scales, v_scales, block_table, kv_lens, rows, cu_k, bfloat16 (or float32), k_out, v_out
PyObject *read_q8(PyObject *, PyObject *const *args, Py_ssize_t n) {
    return call(args, n, 13, [](int dev, attn_stream_t stream, PyObject *const *a) {
        attn_paged_read_q8_params_t p{};
        const at::Tensor &kp = tensor(a[0], dev);
        need(kp.dim() == 4);
        const at::ScalarType dt = truth(a[8]) ? at::kBFloat16 : at::kFloat;
        const int64_t rows = whole(a[6]);
        need(rows >= 0);
        fill_cache(p.cache, dev, dt, true, rows, kp.size(3), a[0], a[1], a[4], a[5], a[7]);
        fill_scales(p.scales, p.cache, dev, a[2], a[3]);
        const int64_t shape[3] = {rows, p.cache.Hkv, p.cache.d};
        const at::Tensor k = output(a[9], dev, dt, shape, kp), v = output(a[10], dev, dt, shape, kp);
        p.k = k.data_ptr();
        p.v = v.data_ptr();
        strides(p.k_stride, k);
        strides(p.v_stride, v);
        return result(unlocked([&] { return lib.attn_paged_read_q8_(&p, stream); }), k, v);
    });
}

// q, k_pages, v_pages, k_scales, v_scales (None: not in 8 bits), block_table, kv_lens, cu_q, max_q, causal, scale, workspace,
// out, lse, and for prefixes prefix_table, prefix_lens, cu_prefix
struct Attention {
    attn_paged_prefix_params_t p{};
    bool q8;
    at::Tensor o, lse, workspace;

    void fill(int dev, PyObject *const *a) {
        attn_paged_fwd_params_t &f = p.fwd;
        q8 = given(a[3]);
        const at::Tensor &q = tensor(a[0], dev);
        need(q.dim() == 3);
        type_of(q);
        const at::ScalarType dt = q.scalar_type();
        tensor(a[0], dev, dt, q.sizes());
        const int64_t T = q.size(0), d = q.size(2);
        fill_cache(f.cache, dev, dt, q8, T, d, a[1], a[2], a[5], a[6], a[7]);
        if (q8) fill_scales(p.scales, f.cache, dev, a[3], a[4]);
        f.max_q = given(a[8]) ? whole(a[8]) : f.cache.cu_q ? 0 : f.cache.B ? T / f.cache.B : 0;
        f.causal = truth(a[9]);
        f.scale = given(a[10]) ? real(a[10]) : (float)(1.0 / std::sqrt((double)d));
        f.Hq = q.size(1);
        f.q = q.data_ptr();
        strides(f.q_stride, q);
        o = output(a[12], dev, dt, q.sizes(), q);
        f.o = o.data_ptr();
        strides(f.o_stride, o);
        const int64_t rows[2] = {T, f.Hq};
        lse = output(a[13], dev, at::kFloat, rows, q);
        need(lse.is_contiguous());
        f.lse = static_cast<float *>(lse.data_ptr());
    }
    // The workspace's address and size: the given one's, or of a new one of `bytes`.
    std::pair<void *, size_t> room(int dev, PyObject *given_one, size_t bytes) {
        if (given(given_one)) {
            workspace = tensor(given_one, dev);
            need(workspace.is_contiguous());
            return {workspace.data_ptr(), (size_t)workspace.nbytes()};
        }
        if (!bytes) return {nullptr, 0};
        workspace = unlocked([&] { return at::empty({(int64_t)bytes}, o.options().dtype(at::kByte)); });
        return {workspace.data_ptr(), bytes};
    }
};

PyObject *fwd(PyObject *, PyObject *const *args, Py_ssize_t n) {
    return call(args, n, 16, [](int dev, attn_stream_t stream, PyObject *const *a) {
        Attention t;
        t.fill(dev, a);
        if (t.q8) {
            attn_paged_fwd_q8_params_t p{t.p.fwd, t.p.scales};
            const auto ws = t.room(dev, a[11], given(a[11]) ? 0 : lib.attn_paged_fwd_q8_workspace_bytes_(&p));
            return result(unlocked([&] { return lib.attn_paged_fwd_q8_(&p, ws.first, ws.second, stream); }), t.o, t.lse);
        }
        const auto ws = t.room(dev, a[11], given(a[11]) ? 0 : lib.attn_paged_fwd_workspace_bytes_(&t.p.fwd));
        return result(unlocked([&] { return lib.attn_paged_fwd_(&t.p.fwd, ws.first, ws.second, stream); }), t.o, t.lse);
    });
}

PyObject *prefix_fwd(PyObject *, PyObject *const *args, Py_ssize_t n) {
    return call(args, n, 19, [](int dev, attn_stream_t stream, PyObject *const *a) {
        Attention t;
        t.fill(dev, a);
        const at::Tensor &pt = tensor(a[14], dev);
        need(pt.dim() == 2);
        tensor(a[14], dev, at::kInt, pt.sizes());
        t.p.P = pt.size(0);
        t.p.prefix_width = pt.size(1);
        t.p.prefix_stride = pt.stride(0);
        t.p.prefix_table = static_cast<const int32_t *>(pt.data_ptr());
        t.p.prefix_lens = static_cast<const int32_t *>(tensor(a[15], dev, at::kInt, {t.p.P}).data_ptr());
        t.p.cu_prefix = static_cast<const int32_t *>(vector(a[16], dev, at::kInt, t.p.P + 1));
        const auto ws = t.room(dev, a[11], given(a[11]) ? 0 : lib.attn_paged_prefix_fwd_workspace_bytes_(&t.p));
        return result(unlocked([&] { return lib.attn_paged_prefix_fwd_(&t.p, ws.first, ws.second, stream); }), t.o, t.lse);
    });
}

// The library's path.
PyObject *open_library(PyObject *, PyObject *path) {
    const char *name = PyUnicode_AsUTF8(path);
    if (!name) return nullptr;
    void *h = dlopen(name, RTLD_NOW);
#define ENTRY(e)                                                        \
    if (!h || !(lib.e##_ = reinterpret_cast<decltype(&e)>(dlsym(h, #e)))) { \
        const char *why = dlerror();                                    \
        PyErr_SetString(PyExc_RuntimeError, why ? why : #e);            \
        return nullptr;                                                 \
    }
    ENTRY(attn_paged_append)
    ENTRY(attn_paged_append_q8)
    ENTRY(attn_paged_read_q8)
    ENTRY(attn_paged_fwd)
    ENTRY(attn_paged_fwd_workspace_bytes)
    ENTRY(attn_paged_fwd_q8)
    ENTRY(attn_paged_fwd_q8_workspace_bytes)
    ENTRY(attn_paged_prefix_fwd)
    ENTRY(attn_paged_prefix_fwd_workspace_bytes)
#undef ENTRY
    Py_RETURN_NONE;
}

template <class F>
PyMethodDef method(const char *name, F f) {
    return {name, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)(void)>(f)), METH_FASTCALL, nullptr};
}
PyMethodDef methods[] = {method("append", append), method("read_q8", read_q8), method("fwd", fwd), method("prefix_fwd", prefix_fwd),
                         {"open", open_library, METH_O, nullptr}, {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_binding", nullptr, -1, methods};

}  // namespace

PyMODINIT_FUNC PyInit__binding() { return PyModule_Create(&module); }
