// Argument marshalling of the serving calls (causal.py) in C++: reading the
// tensors, allocating the output and calling the C ABI takes a third of the time
// that the same steps take over ctypes, which for a single token is longer than
// the kernel runs.
//
// A call whose arguments are all as they should be, on the current device and with a
// workspace that is there and large enough, is made here. Anything else returns
// NotImplemented before anything has been launched: causal.py then takes its own way,
// which has the messages for bad arguments, switches devices and grows workspaces. No
// torch type crosses the C ABI: this module has the entry points' addresses from the
// loaded library.
#include <Python.h>

#include <ATen/ATen.h>
#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAGraphsC10Utils.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/autograd/python_variable.h>

#include <climits>
#include <cstdint>

#include "ssd_bidir.h"

namespace {

decltype(&ssd_causal_fwd) fwd_entry = nullptr;
decltype(&ssd_causal_step) step_entry = nullptr;
decltype(&ssd_cache_copy) copy_entry = nullptr;
decltype(&ssd_cache_compact) compact_entry = nullptr;
PyObject *workspaces = nullptr;   // (device, stream) -> Workspace
PyObject *check = nullptr;        // (status, name): raises for a status other than SSD_OK
PyObject *s_buf, *s_lock, *s_acquire, *s_release;

struct NotHere {};    // an argument that causal.py has to look at

void need(bool ok) {
    if (!ok) throw NotHere();
}

const at::Tensor &tensor(PyObject *o) {
    need(THPVariable_Check(o));
    return THPVariable_Unpack(o);
}

struct Call {
    int dev = -1;
    at::ScalarType io = at::kFloat;

    // the tensor that the others are checked against
    const at::Tensor &lead(PyObject *o, int64_t ndim) {
        const at::Tensor &t = tensor(o);
        need(t.is_cuda() && t.layout() == at::kStrided && t.dim() == ndim);
        dev = t.get_device();
        io = t.scalar_type();
        need(dev == c10::cuda::current_device());
        return t;
    }
    bool like(const at::Tensor &t, at::ScalarType type, at::IntArrayRef shape) const {
        return t.is_cuda() && t.get_device() == dev && t.layout() == at::kStrided && t.scalar_type() == type && t.sizes() == shape;
    }
    // contiguous and of this shape; nullptr for None
    void *whole(PyObject *o, at::ScalarType type, at::IntArrayRef shape) const {
        if (o == Py_None) return nullptr;
        const at::Tensor &t = tensor(o);
        need(like(t, type, shape) && t.is_contiguous());
        return t.data_ptr();
    }
    // the last `dims` dimensions contiguous
    const at::Tensor &rows(PyObject *o, at::IntArrayRef shape, int dims) const {
        const at::Tensor &t = tensor(o);
        need(like(t, io, shape));
        const auto st = t.strides();
        const size_t n = shape.size();
        need((st[n - 1] == 1 || shape[n - 1] <= 1) && (dims == 1 || st[n - 2] == shape[n - 1] || shape[n - 2] <= 1));
        return t;
    }
    // a pool of pages: one a row, or any number where slots name them
    const at::Tensor &pool(PyObject *o, bool slots, int64_t batch, at::IntArrayRef page) const {
        const at::Tensor &t = tensor(o);
        need(t.dim() == 4 && t.sizes().slice(1) == page && (slots || t.size(0) == batch) && t.size(0) <= INT_MAX);
        need(like(t, at::kFloat, t.sizes()) && t.is_contiguous());
        return t;
    }
};

int dtype_of(at::ScalarType t) {
    need(t == at::kFloat || t == at::kBFloat16);
    return t == at::kBFloat16 ? SSD_BF16 : SSD_F32;
}

// The same array, or no byte in common.
void apart(const at::Tensor &a, const at::Tensor &b) {
    const auto pa = reinterpret_cast<uintptr_t>(a.data_ptr()), pb = reinterpret_cast<uintptr_t>(b.data_ptr());
    need(pa == pb || pa + a.nbytes() <= pb || pb + b.nbytes() <= pa);
}

double number(PyObject *o) {
    const double v = PyFloat_AsDouble(o);
    if (v == -1.0 && PyErr_Occurred()) {
        PyErr_Clear();
        throw NotHere();
    }
    return v;
}

int integer(PyObject *o) {
    int overflow = 0;
    need(PyLong_Check(o));
    const long v = PyLong_AsLongAndOverflow(o, &overflow);
    need(!overflow && v >= INT_MIN && v <= INT_MAX);
    return (int)v;
}

// A call's workspace, its lock held: the caller's, or the stream's. Under capture a graph
// gets one of its own, which causal.py makes.
class Scratch {
  public:
    Scratch(PyObject *ws, int dev, cudaStream_t stream) {
        if (ws == Py_None) {
            need(c10::cuda::currentStreamCaptureStatusMayInitCtx() == c10::cuda::CaptureStatus::None);
            PyObject *d = PyLong_FromLong(dev), *s = PyLong_FromVoidPtr(stream);
            PyObject *key = d && s ? PyTuple_Pack(2, d, s) : nullptr;
            Py_XDECREF(d);
            Py_XDECREF(s);
            ws = key ? PyDict_GetItemWithError(workspaces, key) : nullptr;
            Py_XDECREF(key);
            PyErr_Clear();
            need(ws != nullptr);
        }
        ws_ = Py_NewRef(ws);
        lock_ = PyObject_GetAttr(ws, s_lock);
        PyObject *got = lock_ ? PyObject_CallMethodNoArgs(lock_, s_acquire) : nullptr;
        held_ = got != nullptr;
        Py_XDECREF(got);
        if (held_) buf_ = PyObject_GetAttr(ws, s_buf);
        bool ok = buf_ && THPVariable_Check(buf_);
        if (ok) {
            const at::Tensor &t = THPVariable_Unpack(buf_);
            ok = t.is_cuda() && t.get_device() == dev && t.scalar_type() == at::kByte && t.is_contiguous();
            ptr = t.data_ptr();
            bytes = t.nbytes();
        }
        if (!ok) {
            if (PyErr_Occurred() && PyErr_ExceptionMatches(PyExc_AttributeError)) PyErr_Clear();    // not an interrupt's
            release();
            throw NotHere();
        }
    }
    ~Scratch() { release(); }
    void *ptr = nullptr;
    size_t bytes = 0;

  private:
    void release() {
        if (held_) {
            // a refused call's error is kept across this one
#if PY_VERSION_HEX >= 0x030C0000
            PyObject *error = PyErr_GetRaisedException();
#else
            PyObject *type, *value, *trace;
            PyErr_Fetch(&type, &value, &trace);
#endif
            PyObject *got = PyObject_CallMethodNoArgs(lock_, s_release);
            if (!got) PyErr_Clear();
            Py_XDECREF(got);
#if PY_VERSION_HEX >= 0x030C0000
            PyErr_SetRaisedException(error);
#else
            PyErr_Restore(type, value, trace);
#endif
            held_ = false;
        }
        Py_CLEAR(lock_);
        Py_CLEAR(buf_);
        Py_CLEAR(ws_);
    }
    PyObject *ws_ = nullptr, *lock_ = nullptr, *buf_ = nullptr;
    bool held_ = false;
};

// Runs a call of the C ABI without the interpreter's lock. A workspace that is too small is
// refused there before anything is launched.
template <typename F>
bool made(const char *name, F call) {
    int rc;
    Py_BEGIN_ALLOW_THREADS;
    rc = call();
    Py_END_ALLOW_THREADS;
    need(rc != SSD_ERR_WORKSPACE);
    if (rc == SSD_OK) return true;
    PyObject *r = PyObject_CallFunction(check, "is", rc, name);
    Py_XDECREF(r);
    return false;
}

// `out` if it is given, else a new tensor like x.
at::Tensor output(const Call &c, PyObject *out, const at::Tensor &x) {
    if (out == Py_None) return at::empty(x.sizes(), x.options());
    c.whole(out, c.io, x.sizes());
    return THPVariable_Unpack(out);
}

template <int NARGS, typename F>
PyObject *guarded(Py_ssize_t n, F f) {
    if (n != NARGS) {
        PyErr_SetString(PyExc_TypeError, "wrong number of arguments");
        return nullptr;
    }
    try {
        return f();
    } catch (const NotHere &) {
    } catch (const std::exception &) {    // causal.py meets it again and raises it as torch does
    }
    if (PyErr_Occurred()) return nullptr;
    Py_RETURN_NOTIMPLEMENTED;
}

PyObject *causal_fwd(PyObject *, PyObject *const *a, Py_ssize_t n) {
    return guarded<16>(n, [&]() -> PyObject * {
        Call c;
        const at::Tensor &x = c.lead(a[0], 4);
        const int code = dtype_of(c.io);
        const int64_t batch = x.size(0), L = x.size(1), H = x.size(2), P = x.size(3);
        const at::Tensor &B0 = tensor(a[3]);
        need(B0.dim() == 4);
        const int64_t G = B0.size(2), N = B0.size(3);
        const int64_t bc[] = {batch, L, G, N}, dts[] = {batch, L, H}, vec[] = {H}, row[] = {batch}, page[] = {H, P, N};
        c.rows(a[0], x.sizes(), 2);
        const at::Tensor &dt = c.rows(a[1], dts, 1), &B = c.rows(a[3], bc, 2), &C = c.rows(a[4], bc, 2);
        need(a[2] != Py_None && batch <= INT_MAX && L <= INT_MAX && H <= INT_MAX && P <= INT_MAX && G <= INT_MAX && N <= INT_MAX);
        const auto *A = (const float *)c.whole(a[2], at::kFloat, vec), *D = (const float *)c.whole(a[5], at::kFloat, vec);
        PyObject *init = a[6], *state_out = a[13];
        const auto *lens = (const int *)c.whole(a[7], at::kInt, row), *slots = (const int *)c.whole(a[8], at::kInt, row);
        const auto *bias = (const float *)c.whole(a[9], at::kFloat, vec);
        const bool paged = a[8] != Py_None;      // (a list of no slots has no address)
        const float lo = (float)number(a[10]), hi = (float)number(a[11]);
        const int path = integer(a[14]);
        at::Tensor state;
        if (state_out == Py_None && !paged) {
            state = at::empty({batch, H, P, N}, x.options().dtype(at::kFloat));
        } else {
            if (state_out == Py_None) state_out = init;
            need(state_out != Py_None);
            state = c.pool(state_out, paged, batch, page);
        }
        const int pages = (int)state.size(0);
        float *start = nullptr;
        if (init != Py_None) {
            const at::Tensor &s = c.pool(init, true, batch, page);
            need(s.size(0) == pages);
            if (init != state_out) apart(s, state);
            start = (float *)s.data_ptr();
        }
        at::Tensor out = output(c, a[12], x);
        const cudaStream_t stream = c10::cuda::getCurrentCUDAStream((c10::DeviceIndex)c.dev).stream();
        Scratch ws(a[15], c.dev, stream);
        const void *px = x.data_ptr(), *pdt = dt.data_ptr(), *pB = B.data_ptr(), *pC = C.data_ptr();
        float *ps = (float *)state.data_ptr();
        void *po = out.data_ptr();
        if (!made("ssd_causal_fwd", [&] {
                return fwd_entry(px, pdt, A, pB, pC, D, bias, lo, hi, lens, slots, start, ps, po, x.stride(0), x.stride(1),
                                 dt.stride(0), dt.stride(1), B.stride(0), B.stride(1), C.stride(0), C.stride(1), pages, (int)batch,
                                 (int)L, (int)H, (int)P, (int)N, (int)G, code, path, ws.ptr, ws.bytes, stream);
            }))
            return nullptr;
        PyObject *o = a[12] == Py_None ? THPVariable_Wrap(std::move(out)) : Py_NewRef(a[12]);
        PyObject *s = state_out == Py_None ? THPVariable_Wrap(std::move(state)) : Py_NewRef(state_out);
        PyObject *r = o && s ? PyTuple_Pack(2, o, s) : nullptr;
        Py_XDECREF(o);
        Py_XDECREF(s);
        return r;
    });
}

PyObject *causal_step(PyObject *, PyObject *const *a, Py_ssize_t n) {
    return guarded<14>(n, [&]() -> PyObject * {
        Call c;
        const at::Tensor &x = c.lead(a[0], 3);
        const int code = dtype_of(c.io);
        const int64_t batch = x.size(0), H = x.size(1), P = x.size(2);
        const at::Tensor &B0 = tensor(a[3]);
        need(B0.dim() == 3);
        const int64_t G = B0.size(1), N = B0.size(2);
        const int64_t bc[] = {batch, G, N}, dts[] = {batch, H}, vec[] = {H}, row[] = {batch}, page[] = {H, P, N};
        c.rows(a[0], x.sizes(), 2);
        const at::Tensor &dt = c.rows(a[1], dts, 1), &B = c.rows(a[3], bc, 2), &C = c.rows(a[4], bc, 2);
        need(a[2] != Py_None && batch <= INT_MAX && H <= INT_MAX && P <= INT_MAX && G <= INT_MAX && N <= INT_MAX);
        const auto *A = (const float *)c.whole(a[2], at::kFloat, vec), *D = (const float *)c.whole(a[5], at::kFloat, vec);
        const auto *slots = (const int *)c.whole(a[7], at::kInt, row);
        const auto *bias = (const float *)c.whole(a[8], at::kFloat, vec);
        const float lo = (float)number(a[9]), hi = (float)number(a[10]);
        const at::Tensor &from = c.pool(a[6], a[7] != Py_None, batch, page);
        const int pages = (int)from.size(0);
        float *to = (float *)from.data_ptr();
        if (a[12] != Py_None && a[12] != a[6]) {
            const at::Tensor &s = c.pool(a[12], true, batch, page);
            need(s.size(0) == pages);
            apart(from, s);
            to = (float *)s.data_ptr();
        }
        at::Tensor out = output(c, a[11], x);
        const cudaStream_t stream = c10::cuda::getCurrentCUDAStream((c10::DeviceIndex)c.dev).stream();
        const void *px = x.data_ptr(), *pdt = dt.data_ptr(), *pB = B.data_ptr(), *pC = C.data_ptr();
        const float *pf = (const float *)from.data_ptr();
        void *po = out.data_ptr();
        auto run = [&](void *ws, size_t bytes) {
            return made("ssd_causal_step", [&] {
                return step_entry(px, pdt, A, pB, pC, D, bias, lo, hi, slots, pf, to, po, x.stride(0), dt.stride(0), B.stride(0),
                                  C.stride(0), pages, (int)batch, (int)H, (int)P, (int)N, (int)G, code, ws, bytes, stream);
            });
        };
        bool ok;
        if (slots) {
            Scratch ws(a[13], c.dev, stream);
            ok = run(ws.ptr, ws.bytes);
        } else {
            ok = run(nullptr, 0);
        }
        if (!ok) return nullptr;
        return a[11] == Py_None ? THPVariable_Wrap(std::move(out)) : Py_NewRef(a[11]);
    });
}

// A pool (layers, slots, page...): its pages' bytes.
const at::Tensor &pages_of(Call &c, PyObject *o, long long *bytes) {
    const at::Tensor &t = tensor(o);
    need(t.dim() >= 3);
    c.lead(o, t.dim());
    need(t.is_contiguous() && t.size(0) <= INT_MAX && t.size(1) <= INT_MAX);
    *bytes = t.numel() ? (long long)(t.nbytes() / (t.size(0) * t.size(1))) : 0;
    return t;
}

// An int32 list of one dimension: its length.
int list_of(const Call &c, PyObject *o, int **p) {
    const at::Tensor &t = tensor(o);
    need(t.dim() == 1 && t.size(0) <= INT_MAX);
    *p = (int *)c.whole(o, at::kInt, t.sizes());
    return (int)t.size(0);
}

PyObject *cache_copy(PyObject *, PyObject *const *a, Py_ssize_t n) {
    return guarded<4>(n, [&]() -> PyObject * {
        Call c;
        long long bytes;
        const at::Tensor &pool = pages_of(c, a[0], &bytes);
        int *src, *dst;
        const int m = list_of(c, a[1], &src);
        need(list_of(c, a[2], &dst) == m);
        const cudaStream_t stream = c10::cuda::getCurrentCUDAStream((c10::DeviceIndex)c.dev).stream();
        Scratch ws(a[3], c.dev, stream);
        void *p = pool.data_ptr();
        if (!made("ssd_cache_copy", [&] {
                return copy_entry(p, bytes, (int)pool.size(0), (int)pool.size(1), src, dst, m, ws.ptr, ws.bytes, stream);
            }))
            return nullptr;
        return Py_NewRef(a[0]);
    });
}

PyObject *cache_compact(PyObject *, PyObject *const *a, Py_ssize_t n) {
    return guarded<3>(n, [&]() -> PyObject * {
        Call c;
        long long bytes;
        const at::Tensor &pool = pages_of(c, a[0], &bytes);
        int *table;
        const int rows = list_of(c, a[1], &table);
        const auto options = THPVariable_Unpack(a[1]).options();
        at::Tensor moved = at::empty({rows}, options), live = at::empty({1}, options);
        const cudaStream_t stream = c10::cuda::getCurrentCUDAStream((c10::DeviceIndex)c.dev).stream();
        Scratch ws(a[2], c.dev, stream);
        void *p = pool.data_ptr();
        int *pm = (int *)moved.data_ptr(), *pl = (int *)live.data_ptr();
        if (!made("ssd_cache_compact", [&] {
                return compact_entry(p, bytes, (int)pool.size(0), (int)pool.size(1), table, rows, pm, pl, ws.ptr, ws.bytes, stream);
            }))
            return nullptr;
        PyObject *t = THPVariable_Wrap(std::move(moved)), *l = THPVariable_Wrap(std::move(live));
        PyObject *r = t && l ? PyTuple_Pack(2, t, l) : nullptr;
        Py_XDECREF(t);
        Py_XDECREF(l);
        return r;
    });
}

// setup(addresses of the four entry points, workspaces, check)
PyObject *setup(PyObject *, PyObject *const *a, Py_ssize_t n) {
    if (n != 6) {
        PyErr_SetString(PyExc_TypeError, "wrong number of arguments");
        return nullptr;
    }
    void *p[4];
    for (int i = 0; i < 4; ++i)
        if (!(p[i] = PyLong_AsVoidPtr(a[i]))) {
            if (!PyErr_Occurred()) PyErr_SetString(PyExc_ValueError, "no entry point");
            return nullptr;
        }
    fwd_entry = reinterpret_cast<decltype(fwd_entry)>(p[0]);
    step_entry = reinterpret_cast<decltype(step_entry)>(p[1]);
    copy_entry = reinterpret_cast<decltype(copy_entry)>(p[2]);
    compact_entry = reinterpret_cast<decltype(compact_entry)>(p[3]);
    if (!PyDict_Check(a[4])) {
        PyErr_SetString(PyExc_TypeError, "the workspaces are a dict");
        return nullptr;
    }
    Py_XSETREF(workspaces, Py_NewRef(a[4]));
    Py_XSETREF(check, Py_NewRef(a[5]));
    Py_RETURN_NONE;
}

template <PyObject *(*F)(PyObject *, PyObject *const *, Py_ssize_t)>
PyMethodDef method(const char *name) {
    return {name, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(F)), METH_FASTCALL, nullptr};
}

PyMethodDef methods[] = {method<causal_fwd>("causal_fwd"), method<causal_step>("causal_step"),
                         method<cache_copy>("cache_copy"), method<cache_compact>("cache_compact"),
                         method<setup>("setup"), {nullptr, nullptr, 0, nullptr}};

PyModuleDef module = {PyModuleDef_HEAD_INIT, "_binding", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__binding() {
    s_buf = PyUnicode_InternFromString("buf");
    s_lock = PyUnicode_InternFromString("lock");
    s_acquire = PyUnicode_InternFromString("acquire");
    s_release = PyUnicode_InternFromString("release");
    if (!s_buf || !s_lock || !s_acquire || !s_release) return nullptr;
    PyObject *m = PyModule_Create(&module);
    // torch's classes are used as this version lays them out: causal.py compares
    if (m && PyModule_AddStringConstant(m, "torch_version", SSD_TORCH_VERSION) < 0) Py_CLEAR(m);
    return m;
}
