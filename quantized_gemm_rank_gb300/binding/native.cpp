// native.cpp -- the regular case of the binding's calls around the linears, in C++.
//
// A small call takes the GPU two to ten microseconds and the Python marshalling
// (argument checks, three tensors allocated, twenty arguments converted) longer
// than that, so a decode step was bound by it: these functions do the same work
// in a third of the time.  They take the arguments of the Python functions by position
// and return their result; None where anything is not the regular case (a
// shape, type, device or layout that does not fit, an unknown mode), which
// the Python function then handles or refuses in its own words; or, as an
// int, the library's status when it refused the call.
#include <Python.h>

#include <ATen/ops/empty.h>
#include <torch/csrc/Dtype.h>
#include <torch/csrc/autograd/python_variable.h>

#include "mc2_gb300.h"

namespace {

// A tensor argument seen as rows.
struct Rows {
    void *p = nullptr;
    int64_t ld = 0;
};

bool is_tensor(PyObject *o) { return THPVariable_Check(o); }

int dtype_code(at::ScalarType t) {
    switch (t) {
        case at::kHalf: return MC2_F16;
        case at::kBFloat16: return MC2_BF16;
        case at::kFloat: return MC2_F32;
        default: return 0;
    }
}

int code_kind(at::ScalarType t) {
    switch (t) {
        case at::kChar: return MC2_I8;
        case at::kFloat8_e4m3fn: return MC2_F8E4M3;
        case at::kFloat8_e5m2: return MC2_F8E5M2;
        default: return 0;
    }
}

bool on(const at::Tensor &t, int64_t cur) { return t.is_cuda() && t.get_device() == cur; }

// `o` as rows of the given shape, type and device: contiguous, or a matrix of strided rows.
bool rows(PyObject *o, at::IntArrayRef shape, at::ScalarType type, int64_t cur, Rows &r) {
    if (!is_tensor(o)) return false;
    const at::Tensor &t = THPVariable_Unpack(o);
    if (t.sizes() != shape || t.scalar_type() != type || !on(t, cur)) return false;
    const int64_t cols = shape.back();
    r.ld = cols;
    if (!t.is_contiguous()) {
        if (t.dim() != 2 || (cols > 1 && t.stride(1) != 1)) return false;
        if (shape[0] > 1) r.ld = t.stride(0);
        if (r.ld < cols) return false;
    }
    r.p = t.data_ptr();
    return true;
}

// A contiguous tensor of the given shape, type and device.
bool dense(PyObject *o, at::IntArrayRef shape, at::ScalarType type, int64_t cur, void *&p) {
    if (!is_tensor(o)) return false;
    const at::Tensor &t = THPVariable_Unpack(o);
    if (t.sizes() != shape || t.scalar_type() != type || !on(t, cur) || !t.is_contiguous()) return false;
    p = t.data_ptr();
    return true;
}

int64_t row_count(at::IntArrayRef shape) {
    int64_t n = 1;
    for (size_t i = 0; i + 1 < shape.size(); ++i) n *= shape[i];
    return n;
}

at::Tensor make(at::IntArrayRef shape, const at::Tensor &like, at::ScalarType type) {
    return at::empty(shape, like.options().dtype(type).requires_grad(false).memory_format(at::MemoryFormat::Contiguous));
}

// An output: the tensor given, checked, or a new one.  `ref` is a new reference.
bool output(PyObject *given, at::IntArrayRef shape, const at::Tensor &like, at::ScalarType type, int64_t cur, Rows &r,
            PyObject *&ref) {
    if (given != Py_None) {
        if (!rows(given, shape, type, cur, r)) return false;
        Py_INCREF(given);
        ref = given;
        return true;
    }
    at::Tensor t = make(shape, like, type);
    r.p = t.data_ptr();
    r.ld = shape.back();
    ref = THPVariable_Wrap(std::move(t));
    return ref != nullptr;
}

bool output_dense(PyObject *given, at::IntArrayRef shape, const at::Tensor &like, at::ScalarType type, int64_t cur, void *&p,
                  PyObject *&ref) {
    if (given != Py_None) {
        if (!dense(given, shape, type, cur, p)) return false;
        Py_INCREF(given);
        ref = given;
        return true;
    }
    at::Tensor t = make(shape, like, type);
    p = t.data_ptr();
    ref = THPVariable_Wrap(std::move(t));
    return ref != nullptr;
}

// References that are dropped unless they are taken.
struct Owned {
    PyObject *o = nullptr;
    ~Owned() { Py_XDECREF(o); }
    PyObject *take() {
        PyObject *r = o;
        o = nullptr;
        if (!r) {
            r = Py_None;
            Py_INCREF(r);
        }
        return r;
    }
};

PyObject *irregular() {
    if (PyErr_Occurred()) return nullptr;
    Py_RETURN_NONE;
}

// Runs a call without the interpreter's lock; its status.
template <class F>
int unlocked(F f) {
    int st;
    Py_BEGIN_ALLOW_THREADS
    st = f();
    Py_END_ALLOW_THREADS
    return st;
}

// C++ exceptions (an allocation that fails) become Python's.
template <class F>
PyObject *guarded(F f) {
    try {
        return f();
    } catch (const c10::OutOfMemoryError &e) {
        PyObject *torch = PyImport_ImportModule("torch");
        PyObject *type = torch ? PyObject_GetAttrString(torch, "OutOfMemoryError") : nullptr;
        if (type) PyErr_SetString(type, e.what_without_backtrace());
        Py_XDECREF(type);
        Py_XDECREF(torch);
    } catch (const std::exception &e) {
        PyErr_SetString(PyExc_RuntimeError, e.what());
    }
    return nullptr;
}

void *handle(PyObject *o) { return o == Py_None ? nullptr : PyLong_AsVoidPtr(o); }

// add_rms_norm(x, weight, residual, eps, quant_mode, q_dtype, with_out, with_rstd, out,
//              residual_out, rstd, q, scale, device, stream)
PyObject *add_rms_norm(PyObject *, PyObject *const *a, Py_ssize_t n) {
    return guarded([&]() -> PyObject * {
        if (n != 15 || !is_tensor(a[0]) || !is_tensor(a[1])) return irregular();
        const at::Tensor &x = THPVariable_Unpack(a[0]), &w = THPVariable_Unpack(a[1]);
        const int64_t cur = PyLong_AsLongLong(a[13]);
        const double eps = PyFloat_AsDouble(a[3]);
        const long mode = PyLong_AsLong(a[4]);
        if (PyErr_Occurred()) {
            PyErr_Clear();
            return irregular();
        }
        const at::IntArrayRef shape = x.sizes();
        const at::ScalarType dt = x.scalar_type(), wt = w.scalar_type();
        if (shape.size() < 2 || !dtype_code(dt) || !dtype_code(wt)) return irregular();
        const int64_t h = shape.back(), m = row_count(shape);
        const at::IntArrayRef lead = shape.slice(0, shape.size() - 1);
        Rows xr, rr, outr, ror;
        void *wp = nullptr, *sp = nullptr, *qp = nullptr, *scp = nullptr;
        Owned out, ro, rstd, q, scale;
        if (!rows(a[0], shape, dt, cur, xr) || !dense(a[1], at::IntArrayRef(h), wt, cur, wp)) return irregular();
        const bool has_res = a[2] != Py_None;
        if (has_res && !rows(a[2], shape, dt, cur, rr)) return irregular();
        if (a[8] != Py_None || (a[6] == Py_None ? mode == MC2_QUANT_NONE : PyObject_IsTrue(a[6]) == 1))
            if (!output(a[8], shape, x, dt, cur, outr, out.o)) return irregular();
        if (has_res || a[9] != Py_None)
            if (!output(a[9], shape, x, dt, cur, ror, ro.o)) return irregular();
        if (a[10] != Py_None || PyObject_IsTrue(a[7]) == 1)
            if (!output_dense(a[10], lead, x, at::kFloat, cur, sp, rstd.o)) return irregular();
        int qd = 0;
        if (mode != MC2_QUANT_NONE) {
            if (!THPDtype_Check(a[5])) return irregular();
            const at::ScalarType qt = reinterpret_cast<THPDtype *>(a[5])->scalar_type;
            qd = code_kind(qt);
            if (!qd || (mode != MC2_QUANT_PERTOKEN_DYNAMIC && mode != MC2_QUANT_PERGROUP && mode != MC2_QUANT_MX))
                return irregular();
            if (!output_dense(a[11], shape, x, qt, cur, qp, q.o)) return irregular();
            c10::SmallVector<int64_t, 5> ss(lead.begin(), lead.end());
            if (mode == MC2_QUANT_PERGROUP) ss.push_back((h + 127) / 128);
            if (mode == MC2_QUANT_MX) ss.push_back((h + 31) / 32);
            if (!output_dense(a[12], ss, x, mode == MC2_QUANT_MX ? at::kByte : at::kFloat, cur, scp, scale.o)) return irregular();
        } else if (a[11] != Py_None || a[12] != Py_None) {
            return irregular();
        }
        void *stream = handle(a[14]);
        const int st = unlocked([&] {
            return mc2_add_rms_norm(xr.p, xr.ld, rr.p, rr.ld, wp, dtype_code(wt), m, h, static_cast<float>(eps), dtype_code(dt),
                                    outr.p, outr.ld, ror.p, ror.ld, static_cast<float *>(sp), static_cast<int>(mode), qd, qp,
                                    scp, stream);
        });
        if (st != MC2_OK) return PyLong_FromLong(st);
        PyObject *d = PyDict_New();
        if (!d) return nullptr;
        struct { const char *name; Owned *o; } items[] = {{"out", &out}, {"residual", &ro}, {"rstd", &rstd}, {"q", &q}, {"scale", &scale}};
        for (auto &i : items) {
            PyObject *v = i.o->take();
            const int bad = PyDict_SetItemString(d, i.name, v);
            Py_DECREF(v);
            if (bad) {
                Py_DECREF(d);
                return nullptr;
            }
        }
        return d;
    });
}

PyObject *pair(Owned &first, Owned &second) {
    PyObject *t = PyTuple_New(2);
    if (!t) return nullptr;
    PyTuple_SET_ITEM(t, 0, first.take());
    PyTuple_SET_ITEM(t, 1, second.take());
    return t;
}

// rms_norm_grad(dy, x, weight, rstd, dres, with_weight, dx, dw, workspace, device, stream)
PyObject *rms_norm_grad(PyObject *, PyObject *const *a, Py_ssize_t n) {
    return guarded([&]() -> PyObject * {
        if (n != 11 || !is_tensor(a[1]) || !is_tensor(a[2])) return irregular();
        const at::Tensor &x = THPVariable_Unpack(a[1]), &w = THPVariable_Unpack(a[2]);
        const int64_t cur = PyLong_AsLongLong(a[9]);
        const at::IntArrayRef shape = x.sizes();
        const at::ScalarType dt = x.scalar_type(), wt = w.scalar_type();
        if (shape.size() < 2 || !dtype_code(dt) || !dtype_code(wt)) return irregular();
        const int64_t h = shape.back(), m = row_count(shape);
        Rows dyr, xr, dr, dxr;
        void *wp = nullptr, *sp = nullptr, *dwp = nullptr, *wsp = nullptr;
        size_t bytes = 0;
        Owned dx, dw;
        if (!rows(a[1], shape, dt, cur, xr) || !rows(a[0], shape, dt, cur, dyr) || !dense(a[2], at::IntArrayRef(h), wt, cur, wp) ||
            !dense(a[3], shape.slice(0, shape.size() - 1), at::kFloat, cur, sp))
            return irregular();
        if (a[4] != Py_None && !rows(a[4], shape, dt, cur, dr)) return irregular();
        if (!output(a[6], shape, x, dt, cur, dxr, dx.o)) return irregular();
        at::Tensor own;   // the workspace, if none is given
        if (PyObject_IsTrue(a[5]) == 1 || a[7] != Py_None) {
            if (!output_dense(a[7], at::IntArrayRef(h), w, wt, cur, dwp, dw.o)) return irregular();
            if (a[8] != Py_None) {
                if (!is_tensor(a[8])) return irregular();
                const at::Tensor &ws = THPVariable_Unpack(a[8]);
                if (!on(ws, cur) || !ws.is_contiguous()) return irregular();
                wsp = ws.data_ptr();
                bytes = ws.nbytes();
            } else {
                if (mc2_rms_norm_grad_workspace(m, h, &bytes) != MC2_OK) return irregular();
                const int64_t size = static_cast<int64_t>(bytes);
                own = make(at::IntArrayRef(size), x, at::kByte);
                wsp = own.data_ptr();
            }
        }
        void *stream = handle(a[10]);
        const int st = unlocked([&] {
            return mc2_rms_norm_grad(dyr.p, dyr.ld, xr.p, xr.ld, wp, dtype_code(wt), static_cast<float *>(sp), dr.p, dr.ld, m, h,
                                     dtype_code(dt), dxr.p, dxr.ld, dwp, wsp, bytes, stream);
        });
        return st != MC2_OK ? PyLong_FromLong(st) : pair(dx, dw);
    });
}

bool matrix(PyObject *o, at::ScalarType type, int64_t cur, Rows &r, int64_t &d0, int64_t &d1) {
    if (!is_tensor(o)) return false;
    const at::Tensor &t = THPVariable_Unpack(o);
    if (t.dim() != 2) return false;
    d0 = t.size(0), d1 = t.size(1);
    return rows(o, t.sizes(), type, cur, r);
}

// matmul_bias_act(x, w, w_is_nk, bias, activation, residual, with_preact, out, preact, device, stream)
PyObject *matmul_bias_act(PyObject *, PyObject *const *a, Py_ssize_t n) {
    return guarded([&]() -> PyObject * {
        if (n != 11 || !is_tensor(a[0])) return irregular();
        const at::Tensor &x = THPVariable_Unpack(a[0]);
        const int64_t cur = PyLong_AsLongLong(a[9]);
        const int act = static_cast<int>(PyLong_AsLong(a[4]));
        const int nk = PyObject_IsTrue(a[2]);
        const at::IntArrayRef shape = x.sizes();
        const at::ScalarType dt = x.scalar_type();
        if (shape.size() < 2 || !dtype_code(dt)) return irregular();
        const int64_t k = shape.back(), m = row_count(shape);
        Rows xr, wr, rr, outr, pr;
        int64_t w0 = 0, w1 = 0;
        void *bp = nullptr;
        Owned out, pre;
        if (!rows(a[0], shape, dt, cur, xr) || !matrix(a[1], dt, cur, wr, w0, w1) || (nk ? w1 : w0) != k) return irregular();
        const int64_t cols = nk ? w0 : w1;
        if (a[3] != Py_None && !dense(a[3], at::IntArrayRef(cols), dt, cur, bp)) return irregular();
        c10::SmallVector<int64_t, 5> os(shape.begin(), shape.end());
        os.back() = cols;
        if (a[5] != Py_None && !rows(a[5], os, dt, cur, rr)) return irregular();
        if (!output(a[7], os, x, dt, cur, outr, out.o)) return irregular();
        if ((a[8] != Py_None || PyObject_IsTrue(a[6]) == 1) && !output(a[8], os, x, dt, cur, pr, pre.o)) return irregular();
        void *stream = handle(a[10]);
        const int st = unlocked([&] {
            return mc2_matmul_bias_act(xr.p, xr.ld, wr.p, wr.ld, nk, m, cols, k, bp, act, rr.p, rr.ld, dtype_code(dt), outr.p,
                                       outr.ld, pr.p, pr.ld, stream);
        });
        return st != MC2_OK ? PyLong_FromLong(st) : pair(out, pre);
    });
}

// matmul_act_grad(dy, w, z, activation, w_is_nk, dz, device, stream)
PyObject *matmul_act_grad(PyObject *, PyObject *const *a, Py_ssize_t n) {
    return guarded([&]() -> PyObject * {
        if (n != 8 || !is_tensor(a[0])) return irregular();
        const at::Tensor &dy = THPVariable_Unpack(a[0]);
        const int64_t cur = PyLong_AsLongLong(a[6]);
        const int act = static_cast<int>(PyLong_AsLong(a[3]));
        const int nk = PyObject_IsTrue(a[4]);
        const at::IntArrayRef shape = dy.sizes();
        const at::ScalarType dt = dy.scalar_type();
        if (shape.size() < 2 || !dtype_code(dt)) return irregular();
        const int64_t cols = shape.back(), m = row_count(shape);
        Rows dyr, wr, zr, dzr;
        int64_t w0 = 0, w1 = 0;
        Owned dz;
        if (!rows(a[0], shape, dt, cur, dyr) || !matrix(a[1], dt, cur, wr, w0, w1) || (nk ? w0 : w1) != cols) return irregular();
        const int64_t k = nk ? w1 : w0;
        c10::SmallVector<int64_t, 5> zs(shape.begin(), shape.end());
        zs.back() = k;
        if (!rows(a[2], zs, dt, cur, zr) || !output(a[5], zs, dy, dt, cur, dzr, dz.o)) return irregular();
        void *stream = handle(a[7]);
        const int st = unlocked([&] {
            return mc2_matmul_act_grad(dyr.p, dyr.ld, wr.p, wr.ld, nk, zr.p, zr.ld, act, m, cols, k, dtype_code(dt), dzr.p, dzr.ld,
                                       stream);
        });
        return st != MC2_OK ? PyLong_FromLong(st) : dz.take();
    });
}

// act_grad(dy, z, activation, dz, device, stream)
PyObject *act_grad(PyObject *, PyObject *const *a, Py_ssize_t n) {
    return guarded([&]() -> PyObject * {
        if (n != 6 || !is_tensor(a[0])) return irregular();
        const at::Tensor &dy = THPVariable_Unpack(a[0]);
        const int64_t cur = PyLong_AsLongLong(a[4]);
        const int act = static_cast<int>(PyLong_AsLong(a[2]));
        const at::IntArrayRef shape = dy.sizes();
        const at::ScalarType dt = dy.scalar_type();
        if (shape.size() < 2 || !dtype_code(dt)) return irregular();
        Rows dyr, zr, dzr;
        Owned dz;
        if (!rows(a[0], shape, dt, cur, dyr) || !rows(a[1], shape, dt, cur, zr) || !output(a[3], shape, dy, dt, cur, dzr, dz.o))
            return irregular();
        const int64_t m = row_count(shape);
        void *stream = handle(a[5]);
        const int st = unlocked([&] {
            return mc2_act_grad(dyr.p, dyr.ld, zr.p, zr.ld, act, m, shape.back(), dtype_code(dt), dzr.p, dzr.ld, stream);
        });
        return st != MC2_OK ? PyLong_FromLong(st) : dz.take();
    });
}

#define FAST(f) {#f, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(f)), METH_FASTCALL, nullptr}
PyMethodDef kMethods[] = {FAST(add_rms_norm), FAST(rms_norm_grad), FAST(matmul_bias_act), FAST(matmul_act_grad), FAST(act_grad),
                          {nullptr, nullptr, 0, nullptr}};
PyModuleDef kModule = {PyModuleDef_HEAD_INIT, "_native", nullptr, -1, kMethods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__native() { return PyModule_Create(&kModule); }
