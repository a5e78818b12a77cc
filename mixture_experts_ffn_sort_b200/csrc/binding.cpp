// binding.cpp -- the Python binding of the training calls as a CPython module:
// it checks torch tensors, allocates the results, and calls the C ABI
// (include/moe_ffn.h) on the tensors' device and its current stream.
//
// A small call of these is shorter on the GPU (2 to 3 us) than its argument
// checks in Python and ctypes are on the host (7 us of 9.5 us; 3 us of 5 us
// from here), which is why they are here and not beside the others.
#include <ATen/core/Tensor.h>
#include <ATen/cuda/EmptyTensor.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/autograd/python_variable.h>

#include <exception>
#include <memory>
#include <string>
#include <vector>

#include "../../include/moe_ffn.h"

namespace {

using at::Tensor;
using c10::IntArrayRef;
using c10::ScalarType;

PyObject* g_error = nullptr;  // the package's MoEError

struct Refused {};  // a Python exception is set

[[noreturn]] void refuse(const std::string& msg) {
    PyErr_SetString(PyExc_ValueError, msg.c_str());
    throw Refused{};
}

std::string text(IntArrayRef s) {
    std::string t = "(";
    for (size_t i = 0; i < s.size(); ++i) t += (i ? ", " : "") + std::to_string(s[i]);
    return t + (s.size() == 1 ? ",)" : ")");
}

void check(int rc) {
    if (rc == MOE_OK) return;
    PyObject* e = PyObject_CallFunction(g_error, "is", rc, moe_last_error());
    if (e) {
        PyErr_SetObject(g_error, e);
        Py_DECREF(e);
    }
    throw Refused{};
}

const Tensor& tensor(PyObject* o, const char* name) {
    if (!THPVariable_Check(o)) refuse(std::string(name) + " must be a tensor");
    return THPVariable_Unpack(o);
}

// Marks a caller's tensor as changed in place, so that autograd refuses a
// backward pass that saved what it held.  (Inference tensors have no such mark.)
void changed(const Tensor& t) {
    if (!t.is_inference()) t.unsafeGetTensorImpl()->bump_version();
}
void changed_if_given(PyObject* o, const Tensor& t) {
    if (o != Py_None) changed(t);
}

// The device of the call's first tensor; its current stream is the call's.
struct Call {
    int index;
    c10::cuda::OptionalCUDAGuard guard;
    explicit Call(const Tensor& t) : index(t.is_cuda() ? t.get_device() : -1) {
        if (index < 0) refuse("tensors must be CUDA tensors");
        guard.set_index(index);
    }
    explicit Call(int device) : index(device) { guard.set_index(device); }
    moe_stream_t stream() const { return c10::cuda::getCurrentCUDAStream(index).stream(); }
    Tensor empty(IntArrayRef shape, ScalarType type) const {
        return Tensor(at::detail::empty_cuda(shape, type, c10::Device(c10::kCUDA, index), std::nullopt));
    }
    // The address of a contiguous tensor of this type on the call's device.
    void* base(const Tensor& t, const char* name, ScalarType type) const {
        if (!t.is_cuda() || t.get_device() != index)
            refuse(std::string(name) + " must be a CUDA tensor on the device of the call's first tensor");
        if (t.scalar_type() != type)
            refuse(std::string(name) + " must be " + c10::toString(type) + ", not " + c10::toString(t.scalar_type()));
        if (!t.is_contiguous()) refuse(std::string(name) + " must be contiguous");
        return t.data_ptr();
    }
    void* shaped(const Tensor& t, const char* name, ScalarType type, IntArrayRef shape) const {
        if (t.sizes() != shape)
            refuse(std::string(name) + " has shape " + text(t.sizes()) + ", expected " + text(shape));
        return base(t, name, type);
    }
    void* counted(const Tensor& t, const char* name, ScalarType type, int64_t n) const {
        if (t.numel() != n)
            refuse(std::string(name) + " holds " + std::to_string(t.numel()) + " values, expected " +
                   std::to_string(n));
        return base(t, name, type);
    }
    // None, or a status word.
    int32_t* status(PyObject* o) const {
        if (o == Py_None) return nullptr;
        const Tensor& t = tensor(o, "status");
        if (t.numel() < 1) refuse("status must hold a value");
        return static_cast<int32_t*>(base(t, "status", c10::kInt));
    }
    // None, or the last value of expert_offsets: the number of sorted rows in use.
    int32_t* in_use(PyObject* o) const {
        if (o == Py_None) return nullptr;
        const Tensor& t = tensor(o, "expert_offsets");
        if (t.numel() < 1) refuse("expert_offsets must hold E + 1 values");
        return static_cast<int32_t*>(base(t, "expert_offsets", c10::kInt)) + (t.numel() - 1);
    }
    // The tensor given, or a new one.
    Tensor out(PyObject* o, const char* name, ScalarType type, IntArrayRef shape) const {
        if (o == Py_None) return empty(shape, type);
        const Tensor& t = tensor(o, name);
        shaped(t, name, type, shape);
        return t;
    }
};

int row_type(const Tensor& t, const char* name) {
    if (t.dim() != 2) refuse(std::string(name) + " must be a matrix of rows, not of shape " + text(t.sizes()));
    switch (t.scalar_type()) {
        case c10::kBFloat16: return MOE_DTYPE_BF16;
        case c10::kHalf: return MOE_DTYPE_F16;
        case c10::kFloat: return MOE_DTYPE_F32;
        default: refuse(std::string(name) + " must be bfloat16, float16 or float32, not " +
                        c10::toString(t.scalar_type()));
    }
}

int to_int(int64_t v, const char* name) {
    if (v < 0 || v > 0x7fffffff) refuse(std::string(name) + " is out of range");
    return static_cast<int>(v);
}

// Runs a call's launch without the interpreter's lock.
struct Unlocked {
    PyThreadState* state = PyEval_SaveThread();
    ~Unlocked() { PyEval_RestoreThread(state); }
};
template <class F>
void launch(F f) {
    check([&] {
        const Unlocked u;
        return f();
    }());
}

template <class F>
PyObject* guarded(Py_ssize_t n, Py_ssize_t want, F f) {
    if (n != want) {
        PyErr_Format(PyExc_TypeError, "expected %zd arguments, got %zd", want, n);
        return nullptr;
    }
    try {
        return f();
    } catch (const Refused&) {
    } catch (const std::exception& e) {
        PyErr_SetString(PyExc_RuntimeError, e.what());
    } catch (...) {
        PyErr_SetString(PyExc_RuntimeError, "unknown C++ exception");
    }
    return nullptr;
}

// Routes of T tokens: R = T * K.
int slots(int64_t R, int64_t T, const char* what) {
    const int64_t K = T ? R / T : 1;
    if (R != T * K)
        refuse(std::to_string(R) + " " + what + ": not a multiple of " + std::to_string(T) + " tokens");
    return to_int(K, "K");
}

// permute(x, inv_route, expert_offsets, x_sorted, status)
PyObject* permute(PyObject*, PyObject* const* a, Py_ssize_t n) {
    return guarded(n, 5, [&] {
        const Tensor& x = tensor(a[0], "x");
        const Call c(x);
        const int type = row_type(x, "x");
        const Tensor& inv = tensor(a[1], "inv_route");
        const int64_t T = x.size(0), H = x.size(1), R = inv.numel();
        const int K = slots(R, T, "positions in inv_route");
        const void* px = c.base(x, "x", x.scalar_type());
        const auto* pi = static_cast<const int32_t*>(c.base(inv, "inv_route", c10::kInt));
        const int32_t *rows = c.in_use(a[2]);
        int32_t* st = c.status(a[4]);
        const Tensor out = c.out(a[3], "x_sorted", x.scalar_type(), {R, H});
        const int t = to_int(T, "T"), h = to_int(H, "H");
        launch([&] { return moe_permute(px, pi, rows, t, K, h, type, out.data_ptr(), st, c.stream()); });
        changed_if_given(a[3], out);
        return THPVariable_Wrap(out);
    });
}

// unpermute(y_sorted, inv_route, topk_w, y_shared, T, out, status)
PyObject* unpermute(PyObject*, PyObject* const* a, Py_ssize_t n) {
    return guarded(n, 7, [&] {
        const Tensor& y = tensor(a[0], "the sorted rows");
        const Call c(y);
        const int type = row_type(y, "the sorted rows");
        const int64_t T = PyLong_AsLongLong(a[4]);
        if (T == -1 && PyErr_Occurred()) throw Refused{};
        const int t = to_int(T, "T"), h = to_int(y.size(1), "H");
        const int64_t R = y.size(0), H = y.size(1);
        const int K = slots(R, T, "sorted rows");
        const ScalarType row = y.scalar_type();
        const void* py = c.base(y, "the sorted rows", row);
        const auto* pi = static_cast<const int32_t*>(c.counted(tensor(a[1], "inv_route"), "inv_route", c10::kInt, R));
        const float* w = a[2] == Py_None ? nullptr : static_cast<const float*>(
            c.counted(tensor(a[2], "topk_w"), "topk_w", c10::kFloat, R));
        const void* sh = a[3] == Py_None ? nullptr : c.shaped(tensor(a[3], "y_shared"), "y_shared", row, {T, H});
        int32_t* st = c.status(a[6]);
        const Tensor out = c.out(a[5], "out", row, {T, H});
        launch([&] { return moe_unpermute(py, pi, w, sh, t, K, h, type, out.data_ptr(), st, c.stream()); });
        changed_if_given(a[5], out);
        return THPVariable_Wrap(out);
    });
}

// unpermute_bwd(dout, y_sorted, inv_route, topk_w, expert_offsets, need_dy, need_dw, dy_sorted, dtopk_w, status)
PyObject* unpermute_bwd(PyObject*, PyObject* const* a, Py_ssize_t n) {
    return guarded(n, 10, [&]() -> PyObject* {
        const Tensor& d = tensor(a[0], "dout");
        const Call c(d);
        const int type = row_type(d, "dout");
        const Tensor& w = tensor(a[3], "topk_w");
        const int64_t T = d.size(0), H = d.size(1);
        if (w.dim() != 2 || w.size(0) != T)
            refuse("topk_w must be [" + std::to_string(T) + ", K], not " + text(w.sizes()));
        const int64_t K = w.size(1), R = T * K;
        const ScalarType row = d.scalar_type();
        const bool need_dy = PyObject_IsTrue(a[5]) == 1, need_dw = PyObject_IsTrue(a[6]) == 1;
        const void* pd = c.base(d, "dout", row);
        const auto* pi = static_cast<const int32_t*>(c.counted(tensor(a[2], "inv_route"), "inv_route", c10::kInt, R));
        const auto* pw = static_cast<const float*>(c.base(w, "topk_w", c10::kFloat));
        const int32_t* rows = c.in_use(a[4]);
        int32_t* st = c.status(a[9]);
        const void* py = nullptr;
        if (need_dw) {
            if (a[1] == Py_None) refuse("the weights' gradient needs y_sorted");
            py = c.shaped(tensor(a[1], "y_sorted"), "y_sorted", row, {R, H});
        }
        Tensor dy, dw;
        if (need_dy) dy = c.out(a[7], "dy_sorted", row, {R, H});
        if (need_dw) dw = c.out(a[8], "dtopk_w", c10::kFloat, {T, K});
        if (need_dy || need_dw) {
            const int t = to_int(T, "T"), k = to_int(K, "K"), h = to_int(H, "H");
            void* pdy = need_dy ? dy.data_ptr() : nullptr;
            float* pdw = need_dw ? static_cast<float*>(dw.data_ptr()) : nullptr;
            launch([&] { return moe_unpermute_bwd(pd, py, pi, pw, rows, t, k, h, type, pdy, pdw, st, c.stream()); });
            if (need_dy) changed_if_given(a[7], dy);
            if (need_dw) changed_if_given(a[8], dw);
        }
        PyObject* pair = PyTuple_New(2);
        if (!pair) return nullptr;
        PyTuple_SET_ITEM(pair, 0, need_dy ? THPVariable_Wrap(dy) : Py_NewRef(Py_None));
        PyTuple_SET_ITEM(pair, 1, need_dw ? THPVariable_Wrap(dw) : Py_NewRef(Py_None));
        return pair;
    });
}

// route_bwd(logits, topk_ids, dtopk_w, score, n_group, topk_group, renormalize, scaling, zero_mask, dlogits, status)
PyObject* route_bwd(PyObject*, PyObject* const* a, Py_ssize_t n) {
    return guarded(n, 11, [&] {
        const Tensor& lg = tensor(a[0], "logits");
        const Call c(lg);
        const Tensor& ids = tensor(a[1], "topk_ids");
        if (lg.dim() != 2 || ids.dim() != 2) refuse("logits must be [T, E] and topk_ids [T, K]");
        const int64_t T = lg.size(0), E = lg.size(1), K = ids.size(1);
        moe_route_config cfg{};
        cfg.score = static_cast<int>(PyLong_AsLong(a[3]));
        cfg.n_group = static_cast<int>(PyLong_AsLong(a[4]));
        cfg.topk_group = a[5] == Py_None ? cfg.n_group : static_cast<int>(PyLong_AsLong(a[5]));
        cfg.renormalize = PyObject_IsTrue(a[6]) == 1;
        cfg.scaling = static_cast<float>(PyFloat_AsDouble(a[7]));
        if (PyErr_Occurred()) throw Refused{};
        const auto* pl = static_cast<const float*>(c.base(lg, "logits", c10::kFloat));
        const auto* pi = static_cast<const int32_t*>(c.shaped(ids, "topk_ids", c10::kInt, {T, K}));
        const auto* pw = static_cast<const float*>(c.shaped(tensor(a[2], "dtopk_w"), "dtopk_w", c10::kFloat, {T, K}));
        const uint8_t* mask = nullptr;
        if (a[8] != Py_None) {
            const Tensor& m = tensor(a[8], "zero_mask");
            mask = static_cast<const uint8_t*>(
                c.shaped(m, "zero_mask", m.scalar_type() == c10::kBool ? c10::kBool : c10::kByte, {T, K}));
        }
        int32_t* st = c.status(a[10]);
        const Tensor out = c.out(a[9], "dlogits", c10::kFloat, {T, E});
        const int t = to_int(T, "T"), e = to_int(E, "E"), k = to_int(K, "K");
        launch([&] {
            return moe_route_bwd(pl, pi, pw, t, e, k, &cfg, mask, static_cast<float*>(out.data_ptr()), st, c.stream());
        });
        changed_if_given(a[9], out);
        return THPVariable_Wrap(out);
    });
}

// ---------------------------------------------------------------- gradient lists

const char kRefs[] = "moe_tensor_refs";

struct Refs {
    std::vector<moe_tensor_ref> refs;
    std::vector<Tensor> tensors, outs;  // outs: empty in place
    int index;
    // Refuses a list when one of its tensors has other memory, fewer values or
    // another type than when it was checked (Tensor.data, set_, Module.to): the
    // addresses in refs are then no longer its own.
    void check_current() const {
        for (size_t i = 0; i < tensors.size(); ++i)
            if (!same(tensors[i], refs[i].data, refs[i]) || (!outs.empty() && !same(outs[i], refs[i].out, refs[i])))
                refuse("tensor " + std::to_string(i) +
                       " or its output has other memory or another type than when the list was made: make it again");
    }

  private:
    static bool same(const Tensor& t, const void* data, const moe_tensor_ref& r) {
        const ScalarType type = r.dtype == MOE_DTYPE_BF16  ? c10::kBFloat16
                                : r.dtype == MOE_DTYPE_F16 ? c10::kHalf
                                                           : c10::kFloat;
        return t.const_data_ptr() == data && t.numel() == r.numel && t.scalar_type() == type;
    }
};

void free_refs(PyObject* o) { delete static_cast<Refs*>(PyCapsule_GetPointer(o, kRefs)); }

// refs(tensors, outs, device_index): two lists of tensors, checked, as the library takes them.
PyObject* refs(PyObject*, PyObject* const* a, Py_ssize_t n) {
    return guarded(n, 3, [&]() -> PyObject* {
        if (!PyList_Check(a[0]) || !PyList_Check(a[1])) refuse("tensors and out must be lists");
        const Py_ssize_t count = PyList_GET_SIZE(a[0]);
        if (PyList_GET_SIZE(a[1]) != count)
            refuse(std::to_string(count) + " tensors but " + std::to_string(PyList_GET_SIZE(a[1])) + " outputs");
        auto r = std::make_unique<Refs>();
        r->index = static_cast<int>(PyLong_AsLong(a[2]));
        r->refs.resize(static_cast<size_t>(count) + 1);
        r->tensors.reserve(static_cast<size_t>(count));
        if (a[1] != a[0]) r->outs.reserve(static_cast<size_t>(count));
        for (Py_ssize_t i = 0; i < count; ++i) {
            const auto name = [i] { return "tensor " + std::to_string(i); };
            PyObject *pt = PyList_GET_ITEM(a[0], i), *po = PyList_GET_ITEM(a[1], i);
            if (!THPVariable_Check(pt) || !THPVariable_Check(po)) refuse(name() + " and its output must be tensors");
            const Tensor &t = THPVariable_Unpack(pt), &o = THPVariable_Unpack(po);
            int type = -1;
            switch (t.scalar_type()) {
                case c10::kBFloat16: type = MOE_DTYPE_BF16; break;
                case c10::kHalf: type = MOE_DTYPE_F16; break;
                case c10::kFloat: type = MOE_DTYPE_F32; break;
                default: refuse(name() + " must be bfloat16, float16 or float32, not " + c10::toString(t.scalar_type()));
            }
            if (!t.is_cuda() || t.get_device() != r->index || !o.is_cuda() || o.get_device() != r->index)
                refuse(name() + ": the tensors and outputs must be CUDA tensors on one device");
            if (!t.is_non_overlapping_and_dense())
                refuse(name() + " must be dense in memory (strides " + text(t.strides()) + ")");
            if (!t.is_same(o) && (o.scalar_type() != t.scalar_type() || o.sizes() != t.sizes() ||
                                  (t.numel() && o.strides() != t.strides())))
                refuse("output " + std::to_string(i) + " must have the shape, strides and type of its tensor");
            r->refs[static_cast<size_t>(i)] = {t.data_ptr(), o.data_ptr(), t.numel(), type, 0};
            r->tensors.push_back(t);
            if (a[1] != a[0]) r->outs.push_back(o);
        }
        check(moe_grad_refs_check(r->refs.data(), to_int(count, "the number of tensors")));
        return PyCapsule_New(r.release(), kRefs, free_refs);
    });
}

const Refs& unwrap(PyObject* o) {
    auto* r = static_cast<Refs*>(PyCapsule_GetPointer(o, kRefs));
    if (!r) throw Refused{};
    return *r;
}

// grad_sumsq(refs, norm or None) -> sumsq
PyObject* grad_sumsq(PyObject*, PyObject* const* a, Py_ssize_t n) {
    return guarded(n, 2, [&] {
        const Refs& r = unwrap(a[0]);
        r.check_current();
        const Call c(r.index);
        const int count = static_cast<int>(r.refs.size()) - 1;
        float* norm = a[1] == Py_None ? nullptr
                                      : static_cast<float*>(c.shaped(tensor(a[1], "norm"), "norm", c10::kFloat, {}));
        const size_t need = moe_grad_workspace_bytes(count);
        const Tensor sumsq = c.empty({}, c10::kDouble);
        const Tensor ws = c.empty({static_cast<int64_t>(need)}, c10::kByte);
        launch([&] {
            return moe_grad_sumsq(r.refs.data(), count, static_cast<double*>(sumsq.data_ptr()), norm, ws.data_ptr(),
                                  need, c.stream());
        });
        if (norm) changed(tensor(a[1], "norm"));
        return THPVariable_Wrap(sumsq);
    });
}

// grad_clip(refs, max_norm, eps, sumsq or None) -> norm
PyObject* grad_clip(PyObject*, PyObject* const* a, Py_ssize_t n) {
    return guarded(n, 4, [&] {
        const Refs& r = unwrap(a[0]);
        r.check_current();
        const Call c(r.index);
        const int count = static_cast<int>(r.refs.size()) - 1;
        const float max_norm = static_cast<float>(PyFloat_AsDouble(a[1]));
        const float eps = static_cast<float>(PyFloat_AsDouble(a[2]));
        if (PyErr_Occurred()) throw Refused{};
        const double* given = a[3] == Py_None ? nullptr : static_cast<const double*>(
            c.counted(tensor(a[3], "sumsq"), "sumsq", c10::kDouble, 1));
        const size_t need = given ? 0 : moe_grad_workspace_bytes(count);
        const Tensor norm = c.empty({}, c10::kFloat);
        Tensor ws;
        if (need) ws = c.empty({static_cast<int64_t>(need)}, c10::kByte);
        void* work = need ? ws.data_ptr() : nullptr;
        launch([&] {
            return moe_grad_clip(r.refs.data(), count, given, max_norm, eps, static_cast<float*>(norm.data_ptr()),
                                 work, need, c.stream());
        });
        for (const Tensor& t : r.outs.empty() ? r.tensors : r.outs) changed(t);
        return THPVariable_Wrap(norm);
    });
}

// error_class(cls): what a failing call raises, called with (code, message).
PyObject* error_class(PyObject*, PyObject* const* a, Py_ssize_t n) {
    return guarded(n, 1, [&] {
        Py_INCREF(a[0]);
        Py_XDECREF(g_error);
        g_error = a[0];
        return Py_NewRef(Py_None);
    });
}

#define MOE_METHOD(f) {#f, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(f)), METH_FASTCALL, nullptr}
PyMethodDef methods[] = {MOE_METHOD(permute),    MOE_METHOD(unpermute), MOE_METHOD(unpermute_bwd),
                         MOE_METHOD(route_bwd),  MOE_METHOD(refs),      MOE_METHOD(grad_sumsq),
                         MOE_METHOD(grad_clip),  MOE_METHOD(error_class), {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_binding", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__binding() { return PyModule_Create(&module); }
