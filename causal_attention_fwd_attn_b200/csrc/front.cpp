// front.cpp -- the torch front end of the operators around the attention, as a CPython
// module: checks of the tensors' type, shape, layout and device, allocation of outputs, and
// the call of the C ABI on the device's current stream.  No arithmetic happens here.
//
// Checks run with the interpreter's lock; allocations, which may wait for the device, and launches,
// which wait where a stream's queue is full, run without it, so that other Python threads go on.
//
// On a few rows these operators take the GPU a few microseconds.  The same checks written in
// Python cost the host 8 to 30 us a call (a dozen tensors, five attributes each) and would be
// all that a decoding step waits for; here they cost well under one.
#include <Python.h>

#include <ATen/ATen.h>
#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/autograd/python_variable.h>

#include <algorithm>
#include <initializer_list>
#include <memory>
#include <string>
#include <vector>

#include "forge_adamw.h"
#include "forge_attn.h"
#include "forge_linear.h"

namespace {

// Read from the file by build.py and _lib.py before this module is loaded: another torch's inline
// accessors would read its tensors wrongly.
[[gnu::used]] const char kTag[] = "forge front end built for " FORGE_FRONT_TAG;

struct Refusal {  // becomes a ValueError
    std::string what;
};
struct Status {  // becomes a ForgeAttnError
    int status;
    const char* where;
};
struct PythonError {};  // already set

using at::ScalarType;
using at::Tensor;

std::string str(at::IntArrayRef s) {
    std::string r = "(";
    for (size_t i = 0; i < s.size(); ++i) r += (i ? ", " : "") + std::to_string(s[i]);
    return r + (s.size() == 1 ? ",)" : ")");
}

[[noreturn]] void refuse(const std::string& what) { throw Refusal{what}; }

bool given(PyObject* o) { return o != Py_None; }

const Tensor& tensor(PyObject* o, const char* name) {
    if (!THPVariable_Check(o)) refuse(std::string(name) + " must be a torch.Tensor");
    return THPVariable_Unpack(o);
}

// `t` must be on CUDA device `index` (negative: on any), one of `types`, of `shape`.
void check_kind(const Tensor& t, const char* name, std::initializer_list<ScalarType> types, int index,
                const at::IntArrayRef* shape) {
    if (std::find(types.begin(), types.end(), t.scalar_type()) == types.end()) {
        std::string all;
        for (ScalarType s : types) all += (all.empty() ? "" : " or ") + std::string(c10::toString(s));
        refuse(std::string(name) + " has dtype " + c10::toString(t.scalar_type()) + ", expected " + all);
    }
    if (!t.is_cuda())
        refuse(std::string(name) + " must be on a CUDA device (there is no CPU path)");
    if (index >= 0 && t.get_device() != index)
        refuse(std::string(name) + " is on " + t.device().str() + ", expected cuda:" +
               std::to_string(index));
    if (shape && t.sizes() != *shape)
        refuse(std::string(name) + " has shape " + str(t.sizes()) + ", expected " + str(*shape));
}
// The same, contiguous; returns the address.
void* check(const Tensor& t, const char* name, std::initializer_list<ScalarType> types, int index,
            const at::IntArrayRef* shape = nullptr) {
    check_kind(t, name, types, index, shape);
    if (!t.is_contiguous()) refuse(std::string(name) + " must be contiguous");
    return t.data_ptr();
}

Tensor empty(at::IntArrayRef shape, ScalarType type, int index) {
    return at::empty(shape, at::TensorOptions().dtype(type).device(at::kCUDA, (c10::DeviceIndex)index));
}

PyObject* wrap(Tensor t) {
    PyObject* o = THPVariable_Wrap(std::move(t));
    if (!o) throw PythonError{};
    return o;
}

// A reference of our own.
struct Owned {
    PyObject* o;
    explicit Owned(PyObject* p) : o(p) {
        if (!o) throw PythonError{};
    }
    ~Owned() { Py_XDECREF(o); }
    Owned(const Owned&) = delete;
    PyObject* release() {
        PyObject* p = o;
        o = nullptr;
        return p;
    }
};

// The items of a sequence, held: a list that another thread changes meanwhile does not matter.
struct Items {
    PyObject* tuple;
    Items(PyObject* o, const char* what) {
        const Owned fast(PySequence_Fast(o, what));
        tuple = PySequence_Tuple(fast.o);
        if (!tuple) throw PythonError{};
    }
    ~Items() { Py_DECREF(tuple); }
    Items(const Items&) = delete;
    Py_ssize_t size() const { return PyTuple_GET_SIZE(tuple); }
    PyObject* operator[](Py_ssize_t i) const { return PyTuple_GET_ITEM(tuple, i); }
};

// Lets other Python threads run while it lives; nothing in its scope touches a Python object.  The
// tensors that a call was given are held by its caller, or by Items.
struct Unlocked {
    PyThreadState* state = PyEval_SaveThread();
    Unlocked() = default;
    ~Unlocked() { PyEval_RestoreThread(state); }
    Unlocked(const Unlocked&) = delete;
};

bool truth(PyObject* o) {
    const int r = PyObject_IsTrue(o);
    if (r < 0) throw PythonError{};
    return r != 0;
}
double number(PyObject* o) {
    const double v = PyFloat_AsDouble(o);
    if (v == -1.0 && PyErr_Occurred()) throw PythonError{};
    return v;
}

void* stream_of(int index) {
    return c10::cuda::getCurrentCUDAStream((c10::DeviceIndex)index).stream();
}

void done(int status, const char* where) {
    if (status != FORGE_ATTN_OK) throw Status{status, where};
}

// Runs `body`, turning what it throws into a Python exception.
template <typename F>
PyObject* guarded(F body) {
    try {
        return body();
    } catch (const Refusal& r) {
        PyErr_SetString(PyExc_ValueError, r.what.c_str());
    } catch (const PythonError&) {
    } catch (const Status& s) {
        PyObject* module = PyImport_ImportModule("causal_attention_fwd_attn_b200._lib");
        PyObject* type = module ? PyObject_GetAttrString(module, "ForgeAttnError") : nullptr;
        PyObject* error = type ? PyObject_CallFunction(type, "is", s.status, s.where) : nullptr;
        if (error) PyErr_SetObject(type, error);
        Py_XDECREF(error);
        Py_XDECREF(type);
        Py_XDECREF(module);
    } catch (const c10::OutOfMemoryError& e) {
        PyObject* module = PyImport_ImportModule("torch");
        PyObject* type = module ? PyObject_GetAttrString(module, "OutOfMemoryError") : nullptr;
        if (type) PyErr_SetString(type, e.what_without_backtrace());
        Py_XDECREF(type);
        Py_XDECREF(module);
    } catch (const c10::Error& e) {
        PyErr_SetString(PyExc_RuntimeError, e.what_without_backtrace());
    } catch (const std::exception& e) {
        PyErr_SetString(PyExc_RuntimeError, e.what());
    }
    return nullptr;
}

void expect_args(Py_ssize_t n, Py_ssize_t want) {
    if (n != want) {
        PyErr_Format(PyExc_TypeError, "expected %zd arguments, got %zd", want, n);
        throw PythonError{};
    }
}

// ------------------------------------------------------------------- the QKV stage ----
constexpr ScalarType kBf16 = ScalarType::BFloat16, kF16 = ScalarType::Half, kF32 = ScalarType::Float,
                     kF64 = ScalarType::Double, kI32 = ScalarType::Int, kU8 = ScalarType::Byte;

struct Stage {
    int64_t B, T, H, Hkv, d;
    ScalarType type;
    int index, flags;
    forge_qkv_config config;
    forge_qkv_tensor q, k;
};

forge_qkv_tensor view(const Tensor& t, const char* name, const Stage& s, int64_t heads) {
    const int64_t dims[4] = {s.B, s.T, heads, s.d};
    const at::IntArrayRef shape(dims, 4);
    check_kind(t, name, {s.type}, s.index, &shape);
    const auto strides = t.strides();
    if (strides[3] != 1) refuse(std::string(name) + "'s last dimension must be contiguous");
    return forge_qkv_tensor{t.data_ptr(), strides[0], strides[1], strides[2]};
}

int small(int64_t n) {  // sizes the C ABI takes as int
    if (n > 0x7fffffff) refuse("a dimension is larger than 2^31 - 1");
    return (int)n;
}

// a: q, k, q_weight, k_weight, eps, inv_freq, positions, pair_axis, adjacent
Stage stage(PyObject* q, PyObject* k, PyObject* const* a) {
    if (!THPVariable_Check(q) || THPVariable_Unpack(q).dim() != 4 || !THPVariable_Check(k) ||
        THPVariable_Unpack(k).dim() != 4)
        refuse("q and k must be [B, T, heads, d] tensors");
    const Tensor &tq = THPVariable_Unpack(q), &tk = THPVariable_Unpack(k);
    check_kind(tq, "q", {kBf16, kF16}, -1, nullptr);
    Stage s{};
    s.B = tq.size(0);
    s.T = tq.size(1);
    s.H = tq.size(2);
    s.d = tq.size(3);
    s.Hkv = tk.size(2);
    s.type = tq.scalar_type();
    s.index = tq.get_device();
    s.q = view(tq, "q", s, s.H);
    s.k = view(tk, "k", s, s.Hkv);
    forge_qkv_config& c = s.config;
    c.B = small(s.B);
    c.T = small(s.T);
    c.H = small(s.H);
    c.Hkv = small(s.Hkv);
    c.d = small(s.d);
    c.axes = 1;
    c.eps = (float)number(a[2]);
    const at::IntArrayRef head(&s.d, 1);
    if (given(a[0]))
        c.q_weight = (const float*)check(tensor(a[0], "q_weight"), "q_weight", {kF32}, s.index, &head);
    if (given(a[1]))
        c.k_weight = (const float*)check(tensor(a[1], "k_weight"), "k_weight", {kF32}, s.index, &head);
    if (given(a[3])) {
        const Tensor& f = tensor(a[3], "inv_freq");
        c.inv_freq = (const double*)check(f, "inv_freq", {kF64}, s.index);
        if (f.dim() != 1) refuse("inv_freq must be one-dimensional");
        const int64_t pairs = f.numel();
        c.rot = small(2 * pairs);
        if (given(a[4])) {
            const Tensor& p = tensor(a[4], "positions");
            c.positions = (const int*)check(p, "positions", {kI32}, s.index);
            const int64_t n = p.dim();
            if ((n != 2 && n != 3) || p.size(-2) != s.B || p.size(-1) != s.T || p.size(0) < 1)
                refuse("positions has shape " + str(p.sizes()) + ", expected (" + std::to_string(s.B) +
                       ", " + std::to_string(s.T) + "), with the axes before it or without");
            if (n == 3) c.axes = small(p.size(0));
        }
        if (given(a[5])) {
            const at::IntArrayRef shape(&pairs, 1);
            c.pair_axis =
                (const int*)check(tensor(a[5], "pair_axis"), "pair_axis", {kI32}, s.index, &shape);
            if (!c.positions) refuse("pair_axis needs positions");
        }
    } else if (given(a[4]) || given(a[5])) {
        refuse("positions and pair_axis need inv_freq");
    }
    s.flags = (s.type == kF16 ? FORGE_ATTN_FP16 : 0) | (truth(a[6]) ? FORGE_QKV_ADJACENT : 0);
    return s;
}

// q, k, v, q_weight, k_weight, eps, inv_freq, positions, pair_axis, adjacent, out
PyObject* qkv_fwd(PyObject*, PyObject* const* a, Py_ssize_t n) {
    return guarded([&]() -> PyObject* {
        expect_args(n, 11);
        const Stage s = stage(a[0], a[1], a + 3);
        const forge_qkv_tensor v = view(tensor(a[2], "v"), "v", s, s.Hkv);
        const int64_t dims[4] = {s.B, s.H, s.T, s.d};
        const at::IntArrayRef shape(dims, 4);
        const char* names[3] = {"out q", "out k", "out v"};
        const c10::cuda::CUDAGuard guard((c10::DeviceIndex)s.index);
        void* out[3];
        Tensor made[3];
        Owned result(PyTuple_New(3));
        const bool own = !given(a[10]);
        if (!own) {
            const Items items(a[10], "out must be (q, k, v)");
            if (items.size() != 3) refuse("out must be (q, k, v)");
            for (int j = 0; j < 3; ++j) {
                out[j] = check(tensor(items[j], names[j]), names[j], {s.type}, s.index, &shape);
                Py_INCREF(items[j]);
                PyTuple_SET_ITEM(result.o, j, items[j]);
            }
        }
        int status;
        {
            const Unlocked unlocked;
            for (int j = 0; own && j < 3; ++j) {
                made[j] = empty(shape, s.type, s.index);
                out[j] = made[j].data_ptr();
            }
            status = forge_qkv_fwd(&s.config, &s.q, &s.k, &v, out[0], out[1], out[2], s.flags,
                                   stream_of(s.index));
        }
        done(status, "forge_qkv_fwd");
        for (int j = 0; own && j < 3; ++j) PyTuple_SET_ITEM(result.o, j, wrap(std::move(made[j])));
        return result.release();
    });
}

// dq, dk, dv, q, k, q_weight, k_weight, eps, inv_freq, positions, pair_axis, adjacent, out,
// weight_out, accumulate, workspace
PyObject* qkv_bwd(PyObject*, PyObject* const* a, Py_ssize_t n) {
    return guarded([&]() -> PyObject* {
        expect_args(n, 16);
        Stage s = stage(a[3], a[4], a + 5);
        const int64_t dims[4] = {s.B, s.H, s.T, s.d};
        const at::IntArrayRef shape(dims, 4);
        const Tensor& dq = tensor(a[0], "dq");
        const void* dy[3];
        dy[0] = check(dq, "dq", {s.type, kF32}, s.index, &shape);
        dy[1] = check(tensor(a[1], "dk"), "dk", {dq.scalar_type()}, s.index, &shape);
        dy[2] = check(tensor(a[2], "dv"), "dv", {dq.scalar_type()}, s.index, &shape);
        if (dq.scalar_type() == kF32) s.flags |= FORGE_QKV_GRAD_F32;
        const bool accumulate = truth(a[14]);
        const bool norm = s.config.q_weight || s.config.k_weight;
        if (accumulate && !given(a[13])) refuse("accumulate needs weight_out");
        const char* names[3] = {"out q", "out k", "out v"};
        const int64_t heads[3] = {s.H, s.Hkv, s.Hkv};
        const c10::cuda::CUDAGuard guard((c10::DeviceIndex)s.index);
        forge_qkv_tensor out[3];
        float* dw[2] = {nullptr, nullptr};
        Owned result(PyTuple_New(5));
        auto keep = [&](int at, PyObject* o) {
            Py_INCREF(o);
            PyTuple_SET_ITEM(result.o, at, o);
        };
        const bool own = !given(a[12]);
        if (!own) {
            const Items items(a[12], "out must be (q, k, v)");
            if (items.size() != 3) refuse("out must be (q, k, v)");
            for (int j = 0; j < 3; ++j) {
                out[j] = view(tensor(items[j], names[j]), names[j], s, heads[j]);
                keep(j, items[j]);
            }
        }
        const at::IntArrayRef head(&s.d, 1);
        const float* weights[2] = {s.config.q_weight, s.config.k_weight};
        bool own_dw[2] = {weights[0] != nullptr, weights[1] != nullptr};
        for (int j = 0; j < 2; ++j)
            if (!own_dw[j]) keep(3 + j, Py_None);
        if (given(a[13])) {
            const Items items(a[13], "weight_out must be (q_weight, k_weight)");
            if (items.size() != 2) refuse("weight_out must be (q_weight, k_weight)");
            for (int j = 0; j < 2; ++j) {
                if (!own_dw[j] || !given(items[j])) continue;
                dw[j] = (float*)check(tensor(items[j], "weight_out"), "weight_out", {kF32}, s.index,
                                      &head);
                own_dw[j] = false;
                keep(3 + j, items[j]);
            }
        }
        if (accumulate && (own_dw[0] || own_dw[1])) refuse("accumulate needs weight_out");
        Tensor ws, made[3], made_dw[2];
        if (given(a[15])) {
            ws = tensor(a[15], "workspace");
            check(ws, "workspace", {kU8}, s.index);
        }
        int status;
        {
            const Unlocked unlocked;
            if (own) {
                const Tensor packed = empty({s.B, s.T, s.H + 2 * s.Hkv, s.d}, s.type, s.index);
                int64_t first = 0;
                for (int j = 0; j < 3; ++j) {
                    made[j] = packed.narrow(2, first, heads[j]);
                    first += heads[j];
                    out[j] = view(made[j], names[j], s, heads[j]);
                }
            }
            for (int j = 0; j < 2; ++j) {
                if (!own_dw[j]) continue;
                made_dw[j] = empty(head, kF32, s.index);
                dw[j] = made_dw[j].data_ptr<float>();
            }
            if (!ws.defined() && norm)
                ws = empty({(int64_t)forge_qkv_bwd_workspace_size(s.config.d)}, kU8, s.index);
            status = forge_qkv_bwd(&s.config, dy[0], dy[1], dy[2], &s.q, &s.k, &out[0], &out[1],
                                   &out[2], dw[0], dw[1], accumulate,
                                   ws.defined() ? ws.data_ptr() : nullptr,
                                   ws.defined() ? (size_t)ws.numel() : 0, s.flags, stream_of(s.index));
        }
        done(status, "forge_qkv_bwd");
        for (int j = 0; own && j < 3; ++j) PyTuple_SET_ITEM(result.o, j, wrap(std::move(made[j])));
        for (int j = 0; j < 2; ++j)
            if (own_dw[j]) PyTuple_SET_ITEM(result.o, 3 + j, wrap(std::move(made_dw[j])));
        return result.release();
    });
}

// ---------------------------------------------------------------- grouped products ----
struct Pair {
    Tensor a, b;
    const int* offsets;
    int64_t experts;
    int index, flags;
};

Pair operands(PyObject* a, PyObject* b, PyObject* offsets, const char* a_name, const char* b_name,
              int64_t b_dims) {
    Pair p;
    p.a = tensor(a, a_name);
    check(p.a, a_name, {kBf16, kF16}, -1);
    p.index = p.a.get_device();
    p.b = tensor(b, b_name);
    check(p.b, b_name, {p.a.scalar_type()}, p.index);
    if (p.a.dim() != 2 || p.b.dim() != b_dims)
        refuse(std::string(a_name) + " must be 2-dimensional and " + b_name + " " +
               std::to_string(b_dims) + "-dimensional");
    const Tensor& o = tensor(offsets, "offsets");
    p.offsets = (const int*)check(o, "offsets", {kI32}, p.index);
    if (o.dim() != 1 || o.numel() < 2) refuse("offsets must be an int32 tensor [experts + 1]");
    p.experts = o.numel() - 1;
    p.flags = p.a.scalar_type() == kF16 ? FORGE_ATTN_FP16 : 0;
    return p;
}

// (rows, w, offsets, out, fp32): fp32 is None (out's type decides, or the rows') or a bool.
template <bool DX>
PyObject* grouped_rows(PyObject* const* a, Py_ssize_t n) {
    expect_args(n, 5);
    const char* name = DX ? "dy" : "x";
    Pair p = operands(a[0], a[1], a[2], name, "w", 3);
    const int64_t experts = p.b.size(0), fout = p.b.size(1), fin = p.b.size(2), rows = p.a.size(0);
    if (experts != p.experts)
        refuse("w has " + std::to_string(experts) + " experts, offsets " + std::to_string(p.experts));
    if (p.a.size(1) != (DX ? fout : fin))
        refuse(std::string(name) + " has " + std::to_string(p.a.size(1)) + " features, w " +
               (DX ? "gives " : "takes ") + std::to_string(DX ? fout : fin));
    const int64_t dims[2] = {rows, DX ? fin : fout};
    const at::IntArrayRef shape(dims, 2);
    const c10::cuda::CUDAGuard guard((c10::DeviceIndex)p.index);
    Tensor y;
    const bool own = !given(a[3]);
    const bool f32 = given(a[4]) && truth(a[4]);
    if (!own) {
        y = tensor(a[3], "out");
        check(y, "out", {p.a.scalar_type(), kF32}, p.index, &shape);
        if (given(a[4]) && f32 != (y.scalar_type() == kF32)) refuse("out and out_dtype differ");
    }
    const int n_rows = small(rows), n_experts = small(experts), n_in = small(fin), n_out = small(fout);
    int status;
    {
        const Unlocked unlocked;
        if (own) y = empty(shape, f32 ? kF32 : p.a.scalar_type(), p.index);
        const int flags = p.flags | (y.scalar_type() == kF32 ? FORGE_ATTN_OUT_F32 : 0);
        status = (DX ? forge_linear_grouped_bwd_dx : forge_linear_grouped_fwd)(
            p.a.data_ptr(), p.b.data_ptr(), y.data_ptr(), p.offsets, n_rows, n_experts, n_in, n_out,
            flags, stream_of(p.index));
    }
    done(status, DX ? "forge_linear_grouped_bwd_dx" : "forge_linear_grouped_fwd");
    if (own) return wrap(std::move(y));
    Py_INCREF(a[3]);
    return a[3];
}
PyObject* grouped_fwd(PyObject*, PyObject* const* a, Py_ssize_t n) {
    return guarded([&] { return grouped_rows<false>(a, n); });
}
PyObject* grouped_dx(PyObject*, PyObject* const* a, Py_ssize_t n) {
    return guarded([&] { return grouped_rows<true>(a, n); });
}

// dy, x, offsets, out, accumulate
PyObject* grouped_dw(PyObject*, PyObject* const* a, Py_ssize_t n) {
    return guarded([&]() -> PyObject* {
        expect_args(n, 5);
        Pair p = operands(a[0], a[1], a[2], "dy", "x", 2);
        const int64_t rows = p.a.size(0), fout = p.a.size(1), fin = p.b.size(1);
        if (p.b.size(0) != rows)
            refuse("x has " + std::to_string(p.b.size(0)) + " rows, dy " + std::to_string(rows));
        const bool accumulate = truth(a[4]);
        const int64_t dims[3] = {p.experts, fout, fin};
        const at::IntArrayRef shape(dims, 3);
        const c10::cuda::CUDAGuard guard((c10::DeviceIndex)p.index);
        Tensor dw;
        const bool own = !given(a[3]);
        if (!own) {
            dw = tensor(a[3], "out");
            check(dw, "out", {kF32}, p.index, &shape);
        } else if (accumulate) {
            refuse("accumulate needs out");
        }
        const int n_rows = small(rows), n_experts = small(p.experts), n_in = small(fin),
                  n_out = small(fout);
        int status;
        {
            const Unlocked unlocked;
            if (own) dw = empty(shape, kF32, p.index);
            status = forge_linear_grouped_bwd_dw(p.a.data_ptr(), p.b.data_ptr(), (float*)dw.data_ptr(),
                                                 p.offsets, n_rows, n_experts, n_in, n_out, accumulate,
                                                 p.flags, stream_of(p.index));
        }
        done(status, "forge_linear_grouped_bwd_dw");
        if (own) return wrap(std::move(dw));
        Py_INCREF(a[3]);
        return a[3];
    });
}

// ----------------------------------------------------------------------- gradients ----
int code_of(ScalarType t) {
    switch (t) {
        case kF32: return FORGE_GRAD_F32;
        case kBf16: return FORGE_GRAD_BF16;
        case kF16: return FORGE_GRAD_F16;
        default: return -1;
    }
}

const Tensor& flat(PyObject* o, int index, const char* what) {
    if (THPVariable_Check(o)) {
        const Tensor& t = THPVariable_Unpack(o);
        if (t.is_cuda() && t.get_device() == index && code_of(t.scalar_type()) >= 0 &&
            t.is_contiguous())
            return t;
    }
    refuse(std::string(what) + " must be contiguous fp32, bf16 or fp16 tensors on cuda:" +
           std::to_string(index));
}

// In place or not: nothing may be scaled twice, nor written while it is still to be read.
void check_writes(const std::vector<forge_grad_tensor>& table) {
    struct Span {
        uintptr_t from, to;
        bool operator<(const Span& o) const { return from < o.from; }
    };
    auto span = [](const forge_grad_tensor& t, const void* p) {
        const uintptr_t at = reinterpret_cast<uintptr_t>(p);
        return Span{at, at + (uintptr_t)t.n * (t.dtype == FORGE_GRAD_F32 ? 4 : 2)};
    };
    std::vector<Span> written;
    written.reserve(table.size());
    for (const forge_grad_tensor& t : table)
        if (t.n) written.push_back(span(t, t.out));
    if (!std::is_sorted(written.begin(), written.end())) std::sort(written.begin(), written.end());
    for (size_t k = 1; k < written.size(); ++k)
        if (written[k].from < written[k - 1].to) refuse("the same tensor is written twice");
    for (const forge_grad_tensor& t : table) {
        if (!t.n || t.grad == t.out) continue;
        const Span s = span(t, t.grad);
        const auto next = std::lower_bound(written.begin(), written.end(), s);
        if ((next != written.end() && next->from < s.to) ||
            (next != written.begin() && std::prev(next)->to > s.from))
            refuse("an output overlaps a gradient that is read for another");
    }
}

// (grads, clip, max_norm, out, norm, workspace): clip False computes the norm alone.
PyObject* grad(PyObject*, PyObject* const* a, Py_ssize_t nargs) {
    return guarded([&]() -> PyObject* {
        expect_args(nargs, 6);
        const Items grads(a[0], "gradients must be a sequence of tensors");
        const Py_ssize_t n = grads.size();
        if (n < 1) refuse("no gradients");
        if (n > 0x7fffffff) refuse("too many gradients");
        if (!THPVariable_Check(grads[0]) || !THPVariable_Unpack(grads[0]).is_cuda())
            refuse("gradients must be tensors on a CUDA device (there is no CPU path)");
        const int index = THPVariable_Unpack(grads[0]).get_device();
        const bool clip = truth(a[1]);
        const float max_norm = clip ? (float)number(a[2]) : 0.f;
        std::vector<forge_grad_tensor> table((size_t)n);
        for (Py_ssize_t k = 0; k < n; ++k) {
            const Tensor& t = flat(grads[k], index, "gradients");
            table[k] = forge_grad_tensor{t.data_ptr(), t.data_ptr(), t.numel(),
                                         code_of(t.scalar_type())};
        }
        std::unique_ptr<Items> out;  // holds the outputs until the launch
        if (clip && given(a[3])) {
            out = std::make_unique<Items>(a[3], "outputs must be a sequence of tensors");
            if (out->size() != n)
                refuse(std::to_string(n) + " gradients, " + std::to_string(out->size()) + " outputs");
            for (Py_ssize_t k = 0; k < n; ++k) {
                const Tensor& t = flat((*out)[k], index, "outputs");
                if (t.numel() != table[k].n || code_of(t.scalar_type()) != table[k].dtype)
                    refuse("outputs must have their gradients' sizes and types");
                table[k].out = t.data_ptr();
            }
        }
        if (clip) check_writes(table);
        const c10::cuda::CUDAGuard guard((c10::DeviceIndex)index);
        Tensor norm, ws;
        if (given(a[4])) {
            norm = tensor(a[4], "norm");
            check(norm, "norm", {kF32}, index);
            if (norm.numel() != 1) refuse("norm must have one element");
        }
        if (given(a[5])) {
            ws = tensor(a[5], "workspace");
            check(ws, "workspace", {kU8}, index);
        }
        int status;
        {
            const Unlocked unlocked;
            if (!norm.defined()) norm = empty({}, kF32, index);
            if (!ws.defined()) ws = empty({(int64_t)forge_grad_workspace_size((int)n)}, kU8, index);
            float* to = norm.data_ptr<float>();
            const size_t bytes = (size_t)ws.numel();
            status = clip ? forge_grad_clip(table.data(), (int)n, max_norm, to, ws.data_ptr(), bytes,
                                            stream_of(index))
                          : forge_grad_norm(table.data(), (int)n, to, ws.data_ptr(), bytes,
                                            stream_of(index));
        }
        done(status, clip ? "forge_grad_clip" : "forge_grad_norm");
        if (!given(a[4])) return wrap(std::move(norm));
        Py_INCREF(a[4]);
        return a[4];
    });
}

using Fast = PyObject* (*)(PyObject*, PyObject* const*, Py_ssize_t);
PyCFunction as_method(Fast f) {
    return reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(f));
}

PyMethodDef* methods() {
    static PyMethodDef table[] = {
        {"qkv_fwd", as_method(qkv_fwd), METH_FASTCALL, nullptr},
        {"qkv_bwd", as_method(qkv_bwd), METH_FASTCALL, nullptr},
        {"grouped_fwd", as_method(grouped_fwd), METH_FASTCALL, nullptr},
        {"grouped_dx", as_method(grouped_dx), METH_FASTCALL, nullptr},
        {"grouped_dw", as_method(grouped_dw), METH_FASTCALL, nullptr},
        {"grad", as_method(grad), METH_FASTCALL, nullptr},
        {nullptr, nullptr, 0, nullptr},
    };
    return table;
}

}  // namespace

PyMODINIT_FUNC PyInit__front(void) {
    static PyModuleDef def = {PyModuleDef_HEAD_INIT, "_front",
                              "torch front end of the operators around the attention", -1, methods(),
                              nullptr, nullptr, nullptr, nullptr};
    return PyModule_Create(&def);
}
