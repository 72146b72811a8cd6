// binding.cpp -- tensor arguments of the row operators (norm, routing, combine gradient,
// linear layer): reads sizes, strides, types and the current stream from torch tensors,
// checks them and calls the C ABI of include/moe.h. With the same checks in Python and a
// ctypes call, a norm of 128 rows took 7.9 us of host time, more than its kernel runs; with
// this module it takes 4.3 us, as much as the bare ctypes call with addresses at hand (4.2).
//
// The library's functions come by address (bind), so that one loaded libmoe.so serves both
// this module and ctypes. Every function returns the library's status; wrong tensors raise
// ValueError before the library is called. Type, shape and layout are checked before the
// device. No call records a graph, so a tensor that requires a gradient is refused where torch
// would record one, as by torch's own out= forms, and the version counters of the outputs are
// raised, by which torch's backward notices a saved tensor that was overwritten.
#include <ATen/core/grad_mode.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/autograd/python_variable.h>

#include <exception>
#include <sstream>
#include <string>

#include "moe.h"

namespace {

struct Api {
    decltype(&moe_norm) norm;
    decltype(&moe_norm_backward) norm_backward;
    decltype(&moe_route) route;
    decltype(&moe_route_backward) route_backward;
    decltype(&moe_combine_backward) combine_backward;
    decltype(&moe_linear) linear;
    decltype(&moe_linear_backward) linear_backward;
} api;

struct Refused : std::exception {
    std::string text;
    explicit Refused(std::string t) : text(std::move(t)) {}
    const char* what() const noexcept override { return text.c_str(); }
};

std::string shape_text(c10::IntArrayRef s) {
    std::ostringstream o;
    o << "(";
    for (size_t i = 0; i < s.size(); ++i) o << (i ? ", " : "") << s[i];
    o << (s.size() == 1 ? ",)" : ")");
    return o.str();
}

const char* type_text(c10::ScalarType t) {
    switch (t) {
    case c10::ScalarType::BFloat16: return "torch.bfloat16";
    case c10::ScalarType::Half: return "torch.float16";
    case c10::ScalarType::Float: return "torch.float32";
    case c10::ScalarType::Int: return "torch.int32";
    default: return c10::toString(t);
    }
}

constexpr auto F32 = c10::ScalarType::Float;
constexpr auto I32 = c10::ScalarType::Int;
constexpr auto BF16 = c10::ScalarType::BFloat16;

struct Rows {
    void* p = nullptr;
    int64_t ld = 0, rows = 0, cols = 0;
};

// The operands of one call: all on one CUDA device.
class Call {
  public:
    Call(PyObject* const* args, Py_ssize_t n, Py_ssize_t want) : a_(args) {
        if (n != want) throw Refused("wrong number of arguments");
    }
    long number(int i) const {
        const long v = PyLong_AsLong(a_[i]);
        if (v == -1 && PyErr_Occurred()) throw Refused("an integer is wanted");
        return v;
    }
    const moe_config* config(int i) const { return static_cast<const moe_config*>(address(i)); }

    // The first operand: a matrix whose type and sizes the others follow.
    Rows matrix(int i, const char* name) {
        const at::Tensor& t = tensor(i, name);
        type = t.scalar_type();
        if (type != BF16 && type != c10::ScalarType::Half && type != F32)
            throw Refused(std::string(name) + " is " + type_text(type) + ": bfloat16, float16 or float32 is wanted");
        if (t.dim() != 2) throw Refused(std::string(name) + " has shape " + shape_text(t.sizes()) + ": a matrix is wanted");
        return layout(name, t);
    }
    Rows rows(int i, const char* name, int64_t r, int64_t c, bool optional = false) {
        if (optional && a_[i] == Py_None) return Rows{nullptr, c, r, c};
        const at::Tensor& t = tensor(i, name);
        expect(name, t, type, {r, c});
        return layout(name, t);
    }
    Rows out_rows(int i, const char* name, int64_t r, int64_t c, bool optional = false) {
        const Rows o = rows(i, name, r, c, optional);
        written(i);
        return o;
    }
    // A contiguous tensor of the given type and shape; None gives null.
    template <typename T = float>
    T* vec(int i, const char* name, c10::ScalarType st, c10::IntArrayRef shape) {
        if (a_[i] == Py_None) return nullptr;
        const at::Tensor& t = tensor(i, name);
        expect(name, t, st, shape);
        if (!t.is_contiguous()) throw Refused(std::string(name) + " must be contiguous");
        return static_cast<T*>(t.data_ptr());
    }
    template <typename T = float>
    T* out_vec(int i, const char* name, c10::ScalarType st, c10::IntArrayRef shape) {
        T* p = vec<T>(i, name, st, shape);
        written(i);
        return p;
    }
    void* bytes(int i, const char* name, size_t& n) {
        n = 0;
        if (a_[i] == Py_None) return nullptr;
        const at::Tensor& t = tensor(i, name);
        if (!t.is_contiguous()) throw Refused(std::string(name) + " must be contiguous");
        n = t.nbytes();
        written(i);
        return t.data_ptr();
    }
    // Runs f(stream) with the operands' device current, without the interpreter lock.
    template <typename F>
    PyObject* run(int stream_arg, F&& f) {
        if (!first_.is_cuda()) throw Refused(first_name_ + std::string(" is not on a CUDA device"));
        const int dev = first_.index();
        void* stream = a_[stream_arg] == Py_None ? c10::cuda::getCurrentCUDAStream(dev).stream() : address(stream_arg);
        const c10::cuda::CUDAGuard current(first_);
        int status;
        Py_BEGIN_ALLOW_THREADS;
        status = f(stream);
        Py_END_ALLOW_THREADS;
        if (status == MOE_OK)
            for (int i = 0; i < n_written_; ++i) THPVariable_Unpack(a_[written_[i]]).unsafeGetTensorImpl()->bump_version();
        return PyLong_FromLong(status);
    }
    int dtype() const { return type == BF16 ? MOE_T_BF16 : type == F32 ? MOE_T_F32 : MOE_T_F16; }

    c10::ScalarType type = BF16;

  private:
    void* address(int i) const {
        void* p = PyLong_AsVoidPtr(a_[i]);
        if (!p && PyErr_Occurred()) throw Refused("an address is wanted");
        return p;
    }
    const at::Tensor& tensor(int i, const char* name) {
        PyObject* o = a_[i];
        if (o == Py_None) throw Refused(std::string(name) + " is missing");
        if (!THPVariable_Check(o)) throw Refused(std::string(name) + " is not a tensor");
        const at::Tensor& t = THPVariable_Unpack(o);
        if (t.layout() != c10::kStrided) throw Refused(std::string(name) + " is not a strided tensor");
        if (t.requires_grad() && at::GradMode::is_enabled())
            throw Refused(std::string(name) + " requires a gradient, but no graph is recorded here: call under "
                                              "torch.no_grad() or pass its detach()");
        if (!first_name_) {
            first_name_ = name;
            first_ = t.device();
        } else if (t.device() != first_) {
            throw Refused(std::string(name) + " is on " + t.device().str() + ", not on " + first_.str());
        }
        return t;
    }
    static void expect(const char* name, const at::Tensor& t, c10::ScalarType st, c10::IntArrayRef shape) {
        if (t.sizes() != shape)
            throw Refused(std::string(name) + " has shape " + shape_text(t.sizes()) + ", not " + shape_text(shape));
        if (t.scalar_type() != st)
            throw Refused(std::string(name) + " is " + type_text(t.scalar_type()) + ", not " + type_text(st));
    }
    static Rows layout(const char* name, const at::Tensor& t) {
        Rows r{t.data_ptr(), t.stride(0), t.size(0), t.size(1)};
        if (r.rows > 0x7fffffff || r.cols > 0x7fffffff) throw Refused(std::string(name) + " is too large");
        if (r.rows <= 1 && r.ld < r.cols) r.ld = r.cols;  // the stride of a single row is never used
        if (r.ld < r.cols || (t.stride(1) != 1 && r.cols > 1))
            throw Refused(std::string(name) + " has strides " + shape_text(t.strides()) +
                          "; the elements of a row must be adjacent and rows must not overlap");
        return r;
    }
    void written(int i) {
        if (a_[i] != Py_None && !THPVariable_Unpack(a_[i]).is_inference()) written_[n_written_++] = i;
    }
    PyObject* const* a_;
    int written_[6], n_written_ = 0;  // arguments that the call writes
    const char* first_name_ = nullptr;
    c10::Device first_ = c10::Device(c10::kCPU);
};

template <typename F>
PyObject* guarded(F&& f) {
    try {
        return f();
    } catch (const Refused& e) {
        if (!PyErr_Occurred()) PyErr_SetString(PyExc_ValueError, e.what());
    } catch (const std::exception& e) {
        PyErr_SetString(PyExc_RuntimeError, e.what());
    }
    return nullptr;
}

// x, w, b, eps, y, mean, rstd, kind, stream
PyObject* norm(PyObject*, PyObject* const* args, Py_ssize_t n) {
    return guarded([&] {
        Call c(args, n, 9);
        const double eps = PyFloat_AsDouble(args[3]);
        if (PyErr_Occurred()) throw Refused("eps is not a number");
        const Rows x = c.matrix(0, "x");
        const Rows y = c.out_rows(4, "y", x.rows, x.cols);
        const float* w = c.vec(1, "w", F32, {x.cols});
        const float* b = c.vec(2, "b", F32, {x.cols});
        float* mean = c.out_vec(5, "mean", F32, {x.rows});
        float* rstd = c.out_vec(6, "rstd", F32, {x.rows});
        const int kind = c.number(7);
        return c.run(8, [&](void* st) {
            return api.norm(kind, c.dtype(), x.p, x.ld, x.rows, x.cols, w, b, (float)eps, y.p, y.ld, mean, rstd, st);
        });
    });
}

// dy, x, w, mean, rstd, dx, dw, db, ws, kind, stream
PyObject* norm_backward(PyObject*, PyObject* const* args, Py_ssize_t n) {
    return guarded([&] {
        Call c(args, n, 11);
        const Rows x = c.matrix(1, "x");
        const Rows dy = c.rows(0, "dy", x.rows, x.cols);
        const Rows dx = c.out_rows(5, "dx", x.rows, x.cols, true);
        const float* w = c.vec(2, "w", F32, {x.cols});
        const float* mean = c.vec(3, "mean", F32, {x.rows});
        const float* rstd = c.vec(4, "rstd", F32, {x.rows});
        float* dw = c.out_vec(6, "dw", F32, {x.cols});
        float* db = c.out_vec(7, "db", F32, {x.cols});
        size_t nws;
        void* ws = c.bytes(8, "ws", nws);
        const int kind = c.number(9);
        return c.run(10, [&](void* st) {
            return api.norm_backward(kind, c.dtype(), dy.p, dy.ld, x.p, x.ld, x.rows, x.cols, w, mean, rstd, dx.p,
                                     dx.ld, dw, db, ws, nws, st);
        });
    });
}

Rows router(Call& c, int i, const moe_config* cfg) {
    const Rows l = c.matrix(i, "logits");
    if (l.cols != cfg->n_routed_experts)
        throw Refused("logits has " + std::to_string(l.cols) + " columns, not " + std::to_string(cfg->n_routed_experts));
    return l;
}

// cfg, logits, bias, topk_idx, topk_w, stream
PyObject* route(PyObject*, PyObject* const* args, Py_ssize_t n) {
    return guarded([&] {
        Call c(args, n, 6);
        const moe_config* cfg = c.config(0);
        const Rows l = router(c, 1, cfg);
        const float* bias = c.vec(2, "bias", F32, {l.cols});
        int32_t* idx = c.out_vec<int32_t>(3, "topk_idx", I32, {l.rows, cfg->num_experts_per_tok});
        float* w = c.out_vec(4, "topk_w", F32, {l.rows, cfg->num_experts_per_tok});
        return c.run(5, [&](void* st) { return api.route(cfg, c.dtype(), l.p, l.ld, l.rows, bias, idx, w, st); });
    });
}

// cfg, logits, topk_idx, dtopk_w, dlogits, stream
PyObject* route_backward(PyObject*, PyObject* const* args, Py_ssize_t n) {
    return guarded([&] {
        Call c(args, n, 6);
        const moe_config* cfg = c.config(0);
        const Rows l = router(c, 1, cfg);
        const int32_t* idx = c.vec<int32_t>(2, "topk_idx", I32, {l.rows, cfg->num_experts_per_tok});
        const float* dw = c.vec(3, "dtopk_w", F32, {l.rows, cfg->num_experts_per_tok});
        const Rows d = c.out_rows(4, "dlogits", l.rows, l.cols);
        return c.run(5, [&](void* st) {
            return api.route_backward(cfg, c.dtype(), l.p, l.ld, l.rows, idx, dw, d.p, d.ld, st);
        });
    });
}

// cfg, dout, y, row_of, topk_w, dy, dtopk_w, stream
PyObject* combine_backward(PyObject*, PyObject* const* args, Py_ssize_t n) {
    return guarded([&] {
        Call c(args, n, 8);
        const moe_config* cfg = c.config(0);
        const int64_t H = cfg->hidden, k = cfg->num_experts_per_tok;
        const int64_t T = c.matrix(1, "dout").rows;
        const void* dout = c.vec<void>(1, "dout", BF16, {T, H});
        const void* y = c.vec<void>(2, "y", BF16, {T * k, H});
        const int32_t* row_of = c.vec<int32_t>(3, "row_of", I32, {T * k});
        const float* w = c.vec(4, "topk_w", F32, {T, k});
        void* dy = c.out_vec<void>(5, "dy", BF16, {T * k, H});
        float* dw = c.out_vec(6, "dtopk_w", F32, {T, k});
        return c.run(7, [&](void* st) { return api.combine_backward(cfg, dout, y, row_of, w, (int32_t)T, dy, dw, st); });
    });
}

// x, w, bias, residual, y, pre, act, dev_status, stream
PyObject* linear(PyObject*, PyObject* const* args, Py_ssize_t n) {
    return guarded([&] {
        Call c(args, n, 9);
        const Rows x = c.matrix(0, "x");
        const c10::ScalarType t = c.type;
        const int64_t N = c.matrix(1, "w").rows;
        c.type = t;
        const Rows w = c.rows(1, "w", N, x.cols);
        const Rows y = c.out_rows(4, "y", x.rows, N);
        const float* bias = c.vec(2, "bias", F32, {N});
        const Rows res = c.rows(3, "residual", x.rows, N, true), pre = c.out_rows(5, "pre", x.rows, N, true);
        const int act = c.number(6);
        int32_t* status = c.out_vec<int32_t>(7, "dev_status", I32, {1});
        return c.run(8, [&](void* st) {
            return api.linear(c.dtype(), x.p, x.ld, w.p, w.ld, bias, res.p, res.ld, act, x.rows, (int32_t)N, x.cols,
                              y.p, y.ld, pre.p, pre.ld, status, st);
        });
    });
}

// dy, x, w, pre, dx, dw, db, ws, act, dev_status, stream
PyObject* linear_backward(PyObject*, PyObject* const* args, Py_ssize_t n) {
    return guarded([&] {
        Call c(args, n, 11);
        const Rows x = c.matrix(1, "x");
        const c10::ScalarType t = c.type;
        const int64_t N = c.matrix(2, "w").rows;
        c.type = t;
        const Rows w = c.rows(2, "w", N, x.cols);
        const Rows dy = c.rows(0, "dy", x.rows, N);
        const Rows pre = c.rows(3, "pre", x.rows, N, true), dx = c.out_rows(4, "dx", x.rows, x.cols, true),
                   dw = c.out_rows(5, "dw", N, x.cols, true);
        float* db = c.out_vec(6, "db", F32, {N});
        size_t nws;
        void* ws = c.bytes(7, "ws", nws);
        const int act = c.number(8);
        int32_t* status = c.out_vec<int32_t>(9, "dev_status", I32, {1});
        return c.run(10, [&](void* st) {
            return api.linear_backward(c.dtype(), dy.p, dy.ld, x.p, x.ld, w.p, w.ld, pre.p, pre.ld, act, x.rows,
                                       (int32_t)N, x.cols, dx.p, dx.ld, dw.p, dw.ld, db, ws, nws, status, st);
        });
    });
}

// bind(address of moe_norm, ...): the library's functions, in the order of Api
PyObject* bind(PyObject*, PyObject* const* args, Py_ssize_t n) {
    constexpr int kFunctions = sizeof(Api) / sizeof(void*);
    if (n != kFunctions) {
        PyErr_SetString(PyExc_ValueError, "wrong number of addresses");
        return nullptr;
    }
    void* p[kFunctions];
    for (int i = 0; i < kFunctions; ++i) {
        p[i] = PyLong_AsVoidPtr(args[i]);
        if (!p[i]) {
            if (!PyErr_Occurred()) PyErr_SetString(PyExc_ValueError, "null address");
            return nullptr;
        }
    }
    api.norm = reinterpret_cast<decltype(api.norm)>(p[0]);
    api.norm_backward = reinterpret_cast<decltype(api.norm_backward)>(p[1]);
    api.route = reinterpret_cast<decltype(api.route)>(p[2]);
    api.route_backward = reinterpret_cast<decltype(api.route_backward)>(p[3]);
    api.combine_backward = reinterpret_cast<decltype(api.combine_backward)>(p[4]);
    api.linear = reinterpret_cast<decltype(api.linear)>(p[5]);
    api.linear_backward = reinterpret_cast<decltype(api.linear_backward)>(p[6]);
    Py_RETURN_NONE;
}

#define FAST(name) {#name, reinterpret_cast<PyCFunction>(reinterpret_cast<void*>(name)), METH_FASTCALL, nullptr}
PyMethodDef methods[] = {FAST(bind),  FAST(norm),   FAST(norm_backward),   FAST(route), FAST(route_backward),
                         FAST(combine_backward), FAST(linear), FAST(linear_backward), {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_binding", nullptr, -1, methods};

}  // namespace

PyMODINIT_FUNC PyInit__binding() { return PyModule_Create(&module); }
