// The Python binding of the MoE operators' calls: checks the tensors' types, shapes and layout,
// takes their pointers and the current stream, and calls the C ABI.  The decode-size calls run
// for 2-5 us on the GPU; marshalled through ctypes they cost the host 5-10 us each, here 2-4 us
// (1.8 us of it the launch).
//
// Every function takes its tensors first, then plain numbers, then the stream (an address, or
// None for torch's current one), and returns the call's status.  A tensor of a wrong type or
// shape, or of another device than the current one, raises TypeError or ValueError before anything is
// called.
#define PY_SSIZE_T_CLEAN
#include <Python.h>

#include <ATen/core/Tensor.h>
#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/autograd/python_variable.h>

#include <initializer_list>

#include "dg.h"

namespace {

// Element types, by what the library takes them for.
enum : unsigned { BF16 = 1, F32 = 2, I32 = 4, FP8 = 8 };

unsigned kind_of(const at::Tensor& t) {
    switch (t.scalar_type()) {
        case at::kBFloat16:
        case at::kShort:
        case at::kUInt16: return BF16;
        case at::kFloat: return F32;
        case at::kInt: return I32;
        case at::kByte:
        case at::kFloat8_e4m3fn: return FP8;
        default: return 0;
    }
}

const char* name_of(unsigned kinds) {
    switch (kinds) {
        case BF16: return "bfloat16 (or its 16-bit integer view)";
        case F32: return "float32";
        case I32: return "int32";
        case FP8: return "uint8 or float8_e4m3fn";
        default: return "bfloat16 or float32";
    }
}

// Thrown once a Python error is set.
struct Raised {};

[[noreturn]] void raise(PyObject* type, const char* what, const char* must) {
    PyErr_Format(type, "%s must %s", what, must);
    throw Raised();
}

// The current device, as the call under way found it (-1: not asked yet).
thread_local int call_device = -1;

const at::Tensor& tensor(PyObject* o, const char* what) {
    if (!THPVariable_Check(o)) raise(PyExc_TypeError, what, "be a CUDA tensor");
    const at::Tensor& t = THPVariable_Unpack(o);
    if (!t.is_cuda()) raise(PyExc_TypeError, what, "be a CUDA tensor");
    if (call_device < 0) call_device = c10::cuda::current_device();
    // (the launch goes to the current device, whose kernels may not read another's memory)
    if (t.get_device() != call_device) raise(PyExc_ValueError, what, "be on the current CUDA device");
    if (!t.is_contiguous()) raise(PyExc_ValueError, what, "be contiguous");
    return t;
}

unsigned kind(const at::Tensor& t, const char* what, unsigned kinds) {
    const unsigned k = kind_of(t);
    if (!(k & kinds)) {
        PyErr_Format(PyExc_TypeError, "%s must be %s", what, name_of(kinds));
        throw Raised();
    }
    return k;
}

void dims(const at::Tensor& t, const char* what, int64_t n) {
    if (t.dim() != n) {
        PyErr_Format(PyExc_ValueError, "%s must have %d dimensions, got %d", what, static_cast<int>(n),
                     static_cast<int>(t.dim()));
        throw Raised();
    }
}

// A size as the C ABI takes it.
int size(int64_t n, const char* what) {
    if (n > 0x7FFFFFFF) raise(PyExc_ValueError, what, "have sizes below 2^31");
    return static_cast<int>(n);
}

void* pointer(PyObject* o, const char* what, unsigned kinds, std::initializer_list<int64_t> shape) {
    const at::Tensor& t = tensor(o, what);
    kind(t, what, kinds);
    if (t.sizes() != at::IntArrayRef(shape)) {
        PyErr_Format(PyExc_ValueError, "%s has a shape that does not go with the other arguments'", what);
        throw Raised();
    }
    return t.data_ptr();
}

void* optional(PyObject* o, const char* what, unsigned kinds, std::initializer_list<int64_t> shape) {
    return o == Py_None ? nullptr : pointer(o, what, kinds, shape);
}

int64_t number(PyObject* o) {
    const long long v = PyLong_AsLongLong(o);
    if (v == -1 && PyErr_Occurred()) throw Raised();
    return v;
}

int truth(PyObject* o) {
    const int v = PyObject_IsTrue(o);
    if (v < 0) throw Raised();
    return v;
}

int integer(PyObject* o, const char* what) {
    const int64_t v = number(o);
    if (v < -0x7FFFFFFF || v > 0x7FFFFFFF) raise(PyExc_ValueError, what, "be below 2^31");
    return static_cast<int>(v);
}

float real(PyObject* o) {
    const double v = PyFloat_AsDouble(o);
    if (v == -1.0 && PyErr_Occurred()) throw Raised();
    return static_cast<float>(v);
}

void* stream_of(PyObject* o) {
    if (o == Py_None) return c10::cuda::getCurrentCUDAStream().stream();
    return reinterpret_cast<void*>(static_cast<intptr_t>(number(o)));
}

int dtype_of(unsigned kind) { return kind == F32 ? DG_F32 : DG_BF16; }

// Runs f(args) with the argument count checked and every exception turned into a Python error.
template <int N, class F>
PyObject* guarded(Py_ssize_t n, const F& f) {
    if (n != N) {
        PyErr_Format(PyExc_TypeError, "expected %d arguments, got %zd", N, n);
        return nullptr;
    }
    try {
        call_device = -1;
        return PyLong_FromLong(f());
    } catch (const Raised&) {
    } catch (const std::exception& e) {
        PyErr_SetString(PyExc_RuntimeError, e.what());
    } catch (...) {
        PyErr_SetString(PyExc_RuntimeError, "unknown error");
    }
    return nullptr;
}

// logits, topk_idx, topk_w, scoring, renormalize, scale, stream
PyObject* moe_route(PyObject*, PyObject* const* a, Py_ssize_t n) {
    return guarded<7>(n, [&] {
        const at::Tensor& x = tensor(a[0], "logits");
        const at::Tensor& idx = tensor(a[1], "topk_idx");
        dims(x, "logits", 2);
        dims(idx, "topk_idx", 2);
        const unsigned kx = kind(x, "logits", BF16 | F32);
        const int64_t T = x.size(0), E = x.size(1), k = idx.size(1);
        return dg_moe_route(x.data_ptr(), static_cast<int32_t*>(pointer(a[1], "topk_idx", I32, {T, k})),
                            static_cast<float*>(pointer(a[2], "topk_w", F32, {T, k})), size(T, "logits"), size(E, "logits"),
                            size(k, "topk_idx"), dtype_of(kx), integer(a[3], "scoring"), truth(a[4]), real(a[5]),
                            stream_of(a[6]));
    });
}

// logits, topk_idx, dw, dlogits, scoring, renormalize, scale, stream
PyObject* moe_route_backward(PyObject*, PyObject* const* a, Py_ssize_t n) {
    return guarded<8>(n, [&] {
        const at::Tensor& x = tensor(a[0], "logits");
        const at::Tensor& idx = tensor(a[1], "topk_idx");
        dims(x, "logits", 2);
        dims(idx, "topk_idx", 2);
        const unsigned kx = kind(x, "logits", BF16 | F32);
        const int64_t T = x.size(0), E = x.size(1), k = idx.size(1);
        return dg_moe_route_backward(x.data_ptr(), static_cast<int32_t*>(pointer(a[1], "topk_idx", I32, {T, k})),
                                     static_cast<float*>(pointer(a[2], "dw", F32, {T, k})),
                                     pointer(a[3], "dlogits", kx, {T, E}), size(T, "logits"), size(E, "logits"),
                                     size(k, "topk_idx"), dtype_of(kx), integer(a[4], "scoring"), truth(a[5]),
                                     real(a[6]), stream_of(a[7]));
    });
}

// topk_idx, pos, m_indices, counts, ks, stream
PyObject* moe_sort(PyObject*, PyObject* const* a, Py_ssize_t n) {
    return guarded<6>(n, [&] {
        const at::Tensor& idx = tensor(a[0], "topk_idx");
        const at::Tensor& m = tensor(a[2], "m_indices");
        const at::Tensor& counts = tensor(a[3], "counts");
        dims(idx, "topk_idx", 2);
        dims(m, "m_indices", 1);
        dims(counts, "counts", 1);
        const int64_t T = idx.size(0), k = idx.size(1), rows = m.size(0), G = counts.size(0);
        return dg_moe_sort(static_cast<int32_t*>(pointer(a[0], "topk_idx", I32, {T, k})),
                           static_cast<int32_t*>(pointer(a[1], "pos", I32, {T, k})),
                           static_cast<int32_t*>(pointer(a[2], "m_indices", I32, {rows})),
                           static_cast<int32_t*>(pointer(a[3], "counts", I32, {G})),
                           static_cast<int32_t*>(optional(a[4], "ks", I32, {G})), size(T, "topk_idx"), size(k, "topk_idx"),
                           size(G, "counts"), size(rows, "m_indices"), stream_of(a[5]));
    });
}

// topk_idx, pos, masked_m, max_m, stream
PyObject* moe_sort_masked(PyObject*, PyObject* const* a, Py_ssize_t n) {
    return guarded<5>(n, [&] {
        const at::Tensor& idx = tensor(a[0], "topk_idx");
        const at::Tensor& counts = tensor(a[2], "masked_m");
        dims(idx, "topk_idx", 2);
        dims(counts, "masked_m", 1);
        const int64_t T = idx.size(0), k = idx.size(1), G = counts.size(0);
        return dg_moe_sort_masked(static_cast<int32_t*>(pointer(a[0], "topk_idx", I32, {T, k})),
                                  static_cast<int32_t*>(pointer(a[1], "pos", I32, {T, k})),
                                  static_cast<int32_t*>(pointer(a[2], "masked_m", I32, {G})), size(T, "topk_idx"),
                                  size(k, "topk_idx"), size(G, "masked_m"), integer(a[3], "max_m"), stream_of(a[4]));
    });
}

// Rows of a [rows, N] or [G, max_m, N] tensor, whose last dimension is N.
struct Rows {
    const at::Tensor& t;
    int64_t rows, groups, per;
    Rows(PyObject* o, const char* what, int64_t N) : t(tensor(o, what)) {
        if (t.dim() != 2 && t.dim() != 3) raise(PyExc_ValueError, what, "have 2 or 3 dimensions");
        if (t.size(-1) != N) raise(PyExc_ValueError, what, "have rows as long as the tokens'");
        groups = t.dim() == 3 ? t.size(0) : 1;
        per = t.size(-2);
        rows = groups * per;
    }
};

// x, pos, out, m_indices, stream
PyObject* moe_dispatch(PyObject*, PyObject* const* a, Py_ssize_t n) {
    return guarded<5>(n, [&] {
        const at::Tensor& x = tensor(a[0], "x");
        const at::Tensor& pos = tensor(a[1], "pos");
        dims(x, "x", 2);
        dims(pos, "pos", 2);
        const unsigned kx = kind(x, "x", BF16 | F32);
        const int64_t T = x.size(0), K = x.size(1), k = pos.size(1);
        const Rows out(a[2], "out", K);
        kind(out.t, "out", kx);
        return dg_moe_dispatch(x.data_ptr(), static_cast<int32_t*>(pointer(a[1], "pos", I32, {T, k})),
                               static_cast<int32_t*>(optional(a[3], "m_indices", I32, {out.rows})), out.t.data_ptr(),
                               size(T, "x"), size(k, "pos"), size(K, "x"), size(out.rows, "out"), dtype_of(kx),
                               stream_of(a[4]));
    });
}

// x, pos, q, sf, m_indices, stream
PyObject* moe_dispatch_fp8(PyObject*, PyObject* const* a, Py_ssize_t n) {
    return guarded<6>(n, [&] {
        const at::Tensor& x = tensor(a[0], "x");
        const at::Tensor& pos = tensor(a[1], "pos");
        dims(x, "x", 2);
        dims(pos, "pos", 2);
        kind(x, "x", BF16);
        const int64_t T = x.size(0), K = x.size(1), k = pos.size(1);
        const Rows q(a[2], "q", K);
        kind(q.t, "q", FP8);
        const int64_t Kp = (K / 128 + 3) / 4, al = (q.per + 3) / 4 * 4;
        void* sf = q.t.dim() == 3 ? pointer(a[3], "sf", I32, {q.groups, Kp, al}) : pointer(a[3], "sf", I32, {Kp, al});
        return dg_moe_dispatch_fp8(x.data_ptr(), static_cast<int32_t*>(pointer(a[1], "pos", I32, {T, k})),
                                   static_cast<int32_t*>(optional(a[4], "m_indices", I32, {q.rows})), q.t.data_ptr(),
                                   static_cast<int32_t*>(sf), size(T, "x"), size(k, "pos"), size(K, "x"), size(q.groups, "q"),
                                   size(q.per, "q"), stream_of(a[5]));
    });
}

// yp, pos, w, y, residual, stream
PyObject* moe_combine(PyObject*, PyObject* const* a, Py_ssize_t n) {
    return guarded<6>(n, [&] {
        const at::Tensor& y = tensor(a[3], "y");
        const at::Tensor& pos = tensor(a[1], "pos");
        dims(y, "y", 2);
        dims(pos, "pos", 2);
        const unsigned ky = kind(y, "y", BF16 | F32);
        const int64_t T = y.size(0), N = y.size(1), k = pos.size(1);
        const Rows yp(a[0], "yp", N);
        kind(yp.t, "yp", ky);
        return dg_moe_combine(yp.t.data_ptr(), static_cast<int32_t*>(pointer(a[1], "pos", I32, {T, k})),
                              static_cast<float*>(optional(a[2], "w", F32, {T, k})),
                              optional(a[4], "residual", ky, {T, N}), y.data_ptr(), size(T, "y"), size(k, "pos"),
                              size(N, "y"), size(yp.rows, "yp"), dtype_of(ky), stream_of(a[5]));
    });
}

// dy, yp, pos, w, dyp, dw, m_indices, stream
PyObject* moe_combine_backward(PyObject*, PyObject* const* a, Py_ssize_t n) {
    return guarded<8>(n, [&] {
        const at::Tensor& dy = tensor(a[0], "dy");
        const at::Tensor& pos = tensor(a[2], "pos");
        dims(dy, "dy", 2);
        dims(pos, "pos", 2);
        const unsigned kd = kind(dy, "dy", BF16 | F32);
        const int64_t T = dy.size(0), N = dy.size(1), k = pos.size(1);
        const Rows dyp(a[4], "dyp", N);
        kind(dyp.t, "dyp", kd);
        const void* yp = nullptr;
        if (a[1] != Py_None) {
            const Rows r(a[1], "yp", N);
            kind(r.t, "yp", kd);
            if (r.rows != dyp.rows) raise(PyExc_ValueError, "yp", "have as many rows as dyp");
            yp = r.t.data_ptr();
        }
        return dg_moe_combine_backward(dy.data_ptr(), yp, static_cast<int32_t*>(pointer(a[2], "pos", I32, {T, k})),
                                       static_cast<int32_t*>(optional(a[6], "m_indices", I32, {dyp.rows})),
                                       static_cast<float*>(optional(a[3], "w", F32, {T, k})), dyp.t.data_ptr(),
                                       static_cast<float*>(optional(a[5], "dw", F32, {T, k})), size(T, "dy"), size(k, "pos"),
                                       size(N, "dy"), size(dyp.rows, "dyp"), dtype_of(kd), stream_of(a[7]));
    });
}

// The operands of a GEMM, dense (G = 1), contiguous (b [G, N, K]) or masked (a [G, max_m, K] too).
struct Operands {
    const void *a, *b;
    const int32_t *sfa, *sfb;
    int64_t rows, N, K, G;
    Operands(PyObject* ao, PyObject* sao, PyObject* bo, PyObject* sbo, bool a_groups, bool b_groups) {
        const at::Tensor& at_ = tensor(ao, "a");
        const at::Tensor& bt = tensor(bo, "b");
        dims(at_, "a", a_groups ? 3 : 2);
        dims(bt, "b", b_groups ? 3 : 2);
        kind(at_, "a", FP8);
        kind(bt, "b", FP8);
        rows = at_.size(-2);
        K = at_.size(-1);
        N = bt.size(-2);
        G = b_groups ? bt.size(0) : 1;
        if (bt.size(-1) != K) raise(PyExc_ValueError, "b", "have rows as long as a's");
        if (a_groups && at_.size(0) != G) raise(PyExc_ValueError, "b", "have as many groups as a");
        a = at_.data_ptr();
        b = bt.data_ptr();
        const int64_t Kp = (K / 128 + 3) / 4;
        sfa = scales(sao, "sfa", a_groups ? G : 1, Kp * ((rows + 3) / 4 * 4));
        sfb = scales(sbo, "sfb", G, Kp * ((N + 3) / 4 * 4));
    }
    // Packed scales in any shape that has as many words.
    static const int32_t* scales(PyObject* o, const char* what, int64_t groups, int64_t words) {
        const at::Tensor& t = tensor(o, what);
        kind(t, what, I32);
        if (t.numel() != groups * words) raise(PyExc_ValueError, what, "hold the packed scales of its operand");
        return static_cast<const int32_t*>(t.data_ptr());
    }
};

struct Epilogue {
    void *bias, *residual, *z, *d;
    int act, bias_dtype = DG_BF16;
    Epilogue(PyObject* const* p, const Operands& o, bool a_groups, bool b_groups) {
        act = integer(p[4], "act");
        const int64_t H = act == DG_ACT_SWIGLU ? o.N / 2 : o.N;
        bias = nullptr;
        if (p[1] != Py_None) {
            bias_dtype = dtype_of(kind(tensor(p[1], "bias"), "bias", BF16 | F32));
            bias = b_groups ? pointer(p[1], "bias", BF16 | F32, {o.G, o.N}) : pointer(p[1], "bias", BF16 | F32, {o.N});
        }
        if (a_groups) {
            d = pointer(p[0], "d", BF16, {o.G, o.rows, H});
            residual = optional(p[2], "residual", BF16, {o.G, o.rows, H});
            z = optional(p[3], "z", BF16, {o.G, o.rows, o.N});
        } else {
            d = pointer(p[0], "d", BF16, {o.rows, H});
            residual = optional(p[2], "residual", BF16, {o.rows, H});
            z = optional(p[3], "z", BF16, {o.rows, o.N});
        }
    }
};

// a, sfa, b, sfb, d, bias, residual, z, act, stream
PyObject* gemm_act(PyObject*, PyObject* const* a, Py_ssize_t n) {
    return guarded<10>(n, [&] {
        const Operands o(a[0], a[1], a[2], a[3], false, false);
        const Epilogue e(a + 4, o, false, false);
        return dg_fp8_gemm_nt_act(o.a, o.sfa, o.b, o.sfb, e.bias, e.residual, e.z, e.d, size(o.rows, "a"), size(o.N, "b"),
                                  size(o.K, "a"), e.act, e.bias_dtype, stream_of(a[9]));
    });
}

// a, sfa, b, sfb, d, bias, residual, z, act, m_indices, stream
PyObject* gemm_contiguous_act(PyObject*, PyObject* const* a, Py_ssize_t n) {
    return guarded<11>(n, [&] {
        const Operands o(a[0], a[1], a[2], a[3], false, true);
        const Epilogue e(a + 4, o, false, true);
        return dg_m_grouped_fp8_gemm_nt_contiguous_act(
            o.a, o.sfa, o.b, o.sfb, e.bias, e.residual, e.z, e.d,
            static_cast<int32_t*>(pointer(a[9], "m_indices", I32, {o.rows})), size(o.rows, "a"), size(o.N, "b"),
            size(o.K, "a"), size(o.G, "b"), e.act, e.bias_dtype, stream_of(a[10]));
    });
}

// a, sfa, b, sfb, d, bias, residual, z, act, masked_m, stream
PyObject* gemm_masked_act(PyObject*, PyObject* const* a, Py_ssize_t n) {
    return guarded<11>(n, [&] {
        const Operands o(a[0], a[1], a[2], a[3], true, true);
        const Epilogue e(a + 4, o, true, true);
        return dg_m_grouped_fp8_gemm_nt_masked_act(
            o.a, o.sfa, o.b, o.sfb, e.bias, e.residual, e.z, e.d,
            static_cast<int32_t*>(pointer(a[9], "masked_m", I32, {o.G})), size(o.G, "a"), size(o.rows, "a"), size(o.N, "b"),
            size(o.K, "a"), e.act, e.bias_dtype, stream_of(a[10]));
    });
}

// dd, z, dz, act, dbias, workspace, m_indices, stream
PyObject* act_backward(PyObject*, PyObject* const* a, Py_ssize_t n) {
    return guarded<8>(n, [&] {
        const at::Tensor& z = tensor(a[1], "z");
        dims(z, "z", 2);
        kind(z, "z", BF16);
        const int act = integer(a[3], "act");
        const int64_t rows = z.size(0), N = z.size(1), H = act == DG_ACT_SWIGLU ? N / 2 : N;
        const bool grouped = a[6] != Py_None;
        int64_t G = 1;
        void* dbias = nullptr;
        if (a[4] != Py_None) {
            const at::Tensor& b = tensor(a[4], "dbias");
            if (grouped) {
                dims(b, "dbias", 2);
                G = b.size(0);
                dbias = pointer(a[4], "dbias", F32, {G, N});
            } else {
                dbias = pointer(a[4], "dbias", F32, {N});
            }
        }
        return dg_act_backward(pointer(a[0], "dd", BF16, {rows, H}), z.data_ptr(),
                               static_cast<int32_t*>(optional(a[6], "m_indices", I32, {rows})),
                               pointer(a[2], "dz", BF16, {rows, N}), static_cast<float*>(dbias),
                               static_cast<float*>(optional(a[5], "workspace", F32, {(rows + 127) / 128, N})),
                               size(rows, "z"), size(N, "z"), size(G, "dbias"), act, stream_of(a[7]));
    });
}

#define DG_METHOD(NAME) {#NAME, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(NAME)), METH_FASTCALL, nullptr}
PyMethodDef methods[] = {DG_METHOD(moe_route),        DG_METHOD(moe_route_backward), DG_METHOD(moe_sort),
                         DG_METHOD(moe_sort_masked),  DG_METHOD(moe_dispatch),       DG_METHOD(moe_dispatch_fp8),
                         DG_METHOD(moe_combine),      DG_METHOD(moe_combine_backward), DG_METHOD(gemm_act),
                         DG_METHOD(gemm_contiguous_act), DG_METHOD(gemm_masked_act), DG_METHOD(act_backward),
                         {nullptr, nullptr, 0, nullptr}};

PyModuleDef module = {PyModuleDef_HEAD_INIT, "dg_binding", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit_dg_binding() { return PyModule_Create(&module); }
