// Argument marshalling of the operators whose calls are as short as a launch (products by
// group, SwiGLU, int8 codes): reads the tensors' addresses, shapes and strides, checks what
// the C ABI cannot see (types, shapes, devices) and calls it.  Each function returns the
// moe_status; a tensor that does not fit raises ValueError before the call.
//
// Looking a tensor's properties up from Python takes half a microsecond a tensor and a
// ctypes call of fifteen arguments one and a half: together as long as the launch and the
// kernel of a decode step.  Here it is about a tenth of that.
#define PY_SSIZE_T_CLEAN
#include <Python.h>

#include <ATen/core/Tensor.h>
#include <torch/csrc/autograd/python_variable.h>

#include <string>

#include "../../include/moe.h"

namespace {

// The library's entry points, bound by address (the package loads the library itself).
struct {
    decltype(&moe_grouped_mm) grouped_mm;
    decltype(&moe_grouped_wgrad) grouped_wgrad;
    decltype(&moe_swiglu) swiglu;
    decltype(&moe_swiglu_backward) swiglu_backward;
    decltype(&moe_quantize_int8) quantize_int8;
    decltype(&moe_grouped_mm_int8) grouped_mm_int8;
} fn;

// Sets of element types.
enum : unsigned { F32 = 1, BF16 = 2, F16 = 4, I32 = 8, I8 = 16 };
constexpr unsigned kHalves = BF16 | F16, kFloats = F32 | BF16 | F16;

unsigned type_of(const at::Tensor& t) {
    switch (t.scalar_type()) {
        case at::kFloat: return F32;
        case at::kBFloat16: return BF16;
        case at::kHalf: return F16;
        case at::kInt: return I32;
        case at::kChar: return I8;
        default: return 0;
    }
}
moe_dtype code_of(unsigned t) { return t == F32 ? MOE_F32 : t == BF16 ? MOE_BF16 : MOE_F16; }

std::string text(at::IntArrayRef shape) {
    std::string s = "(";
    for (size_t i = 0; i < shape.size(); ++i) s += (i ? ", " : "") + std::to_string(shape[i]);
    return s + (shape.size() == 1 ? ",)" : ")");
}
std::string text(unsigned types) {
    static const char* names[] = {"float32", "bfloat16", "float16", "int32", "int8"};
    std::string s;
    for (int i = 0; i < 5; ++i)
        if (types >> i & 1) s += (s.empty() ? "" : " or ") + std::string(names[i]);
    return s;
}
bool refuse(const std::string& why) {
    PyErr_SetString(PyExc_ValueError, why.c_str());
    return false;
}

// What a call reads of its Python arguments.
struct Args {
    PyObject* const* a;
    long device;   // the current one

    const at::Tensor* tensor(int i, const char* name) const {
        if (!THPVariable_Check(a[i])) {
            refuse(std::string(name) + " must be a tensor");
            return nullptr;
        }
        return &THPVariable_Unpack(a[i]);
    }
    bool fits(const at::Tensor& t, const char* name, at::IntArrayRef shape, unsigned types) const {
        if (!t.is_cuda()) return refuse(std::string(name) + " must be a CUDA tensor");
        if (t.get_device() != device)
            return refuse(std::string(name) + " is on " + t.device().str() + ", the current device is cuda:" +
                          std::to_string(device));
        if (t.sizes() != shape) return refuse(std::string(name) + ": shape " + text(t.sizes()) + ", expected " + text(shape));
        if (!(type_of(t) & types))
            return refuse(std::string(name) + ": dtype " + std::string(toString(t.scalar_type())) + ", expected " + text(types));
        return true;
    }
    // Address of a contiguous tensor of the given shape and one of the types.
    bool dense(int i, const char* name, at::IntArrayRef shape, unsigned types, void** p) const {
        const at::Tensor* t = tensor(i, name);
        if (!t || !fits(*t, name, shape, types)) return false;
        if (!t->is_contiguous()) return refuse(std::string(name) + " must be contiguous");
        *p = t->data_ptr();
        return true;
    }
    bool optional(int i, const char* name, at::IntArrayRef shape, unsigned types, void** p) const {
        *p = nullptr;
        return a[i] == Py_None || dense(i, name, shape, types, p);
    }
    // Address and row distance of a matrix whose rows may lie apart (a slice of a wider buffer).
    bool rows(int i, const char* name, at::IntArrayRef shape, unsigned types, void** p, int64_t* ld) const {
        const at::Tensor* t = tensor(i, name);
        if (!t || !fits(*t, name, shape, types)) return false;
        if (t->stride(1) != 1 && shape[1] != 1) return refuse(std::string(name) + " must have contiguous rows");
        *p = t->data_ptr();
        if (shape[0] > 1) {
            *ld = t->stride(0);
        } else {  // one row or none: the stride says nothing
            const int64_t step = 16 / (int64_t)t->element_size();
            *ld = (shape[1] + step - 1) / step * step;
        }
        return true;
    }
    bool offsets(int i, int64_t groups, void** p) const {
        if (a[i] == Py_None) {
            *p = nullptr;
            return groups == 1 || refuse("offsets: only one group can go without");
        }
        return dense(i, "offsets", {groups + 1}, I32, p);
    }
    bool count(int i, void** p) const {
        *p = nullptr;
        if (a[i] == Py_None) return true;
        const at::Tensor* t = tensor(i, "n_rows");
        if (!t || !fits(*t, "n_rows", t->sizes(), I32)) return false;
        if (t->numel() != 1) return refuse("n_rows: shape " + text(t->sizes()) + ", expected one value");
        *p = t->data_ptr();
        return true;
    }
    bool flag(int i, int* v) const {
        *v = PyObject_IsTrue(a[i]);
        return *v >= 0;  // else the exception of its __bool__ is set
    }
    // two or three dimensions whose sizes the C ABI takes as int
    bool sizes(const at::Tensor& t, const char* name, int dims) const {
        if (t.dim() != dims) return refuse(std::string(name) + ": shape " + text(t.sizes()) + ", expected " + std::to_string(dims) + " dimensions");
        for (int64_t s : t.sizes())
            if (s > INT32_MAX) return refuse(std::string(name) + ": shape " + text(t.sizes()) + " is too large");
        return true;
    }
};

// device and stream are the last two arguments
bool open(PyObject* const* a, Py_ssize_t n, Py_ssize_t want, Args* args, moe_stream_t* stream) {
    if (n != want) return refuse("wrong number of arguments");
    args->a = a;
    args->device = PyLong_AsLong(a[n - 2]);
    if (args->device == -1 && PyErr_Occurred()) return false;
    *stream = static_cast<moe_stream_t>(PyLong_AsVoidPtr(a[n - 1]));
    return !PyErr_Occurred();
}

template <typename F>
PyObject* call(F f) {
    long st;
    Py_BEGIN_ALLOW_THREADS
    st = f();
    Py_END_ALLOW_THREADS
    return PyLong_FromLong(st);
}

const int32_t* i32(void* p) { return static_cast<const int32_t*>(p); }
float* f32(void* p) { return static_cast<float*>(p); }

// x, w, offsets, y, transpose_w, accumulate, device, stream
PyObject* grouped_mm(PyObject*, PyObject* const* a, Py_ssize_t nargs) {
    Args c;
    moe_stream_t s;
    if (!open(a, nargs, 8, &c, &s)) return nullptr;
    const at::Tensor *x = c.tensor(0, "x"), *w = x ? c.tensor(1, "w") : nullptr, *y = w ? c.tensor(3, "y") : nullptr;
    if (!y || !c.sizes(*w, "w", 3) || !c.sizes(*x, "x", 2)) return nullptr;
    int tr, acc;
    if (!c.flag(4, &tr) || !c.flag(5, &acc)) return nullptr;
    const int64_t G = w->size(0), n = w->size(tr ? 2 : 1), k = w->size(tr ? 1 : 2), R = x->size(0);
    const unsigned t = type_of(*w), out = type_of(*y);
    void *px, *pw, *po, *py;
    int64_t ldx, ldy;
    if (!c.dense(1, "w", w->sizes(), kHalves, &pw) || !c.rows(0, "x", {R, k}, t, &px, &ldx) ||
        !c.rows(3, "y", {R, n}, t | F32, &py, &ldy) || !c.offsets(2, G, &po))
        return nullptr;
    return call([&] {
        return fn.grouped_mm((int)G, (int)R, (int)n, (int)k, code_of(t), px, ldx, pw, tr, i32(po), py, ldy, code_of(out),
                             acc, s);
    });
}

// dy, x, offsets, dw, accumulate, device, stream
PyObject* grouped_wgrad(PyObject*, PyObject* const* a, Py_ssize_t nargs) {
    Args c;
    moe_stream_t s;
    if (!open(a, nargs, 7, &c, &s)) return nullptr;
    const at::Tensor *x = c.tensor(1, "x"), *dw = x ? c.tensor(3, "dw") : nullptr;
    if (!dw || !c.sizes(*dw, "dw", 3) || !c.sizes(*x, "x", 2)) return nullptr;
    int acc;
    if (!c.flag(4, &acc)) return nullptr;
    const int64_t G = dw->size(0), n = dw->size(1), k = dw->size(2), R = x->size(0);
    const unsigned t = type_of(*x), out = type_of(*dw);
    void *pdy, *px, *po, *pdw;
    int64_t lddy, ldx;
    if (!c.rows(1, "x", {R, k}, kHalves, &px, &ldx) || !c.rows(0, "dy", {R, n}, t, &pdy, &lddy) ||
        !c.dense(3, "dw", dw->sizes(), t | F32, &pdw) || !c.offsets(2, G, &po))
        return nullptr;
    return call([&] {
        return fn.grouped_wgrad((int)G, (int)R, (int)n, (int)k, code_of(t), pdy, lddy, px, ldx, i32(po), pdw, code_of(out),
                                acc, s);
    });
}

// gate, up, h, coef, n_rows, device, stream
PyObject* swiglu(PyObject*, PyObject* const* a, Py_ssize_t nargs) {
    Args c;
    moe_stream_t s;
    if (!open(a, nargs, 7, &c, &s)) return nullptr;
    const at::Tensor* g = c.tensor(0, "gate");
    if (!g || !c.sizes(*g, "gate", 2)) return nullptr;
    const at::IntArrayRef shape = g->sizes();
    const unsigned t = type_of(*g);
    void *pg, *pu, *ph, *pc, *pn;
    int64_t ldg, ldu, ldh;
    if (!c.rows(0, "gate", shape, kFloats, &pg, &ldg) || !c.rows(1, "up", shape, t, &pu, &ldu) ||
        !c.rows(2, "h", shape, t, &ph, &ldh) || !c.optional(3, "coef", {shape[0]}, F32, &pc) || !c.count(4, &pn))
        return nullptr;
    return call([&] {
        return fn.swiglu((int)shape[0], (int)shape[1], code_of(t), pg, ldg, pu, ldu, f32(pc), i32(pn), ph, ldh, s);
    });
}

// dh, gate, up, dgate, dup, coef, dcoef, n_rows, device, stream
PyObject* swiglu_backward(PyObject*, PyObject* const* a, Py_ssize_t nargs) {
    Args c;
    moe_stream_t s;
    if (!open(a, nargs, 10, &c, &s)) return nullptr;
    const at::Tensor* g = c.tensor(1, "gate");
    if (!g || !c.sizes(*g, "gate", 2)) return nullptr;
    const at::IntArrayRef shape = g->sizes();
    const unsigned t = type_of(*g);
    void *pd, *pg, *pu, *pdg, *pdu, *pc, *pdc, *pn;
    int64_t ldd, ldg, ldu, lddg, lddu;
    if (!c.rows(1, "gate", shape, kFloats, &pg, &ldg) || !c.rows(0, "dh", shape, t, &pd, &ldd) ||
        !c.rows(2, "up", shape, t, &pu, &ldu) || !c.rows(3, "dgate", shape, t, &pdg, &lddg) ||
        !c.rows(4, "dup", shape, t, &pdu, &lddu) || !c.optional(5, "coef", {shape[0]}, F32, &pc) ||
        !c.optional(6, "dcoef", {shape[0]}, F32, &pdc) || !c.count(7, &pn))
        return nullptr;
    return call([&] {
        return fn.swiglu_backward((int)shape[0], (int)shape[1], code_of(t), pd, ldd, pg, ldg, pu, ldu, f32(pc), i32(pn),
                                  pdg, lddg, pdu, lddu, f32(pdc), s);
    });
}

// x, q, sx, n_rows, device, stream
PyObject* quantize_int8(PyObject*, PyObject* const* a, Py_ssize_t nargs) {
    Args c;
    moe_stream_t s;
    if (!open(a, nargs, 6, &c, &s)) return nullptr;
    const at::Tensor* x = c.tensor(0, "x");
    if (!x || !c.sizes(*x, "x", 2)) return nullptr;
    const at::IntArrayRef shape = x->sizes();
    const unsigned t = type_of(*x);
    void *px, *pq, *ps, *pn;
    int64_t ldx;
    if (!c.rows(0, "x", shape, kFloats, &px, &ldx) || !c.dense(1, "q", shape, I8, &pq) ||
        !c.dense(2, "sx", {shape[0]}, F32, &ps) || !c.count(3, &pn))
        return nullptr;
    return call([&] {
        return fn.quantize_int8(px, code_of(t), ldx, (int)shape[0], (int)shape[1], i32(pn), static_cast<int8_t*>(pq),
                                f32(ps), s);
    });
}

// q, sx, w, sw, offsets, y, accumulate, device, stream
PyObject* grouped_mm_int8(PyObject*, PyObject* const* a, Py_ssize_t nargs) {
    Args c;
    moe_stream_t s;
    if (!open(a, nargs, 9, &c, &s)) return nullptr;
    const at::Tensor *q = c.tensor(0, "q"), *w = q ? c.tensor(2, "w") : nullptr, *y = w ? c.tensor(5, "y") : nullptr;
    if (!y || !c.sizes(*w, "w", 3) || !c.sizes(*q, "q", 2)) return nullptr;
    int acc;
    if (!c.flag(6, &acc)) return nullptr;
    const int64_t G = w->size(0), n = w->size(1), k = w->size(2), R = q->size(0);
    const unsigned out = type_of(*y);
    void *pq, *psx, *pw, *psw, *po, *py;
    int64_t ldy;
    if (!c.dense(0, "q", {R, k}, I8, &pq) || !c.dense(1, "sx", {R}, F32, &psx) || !c.dense(2, "w", w->sizes(), I8, &pw) ||
        !c.dense(3, "sw", {G, n}, F32, &psw) || !c.rows(5, "y", {R, n}, kFloats, &py, &ldy) || !c.offsets(4, G, &po))
        return nullptr;
    return call([&] {
        return fn.grouped_mm_int8((int)G, (int)R, (int)n, (int)k, static_cast<const int8_t*>(pq), f32(psx),
                                  static_cast<const int8_t*>(pw), f32(psw), i32(po), py, ldy, code_of(out), acc, s);
    });
}

// the addresses of the library's entry points, in the order of `fn`
PyObject* bind(PyObject*, PyObject* const* a, Py_ssize_t n) {
    void** slots = reinterpret_cast<void**>(&fn);
    if (n != (Py_ssize_t)(sizeof(fn) / sizeof(void*))) return refuse("wrong number of entry points"), nullptr;
    for (Py_ssize_t i = 0; i < n; ++i) {
        slots[i] = PyLong_AsVoidPtr(a[i]);
        if (PyErr_Occurred()) return nullptr;
    }
    Py_RETURN_NONE;
}

// A tensor without strides or memory (sparse, meta) makes ATen throw: a ValueError as well.
template <PyObject* (*F)(PyObject*, PyObject* const*, Py_ssize_t)>
PyObject* guarded(PyObject* self, PyObject* const* a, Py_ssize_t n) {
    try {
        return F(self, a, n);
    } catch (const c10::Error& e) {
        refuse(e.what_without_backtrace());
    } catch (const std::exception& e) {
        refuse(e.what());
    }
    return nullptr;
}

#define FAST(name) \
    {#name, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(guarded<name>)), METH_FASTCALL, nullptr}
PyMethodDef methods[] = {FAST(grouped_mm), FAST(grouped_wgrad), FAST(swiglu), FAST(swiglu_backward), FAST(quantize_int8),
                         FAST(grouped_mm_int8), FAST(bind), {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_binding", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__binding() { return PyModule_Create(&module); }
