// The native half of the Python binding of zsmr_ops.h: checks torch tensors
// against each other and calls the C ABI with their addresses.
//
// The shortest calls take the GPU 3 us; the same checks in Python and a ctypes
// call take 5 us more than the launch itself, these about 1.  Only the CPython
// API is used: tensors are asked for their shape, strides, format and address
// through their Python attributes, so nothing depends on torch's C++ ABI.
//
// Every function takes its arguments by position, returns the library's status
// code, and raises ValueError for tensors that do not fit together.  All shapes
// are checked before the first address is taken.
#define PY_SSIZE_T_CLEAN
#include <Python.h>

#include <cstdint>

#include "zsmr_ops.h"

namespace {

PyObject *n_shape, *n_dtype, *n_stride, *n_data_ptr, *n_is_cuda, *n_is_contiguous, *n_element_size;
PyObject *t_fp16, *t_bf16, *t_fp32, *t_fp64, *t_int32, *t_int64;
PyObject *f_stream, *f_device;          // torch's current raw stream of a device, current device

struct Error {};                        // a Python exception is set
[[noreturn]] void fail() { throw Error{}; }

struct Ref {                            // an owned reference
    PyObject* p;
    explicit Ref(PyObject* q) : p(q) {
        if (!p) fail();
    }
    ~Ref() { Py_DECREF(p); }
    Ref(const Ref&) = delete;
    Ref& operator=(const Ref&) = delete;
};

int64_t as_int(PyObject* x) {
    const long long v = PyLong_AsLongLong(x);
    if (v == -1 && PyErr_Occurred()) {
        if (PyErr_ExceptionMatches(PyExc_OverflowError)) PyErr_Format(PyExc_ValueError, "%R is outside int64", x);
        fail();
    }
    return v;
}
int32_t as_int32(PyObject* x) {
    const int64_t v = as_int(x);
    if (v < INT32_MIN || v > INT32_MAX) {
        PyErr_Format(PyExc_ValueError, "%R is outside int32", x);
        fail();
    }
    return (int32_t)v;
}
double as_double(PyObject* x) {
    const double v = PyFloat_AsDouble(x);
    if (v == -1.0 && PyErr_Occurred()) fail();
    return v;
}
bool truth(PyObject* x) {
    const int v = PyObject_IsTrue(x);
    if (v < 0) fail();
    return v != 0;
}

int code_of(PyObject* dtype) {
    return dtype == t_bf16 ? ZSMR_BF16 : dtype == t_fp16 ? ZSMR_FP16 : dtype == t_fp32 ? ZSMR_FP32 : 0;
}

// Address of a tensor in device memory.
void* address(PyObject* x, const char* what) {
    if (PyLong_Check(x)) return (void*)(intptr_t)as_int(x);     // a raw address: the caller's to check
    Ref cuda(PyObject_GetAttr(x, n_is_cuda));
    if (cuda.p != Py_True) {
        PyErr_Format(PyExc_ValueError, "%s: a tensor in host memory was passed where device memory is required", what);
        fail();
    }
    Ref at(PyObject_CallMethodNoArgs(x, n_data_ptr));
    return (void*)(intptr_t)as_int(at.p);
}
bool none_or_raw(PyObject* x) { return x == Py_None || PyLong_Check(x); }

struct Shape {
    Ref size;
    Py_ssize_t dims;
    explicit Shape(PyObject* x) : size(PyObject_GetAttr(x, n_shape)), dims(PyTuple_Check(size.p) ? PyTuple_GET_SIZE(size.p) : -1) {
        if (dims < 0) {
            PyErr_SetString(PyExc_ValueError, "a tensor is required");
            fail();
        }
    }
    int64_t operator[](Py_ssize_t i) const { return as_int(PyTuple_GET_ITEM(size.p, i)); }
    int64_t numel() const {
        int64_t n = 1;
        for (Py_ssize_t i = 0; i < dims; ++i) n *= (*this)[i];
        return n;
    }
};

// A 16-bit matrix: rows x width, elements of a row contiguous.
struct Matrix {
    int64_t rows = 0, width = 0, stride = 0;
    int32_t dtype = 0;
    PyObject* x = nullptr;
    const char* what;
    Matrix(PyObject* t, const char* name, const Matrix* like = nullptr, int64_t need_rows = -1) : x(t), what(name) {
        Shape shape(t);
        Ref format(PyObject_GetAttr(t, n_dtype));
        dtype = code_of(format.p);
        if (shape.dims != 2 || (dtype != ZSMR_FP16 && dtype != ZSMR_BF16)) {
            PyErr_Format(PyExc_ValueError, "%s: a matrix of 16-bit values is required, got %S of %S", what, format.p, shape.size.p);
            fail();
        }
        rows = shape[0];
        width = shape[1];
        if (like && dtype != like->dtype) {
            PyErr_Format(PyExc_ValueError, "%s: %S, %s has another format", what, format.p, like->what);
            fail();
        }
        if (like && (rows != need_rows || width != like->width)) {
            PyErr_Format(PyExc_ValueError, "%s: %lld x %lld, %lld x %lld is required", what, (long long)rows, (long long)width,
                         (long long)need_rows, (long long)like->width);
            fail();
        }
        Ref strides(PyObject_CallMethodNoArgs(t, n_stride));
        stride = rows > 1 ? as_int(PyTuple_GET_ITEM(strides.p, 0)) : width;
        if (width > 1 && as_int(PyTuple_GET_ITEM(strides.p, 1)) != 1) {
            PyErr_Format(PyExc_ValueError, "%s: elements of a row must be contiguous", what);
            fail();
        }
        if (stride < width) {
            PyErr_Format(PyExc_ValueError, "%s: rows overlap", what);
            fail();
        }
    }
    void* at() const { return address(x, what); }
};

bool contiguous(PyObject* x) {
    Ref c(PyObject_CallMethodNoArgs(x, n_is_contiguous));
    return c.p == Py_True;
}

// Token ids: a contiguous vector of int32 or int64.
struct Ids {
    int64_t n = 0;
    int32_t bytes = 0;
    PyObject* x;
    explicit Ids(PyObject* t) : x(t) {
        Shape shape(t);
        Ref format(PyObject_GetAttr(t, n_dtype));
        bytes = format.p == t_int64 ? 8 : format.p == t_int32 ? 4 : 0;
        if (!bytes || shape.dims != 1 || !contiguous(t)) {
            PyErr_Format(PyExc_ValueError, "token ids: a contiguous vector of int32 or int64 is required, got %S of %S", format.p,
                         shape.size.p);
            fail();
        }
        n = shape[0];
    }
    void* at() const { return address(x, "token ids"); }
};

// A contiguous tensor of at least n elements of a format (NULL: any, n bytes);
// None and raw addresses are the caller's to check.
struct Vector {
    PyObject* x;
    const char* what;
    int64_t bytes = 0;
    Vector(PyObject* t, int64_t n, PyObject* dtype, const char* name) : x(t), what(name) {
        if (none_or_raw(t)) {
            bytes = t == Py_None ? 0 : INT64_MAX;       // of a workspace
            return;
        }
        Shape shape(t);
        int64_t have = shape.numel();
        if (!dtype) {
            Ref size(PyObject_CallMethodNoArgs(t, n_element_size));
            have = bytes = have * as_int(size.p);
        } else {
            Ref format(PyObject_GetAttr(t, n_dtype));
            if (format.p != dtype) {
                PyErr_Format(PyExc_ValueError, "%s: %S is required, got %S", what, dtype, format.p);
                fail();
            }
        }
        if (have < n || !contiguous(t)) {
            PyErr_Format(PyExc_ValueError, "%s: at least %lld contiguous %s are required, got %S", what, (long long)n,
                         dtype ? "elements" : "bytes", shape.size.p);
            fail();
        }
    }
    void* at() const { return x == Py_None ? nullptr : address(x, what); }
};

hipStream_t stream_of(PyObject* s) {
    if (s == Py_None) {
        Ref device(PyObject_CallNoArgs(f_device));
        Ref raw(PyObject_CallOneArg(f_stream, device.p));
        return (hipStream_t)(intptr_t)as_int(raw.p);
    }
    if (PyLong_Check(s)) return (hipStream_t)(intptr_t)as_int(s);
    Ref raw(PyObject_GetAttrString(s, "cuda_stream"));
    return (hipStream_t)(intptr_t)as_int(raw.p);
}

// The three arrays of a tensor list.
struct List {
    Py_buffer b[3]{};
    int held = 0, n = 0;
    List(PyObject* const* a) {
        const char* const kinds[3] = {"int64 addresses", "int64 numels", "int32 dtypes"};
        for (int i = 0; i < 3; ++i) {
            if (PyObject_GetBuffer(a[i], &b[i], PyBUF_FORMAT | PyBUF_C_CONTIGUOUS | PyBUF_ND)) {
                PyErr_Clear();
                refuse(kinds[i]);
            }
            ++held;
            const char f = b[i].format && b[i].format[1] == 0 ? b[i].format[0] : 0;
            const bool format = i < 2 ? f == 'l' || f == 'q' : f == 'i';
            if (b[i].ndim != 1 || !format || b[i].shape[0] != b[0].shape[0]) refuse(kinds[i]);
        }
        n = (int)b[0].shape[0];
    }
    void refuse(const char* kind) {
        release();
        PyErr_Format(PyExc_ValueError, "tensor list: three contiguous vectors of one length are required (%s)", kind);
        fail();
    }
    void release() {
        while (held) PyBuffer_Release(&b[--held]);
    }
    ~List() { release(); }
    void* const* ptrs() const { return static_cast<void* const*>(b[0].buf); }
    const int64_t* numels() const { return static_cast<const int64_t*>(b[1].buf); }
    const int32_t* dtypes() const { return static_cast<const int32_t*>(b[2].buf); }
};

typedef PyObject* const* Args;

int32_t embed_lookup(Args a) {          // table, ids, out, scale, stream
    Ids ids(a[1]);
    Matrix table(a[0], "table"), out(a[2], "out", &table, ids.n);
    const float scale = (float)as_double(a[3]);
    return zsmr_embed_lookup(table.at(), table.rows, table.width, table.stride, table.dtype, ids.at(), ids.bytes, ids.n, scale,
                             out.at(), out.stride, stream_of(a[4]));
}

int32_t embed_grad(Args a) {            // dout, ids, dtable, ws, scale, accumulate, stream
    Ids ids(a[1]);
    Matrix table(a[2], "dtable"), dout(a[0], "dout", &table, ids.n);
    Vector ws(a[3], 0, nullptr, "workspace");
    return zsmr_embed_grad(dout.at(), dout.stride, table.dtype, ids.at(), ids.bytes, ids.n, table.rows, table.width,
                           (float)as_double(a[4]), truth(a[5]), table.at(), table.stride, ws.at(), ws.bytes, stream_of(a[6]));
}

int32_t xent_forward(Args a) {          // x, w, labels, loss, lse, summary, ws, stream
    Ids labels(a[2]);
    Matrix w(a[1], "w"), x(a[0], "x", &w, labels.n);
    Vector loss(a[3], labels.n, t_fp32, "loss"), lse(a[4], labels.n, t_fp32, "lse"), summary(a[5], 3, t_fp32, "summary");
    Vector ws(a[6], 0, nullptr, "workspace");
    return zsmr_xent_forward(x.at(), x.stride, w.at(), w.stride, w.dtype, labels.at(), labels.bytes, labels.n, w.rows, w.width,
                             (float*)loss.at(), (float*)lse.at(), (float*)summary.at(), ws.at(), ws.bytes, stream_of(a[7]));
}

int32_t xent_backward(Args a) {         // x, w, labels, lse, dx, dw, ws, grad, scale, accumulate, stream
    Ids labels(a[2]);
    Matrix w(a[1], "w"), x(a[0], "x", &w, labels.n);
    // a gradient that is left out stands for its operand in the checks
    const bool has_dx = a[4] != Py_None, has_dw = a[5] != Py_None;
    Matrix dx(has_dx ? a[4] : a[0], "dx", &w, labels.n), dw(has_dw ? a[5] : a[1], "dw", &w, w.rows);
    Vector lse(a[3], labels.n, t_fp32, "lse"), grad(a[7], labels.n, t_fp32, "grad"), scale(a[8], 1, t_fp32, "scale");
    Vector ws(a[6], 0, nullptr, "workspace");
    return zsmr_xent_backward(x.at(), x.stride, w.at(), w.stride, w.dtype, labels.at(), labels.bytes, labels.n, w.rows, w.width,
                              (float*)lse.at(), (float*)grad.at(), (float*)scale.at(), has_dx ? dx.at() : nullptr, dx.stride,
                              has_dw ? dw.at() : nullptr, dw.stride, truth(a[9]), ws.at(), ws.bytes, stream_of(a[10]));
}

int32_t grad_norm(Args a) {             // addresses, numels, dtypes, max_norm, norm_coef, ws, eps, stream
    List list(a);
    Vector out(a[4], 2, t_fp32, "norm_coef"), ws(a[5], 0, nullptr, "workspace");
    return zsmr_grad_norm(list.ptrs(), list.numels(), list.dtypes(), list.n, as_double(a[3]), as_double(a[6]), (float*)out.at(),
                          ws.at(), ws.bytes, stream_of(a[7]));
}

int32_t clip_coef(Args a) {             // sums, n, max_norm, norm_coef, eps, stream
    const int64_t n = as_int(a[1]);
    Vector sums(a[0], n, t_fp64, "sums"), out(a[3], 2, t_fp32, "norm_coef");
    return zsmr_clip_coef((const double*)sums.at(), n, as_double(a[2]), as_double(a[4]), (float*)out.at(), stream_of(a[5]));
}

int32_t clip_grads(Args a) {            // addresses, numels, dtypes, coef, stream
    List list(a);
    Vector coef(a[3], 1, t_fp32, "coef");
    return zsmr_clip_grads(list.ptrs(), list.numels(), list.dtypes(), list.n, (const float*)coef.at(), stream_of(a[4]));
}

int32_t clip_flatten(Args a) {          // addresses, numels, dtypes, coef, flat, stream
    List list(a);
    Vector coef(a[3], 1, t_fp32, "coef");
    if (none_or_raw(a[4])) {
        PyErr_SetString(PyExc_ValueError, "flat: a tensor is required, which says the row's format and length");
        fail();
    }
    Ref format(PyObject_GetAttr(a[4], n_dtype));
    const int dtype = code_of(format.p);
    if (dtype != ZSMR_FP16 && dtype != ZSMR_BF16) {
        PyErr_Format(PyExc_ValueError, "flat: a contiguous fp16 or bf16 tensor is required, got %S", format.p);
        fail();
    }
    Vector flat(a[4], 0, format.p, "flat");
    const int64_t n = Shape(a[4]).numel();
    return zsmr_clip_flatten(list.ptrs(), list.numels(), list.dtypes(), list.n, (const float*)coef.at(), flat.at(), n, dtype,
                             stream_of(a[5]));
}

zsmr_ctx* context(PyObject* handle) { return handle == Py_None ? nullptr : (zsmr_ctx*)(intptr_t)as_int(handle); }

// Elements of the (rank, unit) piece, or 0 where the layout refuses the pair
// (the call itself then reports it).
int64_t piece_of(const zsmr_ctx* ctx, int32_t rank, int32_t unit) {
    int64_t n = 0;
    return zero_layout(ctx, rank, unit, nullptr, &n, nullptr) == ZSMR_OK ? n : 0;
}

int32_t reduce_shard_sumsq(Args a) {    // ctx, rank, unit, grads, stride, base, mean, g_out, sumsq, ws, stream
    zsmr_ctx* ctx = context(a[0]);
    const int32_t rank = as_int32(a[1]), unit = as_int32(a[2]);
    const int64_t stride = as_int(a[4]), base = as_int(a[5]), n = piece_of(ctx, rank, unit);
    zsmr_layout_info info{};
    int64_t reach = 0;                  // elements from the first one on; what the call refuses anyway reaches nothing
    if (n > 0 && base >= 0 && stride >= 0 && zero_layout_info(ctx, &info) == ZSMR_OK) {
        const __int128 all = (__int128)base + (__int128)(info.world - 1) * stride + n;
        reach = all > INT64_MAX / 4 ? INT64_MAX / 4 : (int64_t)all;
    }
    Vector grads(a[3], 2 * reach, nullptr, "grads"), g(a[7], 4 * n, nullptr, "g_out");
    Vector sumsq(a[8], 1, t_fp64, "sumsq"), ws(a[9], 0, nullptr, "workspace");
    return zero_reduce_shard_sumsq(ctx, rank, unit, grads.at(), stride, base, truth(a[6]), (float*)g.at(), (double*)sumsq.at(),
                                   ws.at(), ws.bytes, stream_of(a[10]));
}

int32_t clipped_step(Args a) {  // ctx, rank, unit, g, coef, master, m, v, p16, t, lr, beta1, beta2, eps, stream
    zsmr_ctx* ctx = context(a[0]);
    const int32_t rank = as_int32(a[1]), unit = as_int32(a[2]), t = as_int32(a[9]);
    const int64_t n = piece_of(ctx, rank, unit);
    Vector g(a[3], 4 * n, nullptr, "g"), coef(a[4], 1, t_fp32, "coef"), master(a[5], 4 * n, nullptr, "master");
    Vector m(a[6], 4 * n, nullptr, "m"), v(a[7], 4 * n, nullptr, "v"), p16(a[8], 2 * n, nullptr, "p16_dst");
    const zsmr_adam hp{as_double(a[10]), as_double(a[11]), as_double(a[12]), as_double(a[13])};
    return zero_clipped_step(ctx, rank, unit, (const float*)g.at(), (const float*)coef.at(), (float*)master.at(), (float*)m.at(),
                             (float*)v.at(), p16.at(), t, &hp, stream_of(a[14]));
}

template <int32_t (*F)(Args), int N>
PyObject* entry(PyObject*, PyObject* const* args, Py_ssize_t n) {
    if (n != N) return PyErr_Format(PyExc_TypeError, "%d arguments are required, got %zd", N, n);
    try {
        const int32_t code = F(args);
        return PyLong_FromLong(code);
    } catch (const Error&) {
        return nullptr;
    }
}

#define ENTRY(f, n) {#f, (PyCFunction)(void (*)(void))entry<f, n>, METH_FASTCALL, nullptr}
PyMethodDef methods[] = {ENTRY(embed_lookup, 5),  ENTRY(embed_grad, 7),   ENTRY(xent_forward, 8),        ENTRY(xent_backward, 11),
                         ENTRY(grad_norm, 8),     ENTRY(clip_coef, 6),    ENTRY(clip_grads, 5),          ENTRY(clip_flatten, 6),
                         ENTRY(reduce_shard_sumsq, 11), ENTRY(clipped_step, 15), {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_ops", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__ops(void) {
    try {
        struct {
            PyObject** to;
            const char* name;
        } const names[] = {{&n_shape, "shape"},       {&n_dtype, "dtype"},     {&n_stride, "stride"},
                           {&n_data_ptr, "data_ptr"}, {&n_is_cuda, "is_cuda"}, {&n_is_contiguous, "is_contiguous"},
                           {&n_element_size, "element_size"}},
          types[] = {{&t_fp16, "float16"}, {&t_bf16, "bfloat16"}, {&t_fp32, "float32"},
                     {&t_fp64, "float64"}, {&t_int32, "int32"},   {&t_int64, "int64"}};
        for (const auto& n : names)
            if (!(*n.to = PyUnicode_InternFromString(n.name))) fail();
        Ref torch(PyImport_ImportModule("torch")), c(PyObject_GetAttrString(torch.p, "_C"));
        for (const auto& t : types)
            if (!(*t.to = PyObject_GetAttrString(torch.p, t.name))) fail();
        if (!(f_stream = PyObject_GetAttrString(c.p, "_cuda_getCurrentRawStream"))) fail();
        if (!(f_device = PyObject_GetAttrString(c.p, "_cuda_getDevice"))) fail();
        return PyModule_Create(&module);
    } catch (const Error&) {
        return nullptr;
    }
}
