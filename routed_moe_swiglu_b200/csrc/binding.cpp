// binding.cpp -- the short way from Python to the operators whose calls are
// shorter than reading their arguments through Python.
//
// A call of these operators takes up to eleven tensors.  Asking each for its
// type, shape, strides, device and address through Python attributes costs about
// 0.6 us a tensor, which with few tokens is more than the kernels take.  Here the
// tensors are read through DLPack's C exchange functions (a table that the tensor
// type offers as a capsule).  On one host, a call on the host alone: the losses
// 10.1 us before and 3.8 here, int8_linear of a token 10.7 and 3.9, of which the
// launch takes 2.5.
//
// A function of this module either finds every argument as its operator wants it,
// calls the entry point and returns the status, or does nothing and returns None:
// the caller then goes the long way, whose checks say what is wrong.  Nothing is
// accepted here that those refuse.
#define PY_SSIZE_T_CLEAN
#include <Python.h>

#include <cstdint>

#include "moe.h"

namespace {

// DLPack: a tensor as seen by C, and the table of exchange functions.
struct DlTensor {
    void* data;
    int32_t device_type, device_id;
    int32_t ndim;
    uint8_t code, bits;
    uint16_t lanes;
    const int64_t* shape;
    const int64_t* strides;
    uint64_t byte_offset;
};
struct DlExchange {
    uint32_t major, minor;
    const DlExchange* prev;
    void* allocate;
    void* managed_from_object;
    void* managed_to_object;
    int (*tensor_from_object)(void* object, DlTensor* out);                     // borrows; 0: fine
    int (*current_stream)(int32_t device_type, int32_t device_id, void** out);  // 0: fine
};
constexpr int32_t kCuda = 2;
constexpr uint8_t kInt = 0, kUInt = 1, kFloat = 2, kBfloat = 4;

const DlExchange* g_api = nullptr;
PyTypeObject *g_tensor = nullptr, *g_parameter = nullptr;

struct Entries {
    int (*get_device)(int*);  // cudaGetDevice
    decltype(&moe_plan_get_desc) plan_desc;
    decltype(&moe_balance_loss) balance_loss;
    decltype(&moe_route_backward) route_backward;
    decltype(&moe_combine_backward) combine_backward;
    decltype(&int8_quantize_rows) quantize_rows;
    decltype(&int8_matmul) matmul;
    decltype(&int8_linear) linear;
} g_lib;

struct Type {
    uint8_t code, bits;
};
constexpr Type kF32{kFloat, 32}, kBf16{kBfloat, 16}, kI32{kInt, 32}, kI8{kInt, 8}, kU8{kUInt, 8};

// The arguments of one call: `ok` stays true while all are as they should be.
struct Args {
    int32_t device = -1;  // the current one, asked for with the first tensor
    bool ok = true;

    DlTensor tensor(PyObject* o, Type type) {
        DlTensor d{};
        if (!ok) return d;
        if (Py_TYPE(o) != g_tensor && Py_TYPE(o) != g_parameter) {
            ok = false;
        } else if (g_api->tensor_from_object(o, &d) != 0) {
            PyErr_Clear();
            ok = false;
        } else {
            ok = d.device_type == kCuda && (device >= 0 || ask_device()) && d.device_id == device &&
                 d.code == type.code && d.bits == type.bits && d.lanes == 1 && d.data != nullptr &&
                 d.strides != nullptr;
        }
        return d;
    }
    bool ask_device() {
        int i = -1;
        if (g_lib.get_device(&i) != 0) return false;
        device = i;
        return true;
    }
    static void* at(const DlTensor& d) { return static_cast<char*>(d.data) + d.byte_offset; }
    // A dense tensor with its number of elements.
    DlTensor dense(PyObject* o, Type type, int64_t& count) {
        const DlTensor d = tensor(o, type);
        count = 1;
        if (!ok) return d;
        for (int i = d.ndim - 1; i >= 0; --i) {
            if (d.shape[i] != 1 && d.strides[i] != count) ok = false;
            count *= d.shape[i];
        }
        return d;
    }
    // Pointers (None: null, where it may be) of dense tensors: of at least `least` elements,
    void* items(PyObject* o, Type type, int64_t least, bool optional = false) {
        if (optional && o == Py_None) return nullptr;
        int64_t count;
        const DlTensor d = dense(o, type, count);
        ok = ok && count >= least;
        return ok ? at(d) : nullptr;
    }
    // of `rows` (at_least: or more) rows of `cols`,
    void* matrix(PyObject* o, Type type, int64_t rows, int64_t cols, bool at_least, bool optional = false) {
        if (optional && o == Py_None) return nullptr;
        int64_t count;
        const DlTensor d = dense(o, type, count);
        ok = ok && d.ndim == 2 && d.shape[1] == cols && (at_least ? d.shape[0] >= rows : d.shape[0] == rows);
        return ok ? at(d) : nullptr;
    }
    // of exactly `n` elements in one dimension.
    void* vector(PyObject* o, Type type, int64_t n, bool optional = false) {
        if (optional && o == Py_None) return nullptr;
        int64_t count;
        const DlTensor d = dense(o, type, count);
        ok = ok && d.ndim == 1 && d.shape[0] == n;
        return ok ? at(d) : nullptr;
    }
    // A matrix whose rows are dense, with its pitch.
    void* strided(PyObject* o, Type type, int64_t& rows, int64_t& cols, int64_t& ld) {
        const DlTensor d = tensor(o, type);
        ok = ok && d.ndim == 2 && d.strides[1] == 1;
        if (!ok) return nullptr;
        rows = d.shape[0];
        cols = d.shape[1];
        ld = rows > 1 ? d.strides[0] : cols;
        ok = cols <= INT32_MAX;
        return at(d);
    }
    int64_t whole(PyObject* o) {
        const long long v = PyLong_AsLongLong(o);
        if (v == -1 && PyErr_Occurred()) {
            PyErr_Clear();
            ok = false;
        }
        return v;
    }
    float number(PyObject* o) {
        if (!PyFloat_Check(o) && !PyLong_Check(o)) ok = false;
        const double v = ok ? PyFloat_AsDouble(o) : 0.0;
        if (PyErr_Occurred()) {
            PyErr_Clear();
            ok = false;
        }
        return static_cast<float>(v);
    }
    // The stream given, or the current one.
    void* stream(PyObject* o) {
        if (o != Py_None) return reinterpret_cast<void*>(static_cast<uintptr_t>(whole(o)));
        void* s = nullptr;
        if (ok && g_api->current_stream(kCuda, device, &s) != 0) {
            PyErr_Clear();
            ok = false;
        }
        return s;
    }
    const moe_plan* plan(PyObject* handle, moe_desc& d) {
        const moe_plan* p = reinterpret_cast<const moe_plan*>(static_cast<uintptr_t>(whole(handle)));
        if (ok && (p == nullptr || g_lib.plan_desc(p, &d) != MOE_OK)) ok = false;
        return p;
    }
};

// Calls f without the interpreter's lock and returns its status; None unless a.ok.
template <class F>
PyObject* finish(const Args& a, F f) {
    if (!a.ok) Py_RETURN_NONE;
    moe_status st;
    Py_BEGIN_ALLOW_THREADS st = f();
    Py_END_ALLOW_THREADS return PyLong_FromLong(st);
}

bool started(Py_ssize_t n, Py_ssize_t wanted) { return g_api != nullptr && n == wanted; }

// The functions' arguments (stream None: the current one; plan: its address).
//
// stream, plan, logits, ids, live, counts, prob_sums, lse, losses, grad_scales, workspace,
// balance_coef, z_coef, mask, offsets
PyObject* balance_loss(PyObject*, PyObject* const* v, Py_ssize_t n) {
    Args a;
    if (!started(n, 15)) Py_RETURN_NONE;
    moe_desc d;
    const moe_plan* p = a.plan(v[1], d);
    int64_t count = 0, bytes = 0;
    const DlTensor c = a.dense(v[5], kI32, count);
    if (!a.ok || c.ndim != 2 || c.shape[0] > INT32_MAX || c.shape[1] != d.num_experts) Py_RETURN_NONE;
    const int64_t S = c.shape[0], E = d.num_experts, k = d.top_k, rows = d.max_live_rows;
    const float* logits = static_cast<const float*>(a.matrix(v[2], kF32, rows, E, true));
    const int* ids = static_cast<const int*>(a.matrix(v[3], kI32, rows, k, true));
    const int* live = static_cast<const int*>(a.items(v[4], kI32, 1));
    float* sums = static_cast<float*>(a.matrix(v[6], kF32, S, E, false));
    float* lse = static_cast<float*>(a.items(v[7], kF32, rows));
    float* losses = static_cast<float*>(a.vector(v[8], kF32, 2));
    float* scales = static_cast<float*>(a.vector(v[9], kF32, S + 1));
    const DlTensor ws = a.dense(v[10], kU8, bytes);
    const float coef = a.number(v[11]), z = a.number(v[12]);
    const uint8_t* mask = static_cast<const uint8_t*>(a.items(v[13], kU8, rows, true));
    const int* off = static_cast<const int*>(a.vector(v[14], kI32, S + 1, true));
    void* s = a.stream(v[0]);
    return finish(a, [&] {
        return g_lib.balance_loss(p, logits, ids, mask, off, static_cast<int>(S), coef, z, live,
                                  static_cast<int*>(Args::at(c)), sums, lse, losses, scales, Args::at(ws),
                                  static_cast<size_t>(bytes), s);
    });
}

// stream, plan, logits, ids, live, dlogits, lse, counts, grad_scales, grad_losses, probs, dprobs, offsets
PyObject* route_backward(PyObject*, PyObject* const* v, Py_ssize_t n) {
    Args a;
    if (!started(n, 13)) Py_RETURN_NONE;
    moe_desc d;
    const moe_plan* p = a.plan(v[1], d);
    if (!a.ok) Py_RETURN_NONE;
    const int64_t E = d.num_experts, k = d.top_k, rows = d.max_live_rows;
    int64_t S = 1, count = 0;
    int* counts = nullptr;
    if (v[7] != Py_None) {
        const DlTensor c = a.dense(v[7], kI32, count);
        if (!a.ok || c.ndim != 2 || c.shape[0] > INT32_MAX || c.shape[1] != E) Py_RETURN_NONE;
        S = c.shape[0];
        counts = static_cast<int*>(Args::at(c));
    }
    const float* logits = static_cast<const float*>(a.matrix(v[2], kF32, rows, E, true, true));
    const int* ids = static_cast<const int*>(a.matrix(v[3], kI32, rows, k, true, true));
    const int* live = static_cast<const int*>(a.items(v[4], kI32, 1));
    float* dlogits = static_cast<float*>(a.matrix(v[5], kF32, rows, E, true));
    const float* lse = static_cast<const float*>(a.items(v[6], kF32, rows, true));
    const float* scales = static_cast<const float*>(a.vector(v[8], kF32, S + 1, true));
    const float* grads = static_cast<const float*>(a.vector(v[9], kF32, 2, true));
    const float* probs = static_cast<const float*>(a.matrix(v[10], kF32, rows, k, true, true));
    const float* dprobs = static_cast<const float*>(a.matrix(v[11], kF32, rows, k, true, true));
    // the chosen part alone knows no sequences
    const int* off = counts == nullptr ? nullptr : static_cast<const int*>(a.vector(v[12], kI32, S + 1, true));
    void* s = a.stream(v[0]);
    return finish(a, [&] {
        return g_lib.route_backward(p, logits, ids, lse, counts, scales, grads, probs, dprobs, off, static_cast<int>(S),
                                    live, dlogits, s);
    });
}

// stream, plan, dout, y_rows, route_rows, route_probs, live, dprobs, dy_rows
PyObject* combine_backward(PyObject*, PyObject* const* v, Py_ssize_t n) {
    Args a;
    if (!started(n, 9)) Py_RETURN_NONE;
    moe_desc d;
    const moe_plan* p = a.plan(v[1], d);
    if (!a.ok) Py_RETURN_NONE;
    const int64_t H = d.hidden, k = d.top_k, rows = d.max_live_rows;
    const void* dout = a.matrix(v[2], (d.flags & MOE_FLAG_OUT_BF16) != 0 ? kBf16 : kF32, rows, H, true);
    const float* y = static_cast<const float*>(a.matrix(v[3], kF32, 0, H, true, true));
    const int* route_rows = static_cast<const int*>(a.matrix(v[4], kI32, rows, k, true));
    const float* probs = static_cast<const float*>(a.matrix(v[5], kF32, rows, k, true));
    const int* live = static_cast<const int*>(a.items(v[6], kI32, 1));
    float* dprobs = static_cast<float*>(a.matrix(v[7], kF32, rows, k, true, true));
    float* dy = static_cast<float*>(a.matrix(v[8], kF32, 0, H, true, true));
    void* s = a.stream(v[0]);
    return finish(a, [&] { return g_lib.combine_backward(p, dout, y, route_rows, probs, live, dprobs, dy, s); });
}

// stream, x, q, scales, live_rows
PyObject* quantize_rows(PyObject*, PyObject* const* v, Py_ssize_t n) {
    Args a;
    if (!started(n, 5)) Py_RETURN_NONE;
    int64_t rows = 0, cols = 0, ld = 0;
    const void* x = a.strided(v[1], kBf16, rows, cols, ld);
    int8_t* q = static_cast<int8_t*>(a.matrix(v[2], kI8, rows, cols, false));
    float* scales = static_cast<float*>(a.vector(v[3], kF32, rows));
    const int* live = static_cast<const int*>(a.items(v[4], kI32, 1, true));
    void* s = a.stream(v[0]);
    return finish(a, [&] { return g_lib.quantize_rows(x, rows, static_cast<int>(cols), ld, q, scales, live, s); });
}

// What the two products share: wq, w_scales, out, live_rows, status.
struct Product {
    const int8_t* w = nullptr;
    const float* w_scales = nullptr;
    void* out = nullptr;
    const int* live = nullptr;
    unsigned* status = nullptr;
    int64_t N = 0, ld_out = 0;
    bool bf16 = false;

    Product(Args& a, PyObject* const* v, int64_t rows, int64_t K) {
        int64_t count = 0, out_rows = 0, out_cols = 0;
        const DlTensor d = a.dense(v[0], kI8, count);
        a.ok = a.ok && d.ndim == 2 && d.shape[1] == K && d.shape[0] <= INT32_MAX;
        if (!a.ok) return;
        w = static_cast<const int8_t*>(Args::at(d));
        N = d.shape[0];
        w_scales = static_cast<const float*>(a.vector(v[1], kF32, N));
        Args probe = a;  // out is fp32 or bf16
        out = probe.strided(v[2], kBf16, out_rows, out_cols, ld_out);
        bf16 = probe.ok;
        if (!bf16) out = a.strided(v[2], kF32, out_rows, out_cols, ld_out);
        a.ok = a.ok && out_rows == rows && out_cols == N;
        live = static_cast<const int*>(a.items(v[3], kI32, 1, true));
        status = static_cast<unsigned*>(a.items(v[4], kI32, 1, true));
    }
};

// stream, xq, x_scales, wq, w_scales, out, live_rows, status
PyObject* matmul(PyObject*, PyObject* const* v, Py_ssize_t n) {
    Args a;
    if (!started(n, 8)) Py_RETURN_NONE;
    int64_t rows = 0, K = 0, ld = 0;
    const int8_t* x = static_cast<const int8_t*>(a.strided(v[1], kI8, rows, K, ld));
    const float* x_scales = static_cast<const float*>(a.vector(v[2], kF32, rows));
    if (!a.ok) Py_RETURN_NONE;
    const Product m(a, v + 3, rows, K);
    void* s = a.stream(v[0]);
    return finish(a, [&] {
        return g_lib.matmul(x, x_scales, rows, static_cast<int>(K), ld, m.w, m.w_scales, static_cast<int>(m.N), m.out,
                            m.ld_out, m.bf16 ? 1 : 0, m.live, m.status, s);
    });
}

// stream, x, workspace, wq, w_scales, out, live_rows, status
PyObject* linear(PyObject*, PyObject* const* v, Py_ssize_t n) {
    Args a;
    if (!started(n, 8)) Py_RETURN_NONE;
    int64_t rows = 0, K = 0, ld = 0, bytes = 0;
    const void* x = a.strided(v[1], kBf16, rows, K, ld);
    const DlTensor ws = a.dense(v[2], kU8, bytes);
    if (!a.ok) Py_RETURN_NONE;
    const Product m(a, v + 3, rows, K);
    void* s = a.stream(v[0]);
    return finish(a, [&] {
        return g_lib.linear(x, rows, static_cast<int>(K), ld, m.w, m.w_scales, static_cast<int>(m.N), m.out, m.ld_out,
                            m.bf16 ? 1 : 0, m.live, Args::at(ws), static_cast<size_t>(bytes), m.status, s);
    });
}

// exchange capsule, tensor type, parameter type, then the entry points' addresses in the order of
// Entries; True when this module can serve, False (and no error) when it cannot.
PyObject* start_module(PyObject*, PyObject* const* v, Py_ssize_t n) {
    constexpr Py_ssize_t kEntries = sizeof(Entries) / sizeof(void*);
    if (n != 3 + kEntries || !PyType_Check(v[1]) || !PyType_Check(v[2])) Py_RETURN_FALSE;
    constexpr const char* kName = "dlpack_exchange_api";
    if (!PyCapsule_IsValid(v[0], kName)) Py_RETURN_FALSE;  // (sets no error)
    const DlExchange* api = static_cast<const DlExchange*>(PyCapsule_GetPointer(v[0], kName));
    if (api->major != 1 || api->tensor_from_object == nullptr || api->current_stream == nullptr) Py_RETURN_FALSE;
    uintptr_t at[kEntries];
    for (Py_ssize_t i = 0; i < kEntries; ++i) {
        at[i] = static_cast<uintptr_t>(PyLong_AsUnsignedLongLong(v[3 + i]));
        const bool wrong = PyErr_Occurred() != nullptr;
        PyErr_Clear();
        if (wrong || at[i] == 0) Py_RETURN_FALSE;
    }
    g_lib.get_device = reinterpret_cast<decltype(g_lib.get_device)>(at[0]);
    g_lib.plan_desc = reinterpret_cast<decltype(g_lib.plan_desc)>(at[1]);
    g_lib.balance_loss = reinterpret_cast<decltype(g_lib.balance_loss)>(at[2]);
    g_lib.route_backward = reinterpret_cast<decltype(g_lib.route_backward)>(at[3]);
    g_lib.combine_backward = reinterpret_cast<decltype(g_lib.combine_backward)>(at[4]);
    g_lib.quantize_rows = reinterpret_cast<decltype(g_lib.quantize_rows)>(at[5]);
    g_lib.matmul = reinterpret_cast<decltype(g_lib.matmul)>(at[6]);
    g_lib.linear = reinterpret_cast<decltype(g_lib.linear)>(at[7]);
    Py_INCREF(v[1]);
    Py_INCREF(v[2]);
    g_tensor = reinterpret_cast<PyTypeObject*>(v[1]);
    g_parameter = reinterpret_cast<PyTypeObject*>(v[2]);
    g_api = api;
    Py_RETURN_TRUE;
}

#define ENTRY(name, fn) {name, reinterpret_cast<PyCFunction>(reinterpret_cast<void*>(fn)), METH_FASTCALL, nullptr}
PyMethodDef kMethods[] = {ENTRY("start", start_module),
                          ENTRY("moe_balance_loss", balance_loss),
                          ENTRY("moe_route_backward", route_backward),
                          ENTRY("moe_combine_backward", combine_backward),
                          ENTRY("int8_quantize_rows", quantize_rows),
                          ENTRY("int8_matmul", matmul),
                          ENTRY("int8_linear", linear),
                          {nullptr, nullptr, 0, nullptr}};
PyModuleDef kModule = {PyModuleDef_HEAD_INIT, "_binding", nullptr, -1, kMethods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__binding() { return PyModule_Create(&kModule); }
