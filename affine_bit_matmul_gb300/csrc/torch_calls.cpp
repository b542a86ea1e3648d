// The cache operators' calls with little work on the host: a small decode step's kernels
// take 2 to 8 us, and a call that reads its tensors in Python takes 15 to 20.
//
// Each function takes the arguments of the Python function of its name in order, checks
// them in the same way, allocates what is to be returned and calls the library's C
// function on the current stream.  It returns None, without having done anything,
// where something is not as it has to be or not usual (another device, empty tensors): the
// Python function then goes its own way, which says what is wrong.  Measured for 16 rows
// of qk_norm_rope: 19 us in Python, 5.6 through here, outputs and launch included.
#define PY_SSIZE_T_CLEAN
#include <Python.h>

#include <ATen/core/Tensor.h>
#include <ATen/ops/empty.h>
#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/autograd/python_variable.h>

#include <cmath>

#include "mxq.h"

namespace {

// The library's functions; it is loaded by the package.
struct Library {
    decltype(&mxq_qk_norm_rope) qk_norm_rope = nullptr;
    decltype(&mxq_kv_append) kv_append = nullptr;
    decltype(&mxq_kv_read) kv_read = nullptr;
    decltype(&mxq_kv_attention) kv_attention = nullptr;
    decltype(&mxq_kv_attention_workspace_bytes) workspace_bytes = nullptr;
} lib;

// An argument that is not what it should be ends the call with None.
struct Unusual {};

void need(bool ok) {
    if (!ok) throw Unusual();
}

struct Args {
    PyObject* const* at;
    int device = -1;

    bool none(int i) const { return at[i] == Py_None; }
    const at::Tensor& tensor(int i) {
        need(THPVariable_Check(at[i]));
        const at::Tensor& t = THPVariable_Unpack(at[i]);
        need(t.is_cuda());
        if (device < 0) device = t.get_device();
        need(t.get_device() == device);
        return t;
    }
    int whole(int i) const {
        need(PyLong_CheckExact(at[i]));
        int over = 0;
        const long v = PyLong_AsLongAndOverflow(at[i], &over);
        need(!over && v >= -0x7FFFFFFFL && v <= 0x7FFFFFFFL);
        return (int)v;
    }
    double real(int i) const {
        need(PyFloat_CheckExact(at[i]) || PyLong_CheckExact(at[i]));
        return PyFloat_AsDouble(at[i]);
    }
    bool truth(int i) const {
        need(PyBool_Check(at[i]));
        return at[i] == Py_True;
    }
    // contiguous, of `type`: its address
    void* flat(int i, at::ScalarType type) {
        const at::Tensor& t = tensor(i);
        need(t.scalar_type() == type && t.is_contiguous());
        return t.data_ptr();
    }
    void* flat_or_none(int i, at::ScalarType type) { return none(i) ? nullptr : flat(i, type); }
};

// bf16 [T, heads, D] with contiguous heads.
struct Heads {
    int T, H, D;
    long long row, head;
    void* at;
};

int small(int64_t n) {
    need(n >= 0 && n <= 0x7FFFFFFF);
    return (int)n;
}

Heads heads_of(const at::Tensor& t, bool out) {
    need(t.scalar_type() == at::kBFloat16 && t.dim() == 3);
    Heads r;
    r.T = small(t.size(0)), r.H = small(t.size(1)), r.D = small(t.size(2));
    need(r.T > 0 && r.H > 0 && r.D > 1 && t.stride(2) == 1);
    r.head = r.H <= 1 ? r.D : t.stride(1);
    r.row = r.T <= 1 ? (long long)r.H * r.D : t.stride(0);
    need(r.row % 8 == 0 && r.head % 8 == 0);
    if (out) {
        need(r.H <= 1 || r.head >= r.D);
        need(r.T <= 1 || r.row >= r.D);
        need(r.T <= 1 || r.H <= 1 || r.row >= r.H * r.head || r.head >= r.T * r.row);
    }
    r.at = t.data_ptr();
    return r;
}

struct Pages {
    int n, H, size;
    void* at;
};

Pages pages_of(Args& a, int i, int head_dim, int group) {
    const at::Tensor& t = a.tensor(i);
    need(t.scalar_type() == at::kByte && t.is_contiguous() && t.dim() == 3);
    need(head_dim == 64 || head_dim == 128 || head_dim == 256);
    need((group == 32 || group == 64 || group == 128) && group <= head_dim);
    const int block = small(t.size(2)), per = head_dim + 8 * (head_dim / group);
    Pages p;
    p.n = small(t.size(0)), p.H = small(t.size(1));
    need(p.n > 0 && p.H > 0 && block % per == 0);
    p.size = block / per;
    need(p.size == 16 || p.size == 32 || p.size == 64 || p.size == 128);
    p.at = t.data_ptr();
    return p;
}

void* stream_of(const Args& a) {
    need(c10::cuda::current_device() == a.device);
    return c10::cuda::getCurrentCUDAStream((c10::DeviceIndex)a.device).stream();
}

// A tensor for the call, beside `like`.
at::Tensor empty(at::IntArrayRef shape, const at::Tensor& like, at::ScalarType type) {
    return at::empty(shape, at::TensorOptions().device(like.device()).dtype(type));
}

PyObject* pair_of(PyObject* a, PyObject* b) {  // takes over both
    PyObject* r = PyTuple_Pack(2, a, b);
    Py_DECREF(a);
    Py_DECREF(b);
    return r;
}

// The object of argument i, or of a tensor that the call made.
PyObject* object_of(const Args& a, int i, const at::Tensor& made) {
    if (made.defined()) return THPVariable_Wrap(made);
    Py_INCREF(a.at[i]);
    return a.at[i];
}

// q, k, positions, inv_freq, q_weight, k_weight, eps, weight_offset, interleaved, rope_scale,
// q_out, k_out
PyObject* qk_norm_rope(Args& a) {
    const at::Tensor& qt = a.tensor(0);
    const Heads q = heads_of(qt, false);
    const bool with_k = !a.none(1);
    Heads k{};
    if (with_k) {
        k = heads_of(a.tensor(1), false);
        need(k.T == q.T && k.D == q.D);
    } else {
        need(a.none(5) && a.none(11));
    }
    void *positions = nullptr, *freq = nullptr;
    int rot = 0;
    if (!a.none(3)) {
        freq = a.flat(3, at::kFloat);
        positions = a.flat(2, at::kInt);
        const at::Tensor &f = a.tensor(3), &p = a.tensor(2);
        need(f.dim() == 1 && f.numel() > 0 && f.numel() <= 1024 && p.numel() == q.T);
        rot = 2 * (int)f.numel();
    }
    void* weight[2] = {};
    for (int i = 0; i < 2; ++i) {
        weight[i] = a.flat_or_none(4 + i, at::kBFloat16);
        if (weight[i]) need(a.tensor(4 + i).dim() == 1 && a.tensor(4 + i).numel() == q.D);
    }
    const double eps = a.real(6), offset = a.real(7), scale = a.real(9);
    const bool interleaved = a.truth(8);
    void* stream = stream_of(a);
    at::Tensor q_made, k_made;
    Heads qo{}, ko{};
    if (a.none(10)) {
        q_made = empty({q.T, q.H, q.D}, qt, at::kBFloat16);
        qo = heads_of(q_made, true);
    } else {
        qo = heads_of(a.tensor(10), true);
        need(qo.T == q.T && qo.H == q.H && qo.D == q.D);
    }
    if (with_k) {
        if (a.none(11)) {
            k_made = empty({k.T, k.H, k.D}, qt, at::kBFloat16);
            ko = heads_of(k_made, true);
        } else {
            ko = heads_of(a.tensor(11), true);
            need(ko.T == k.T && ko.H == k.H && ko.D == k.D);
        }
    }
    need(lib.qk_norm_rope(q.at, q.row, q.head, k.at, k.row, k.head, (const int32_t*)positions,
                          (const float*)freq, weight[0], weight[1], qo.at, qo.row, qo.head, ko.at, ko.row,
                          ko.head, q.T, q.H, k.H, q.D, rot, interleaved ? 1 : 0, (float)eps, (float)offset,
                          (float)scale, stream) == MXQ_OK);
    return pair_of(object_of(a, 10, q_made), object_of(a, 11, k_made));
}

// k, v, pages, slots, group_size, dev_status
PyObject* kv_append(Args& a) {
    const Heads k = heads_of(a.tensor(0), false), v = heads_of(a.tensor(1), false);
    need(v.T == k.T && v.H == k.H && v.D == k.D);
    const int group = a.whole(4);
    const Pages p = pages_of(a, 2, k.D, group);
    need(p.H == k.H);
    void* slots = a.flat(3, at::kInt);
    need(a.tensor(3).numel() == k.T);
    void* status = a.flat_or_none(5, at::kInt);
    need(lib.kv_append(k.at, k.row, k.head, v.at, v.row, v.head, p.at, (const int32_t*)slots, k.T, k.H, k.D,
                       p.n, p.size, group, (int32_t*)status, stream_of(a)) == MXQ_OK);
    Py_INCREF(a.at[2]);
    return a.at[2];
}

// pages, slots, head_dim, group_size, k_out, v_out, dev_status
PyObject* kv_read(Args& a) {
    const int D = a.whole(2), group = a.whole(3);
    const Pages p = pages_of(a, 0, D, group);
    const at::Tensor& like = a.tensor(0);
    void* slots = a.flat(1, at::kInt);
    const int T = small(a.tensor(1).numel());
    need(T > 0);
    void* stream = stream_of(a);
    at::Tensor made[2];
    void* out[2];
    for (int i = 0; i < 2; ++i) {
        if (a.none(4 + i)) {
            made[i] = empty({T, p.H, D}, like, at::kBFloat16);
            out[i] = made[i].data_ptr();
        } else {
            out[i] = a.flat(4 + i, at::kBFloat16);
            const at::Tensor& t = a.tensor(4 + i);
            need(t.dim() == 3 && t.size(0) == T && t.size(1) == p.H && t.size(2) == D);
        }
    }
    void* status = a.flat_or_none(6, at::kInt);
    need(lib.kv_read(p.at, (const int32_t*)slots, out[0], out[1], T, p.H, D, p.n, p.size, group,
                     (int32_t*)status, stream) == MXQ_OK);
    return pair_of(object_of(a, 4, made[0]), object_of(a, 5, made[1]));
}

// q, pages, page_table, ctx_lens, q_starts, max_q_len, group_size, scale, window, sinks, out, lse,
// workspace, dev_status
PyObject* kv_attention(Args& a) {
    const at::Tensor& qt = a.tensor(0);
    const Heads q = heads_of(qt, false);
    const int max_q = a.whole(5), group = a.whole(6), window = a.whole(8), sinks = a.whole(9);
    const Pages p = pages_of(a, 1, q.D, group);
    need(q.H % p.H == 0 && max_q > 0);
    void* table = a.flat(2, at::kInt);
    const at::Tensor& tt = a.tensor(2);
    need(tt.dim() == 2);
    const int S = small(tt.size(0)), max_pages = small(tt.size(1));
    void* lens = a.flat(3, at::kInt);
    need(a.tensor(3).numel() == S);
    void* starts = a.flat_or_none(4, at::kInt);
    if (starts)
        need(a.tensor(4).numel() == S + 1LL);
    else
        need(q.T == S && max_q == 1);
    const double scale = a.none(7) ? 1.0 / std::sqrt((double)q.D) : a.real(7);
    void* stream = stream_of(a);
    at::Tensor made, ws_made;
    void* out;
    if (a.none(10)) {
        made = empty({q.T, q.H, q.D}, qt, at::kBFloat16);
        out = made.data_ptr();
    } else {
        out = a.flat(10, at::kBFloat16);
        const at::Tensor& t = a.tensor(10);
        need(t.dim() == 3 && t.size(0) == q.T && t.size(1) == q.H && t.size(2) == q.D);
    }
    void* lse = a.flat_or_none(11, at::kFloat);
    if (lse) {
        const at::Tensor& t = a.tensor(11);
        need(t.dim() == 2 && t.size(0) == q.T && t.size(1) == q.H);
    }
    void* status = a.flat_or_none(13, at::kInt);
    void* ws;
    size_t ws_bytes;
    if (a.none(12)) {
        ws_bytes = lib.workspace_bytes(q.T, S, q.H, p.H, q.D, max_q);
        ws_made = empty({(int64_t)ws_bytes}, qt, at::kByte);
        ws = ws_made.data_ptr();
    } else {
        ws = a.flat(12, at::kByte);
        ws_bytes = (size_t)a.tensor(12).numel();
    }
    need(lib.kv_attention(q.at, q.row, q.head, p.at, (const int32_t*)table, (const int32_t*)lens,
                          (const int32_t*)starts, out, (float*)lse, q.T, S, q.H, p.H, q.D, p.n, max_pages,
                          p.size, group, max_q, (float)scale, window, sinks, ws, ws_bytes,
                          (int32_t*)status, stream) == MXQ_OK);
    return object_of(a, 10, made);
}

// No C++ exception leaves a call: torch's (out of memory, a failing CUDA call) end it with None as
// well, and the Python function meets and reports them.
template <PyObject* (*F)(Args&), int N>
PyObject* call(PyObject*, PyObject* const* at, Py_ssize_t n) {
    try {
        if (n == N) {
            Args a{at};
            PyObject* r = F(a);
            if (r) return r;
        }
    } catch (...) {
    }
    PyErr_Clear();
    Py_RETURN_NONE;
}

// Addresses of the five library functions.
PyObject* bind(PyObject*, PyObject* args) {
    unsigned long long at[5];
    if (!PyArg_ParseTuple(args, "KKKKK", &at[0], &at[1], &at[2], &at[3], &at[4])) return nullptr;
    lib.qk_norm_rope = (decltype(lib.qk_norm_rope))(uintptr_t)at[0];
    lib.kv_append = (decltype(lib.kv_append))(uintptr_t)at[1];
    lib.kv_read = (decltype(lib.kv_read))(uintptr_t)at[2];
    lib.kv_attention = (decltype(lib.kv_attention))(uintptr_t)at[3];
    lib.workspace_bytes = (decltype(lib.workspace_bytes))(uintptr_t)at[4];
    Py_RETURN_NONE;
}

#define MXQ_CALL(f, n) {#f, (PyCFunction)(void (*)(void))call<f, n>, METH_FASTCALL, nullptr}
PyMethodDef methods[] = {{"bind", bind, METH_VARARGS, nullptr},
                         MXQ_CALL(qk_norm_rope, 12),
                         MXQ_CALL(kv_append, 6),
                         MXQ_CALL(kv_read, 7),
                         MXQ_CALL(kv_attention, 14),
                         {nullptr, nullptr, 0, nullptr}};
#undef MXQ_CALL
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_calls", nullptr, -1, methods,
                      nullptr,               nullptr,  nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__calls(void) { return PyModule_Create(&module); }
