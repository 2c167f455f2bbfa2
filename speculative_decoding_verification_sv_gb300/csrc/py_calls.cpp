// py_calls.cpp -- the Python side of the cache and logits calls (a CPython
// extension over libsv.so's C ABI).
//
// These calls are short on the GPU (3 to 12 us at batch 1) and take eight to
// fifteen tensors each; checked and marshalled in Python they cost the host 12
// to 22 us.  Here the checks read the tensors directly.  What a call wants is
// written out in binding.py, whose functions these are; a tensor of another
// type, shape, device or layout is refused with TypeError or ValueError before
// anything is enqueued.
#include <Python.h>

#include <ATen/core/Tensor.h>
#include <ATen/ops/empty.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>
#include <torch/csrc/utils/object_ptr.h>

#include <array>
#include <cmath>
#include <utility>

#include "sv.h"

namespace {

PyObject* g_check = nullptr;   // binding._check(fn, status): raises SVError

const char* type_name(at::ScalarType t) {
    switch (t) {
        case at::kBFloat16: return "torch.bfloat16";
        case at::kFloat: return "torch.float32";
        case at::kInt: return "torch.int32";
        case at::kLong: return "torch.int64";
        case at::kByte: return "torch.uint8";
        default: return c10::toString(t);
    }
}

const at::Tensor& tensor(PyObject* o, const char* name) {
    TORCH_CHECK_TYPE(THPVariable_Check(o), name, " must be a tensor, got ", Py_TYPE(o)->tp_name);
    return THPVariable_Unpack(o);
}

// The call's first tensor: it names the device.
const at::Tensor& first(PyObject* o, const char* name, int64_t dims) {
    const at::Tensor& t = tensor(o, name);
    TORCH_CHECK_VALUE(t.is_cuda(), name, " must be a CUDA tensor");
    TORCH_CHECK_VALUE(t.dim() == dims, name, " must have ", dims, " dimensions, got shape ", t.sizes());
    return t;
}

const at::Tensor& dims_of(PyObject* o, const char* name, int64_t dims) {
    const at::Tensor& t = tensor(o, name);
    TORCH_CHECK_VALUE(t.dim() == dims, name, " must have ", dims, " dimensions, got shape ", t.sizes());
    return t;
}

struct Args {
    c10::Device device;

    void common(const at::Tensor& t, const char* name, at::ScalarType type, at::IntArrayRef shape) const {
        TORCH_CHECK_TYPE(t.scalar_type() == type, name, " must be ", type_name(type), ", got ", type_name(t.scalar_type()));
        TORCH_CHECK_VALUE(t.sizes() == shape, name, " must have shape ", shape, ", got ", t.sizes());
        TORCH_CHECK_VALUE(t.device() == device, name, " must be on ", device, ", got ", t.device());
    }
    // The pointer of an argument; None is NULL.
    void* get(PyObject* o, const char* name, at::ScalarType type, at::IntArrayRef shape) const {
        if (o == Py_None) return nullptr;
        const at::Tensor& t = tensor(o, name);
        common(t, name, type, shape);
        TORCH_CHECK_VALUE(t.is_contiguous(), name, " must be contiguous");
        return t.data_ptr();
    }
    template <typename T>
    T* as(PyObject* o, const char* name, at::ScalarType type, at::IntArrayRef shape) const {
        return static_cast<T*>(get(o, name, type, shape));
    }
    const int32_t* ints(PyObject* o, const char* name, at::IntArrayRef shape) const {
        return as<const int32_t>(o, name, at::kInt, shape);
    }
    const float* floats(PyObject* o, const char* name, at::IntArrayRef shape) const {
        return as<const float>(o, name, at::kFloat, shape);
    }
    uint16_t* bf16(PyObject* o, const char* name, at::IntArrayRef shape) const {
        return as<uint16_t>(o, name, at::kBFloat16, shape);
    }
    at::Tensor empty(at::IntArrayRef shape, at::ScalarType type) const {
        return at::empty(shape, at::TensorOptions().dtype(type).device(device));
    }
    void* stream() const { return c10::cuda::getCurrentCUDAStream(device.index()).stream(); }
};

bool truth(PyObject* o) {
    const int r = PyObject_IsTrue(o);
    if (r < 0) throw python_error();
    return r != 0;
}

double number(PyObject* o) {
    const double x = PyFloat_AsDouble(o);
    if (x == -1.0 && PyErr_Occurred()) throw python_error();
    return x;
}

int64_t whole(PyObject* o) {
    const long long x = PyLong_AsLongLong(o);
    if (x == -1 && PyErr_Occurred()) throw python_error();
    return x;
}

int32_t size32(int64_t n, const char* name) {
    TORCH_CHECK_VALUE(n >= 0 && n <= 2147483647, name, " is out of range: ", n);
    return static_cast<int32_t>(n);
}

// Lets other threads of the interpreter run.
struct Unlocked {
    PyThreadState* state = PyEval_SaveThread();
    ~Unlocked() { PyEval_RestoreThread(state); }
};

// Runs a C call without the interpreter's lock; raises on a status.
template <typename F>
void enqueue(const char* fn, F&& f) {
    sv_status s;
    {
        const Unlocked unlocked;
        s = f();
    }
    if (s == SV_OK) return;
    PyObject* r = PyObject_CallFunction(g_check, "si", fn, static_cast<int>(s));
    Py_XDECREF(r);
    if (r) PyErr_Format(PyExc_RuntimeError, "%s: status %d", fn, static_cast<int>(s));
    throw python_error();
}

void want(Py_ssize_t got, Py_ssize_t n) { TORCH_CHECK_TYPE(got == n, "expected ", n, " arguments, got ", got); }

// [N] rows of [Hkv][D] that may lie apart.
const uint16_t* rows(const Args& a, PyObject* o, const char* name, at::IntArrayRef shape, int64_t& stride) {
    const at::Tensor& t = tensor(o, name);
    a.common(t, name, at::kBFloat16, shape);
    TORCH_CHECK_VALUE((shape[2] <= 1 || t.stride(2) == 1) && (shape[1] <= 1 || t.stride(1) == shape[2]), name,
                      ": the heads of a row must be contiguous");
    stride = shape[0] > 1 ? t.stride(0) : shape[1] * shape[2];
    return static_cast<const uint16_t*>(t.data_ptr());
}

// (q4, k, v, row_off, k_pool, v_pool, page_table, length, rope, interleaved)
PyObject* kv_append(PyObject*, PyObject* const* o, Py_ssize_t n) {
    HANDLE_TH_ERRORS
    want(n, 10);
    const bool q4 = truth(o[0]);
    const at::Tensor& k = first(o[1], "k", 3);
    const Args a{k.device()};
    const c10::cuda::CUDAGuard guard(a.device);
    const int64_t N = k.size(0), H = k.size(1), D = k.size(2);
    TORCH_CHECK_VALUE(!q4 || D == 128, "a 4-bit cache holds rows of 128 dims, got ", D);
    int64_t ks, vs;
    const uint16_t* kp = rows(a, o[1], "k", {N, H, D}, ks);
    const uint16_t* vp = rows(a, o[2], "v", {N, H, D}, vs);
    const at::Tensor& table = dims_of(o[6], "page_table", 2);
    const int64_t B = table.size(0), max_pages = table.size(1);
    const int64_t P = dims_of(o[4], "k_pool", q4 ? 3 : 4).size(0);
    const int32_t* off = a.ints(o[3], "row_off", {B + 1});
    int64_t positions = 0, rot = 0;
    if (o[8] != Py_None) {
        const at::Tensor& rope = dims_of(o[8], "rope", 2);
        positions = rope.size(0), rot = rope.size(1);
    }
    const float* rp = a.floats(o[8], "rope", {positions, rot});
    const int32_t* tab = a.ints(o[6], "page_table", {B, max_pages});
    const int32_t* len = a.ints(o[7], "length", {B});
    const uint32_t flags = truth(o[9]) ? SV_ROPE_INTERLEAVED : 0u;
    const int32_t n32 = size32(N, "N"), b32 = size32(B, "B"), h32 = size32(H, "Hkv"), p32 = size32(P, "num_pages"),
                  m32 = size32(max_pages, "max_pages"), pos32 = size32(positions, "rope's positions"), r32 = size32(rot, "rot");
    if (q4) {
        void* kc = a.get(o[4], "k_pool", at::kByte, {P, H, SV_KV_Q4_BYTES});
        void* vc = a.get(o[5], "v_pool", at::kByte, {P, H, SV_KV_Q4_BYTES});
        enqueue("sv_kv_append_q4", [&] {
            return sv_kv_append_q4(kp, vp, ks, vs, n32, off, b32, h32, rp, pos32, r32, kc, vc, p32, tab, m32, len, flags,
                                   a.stream());
        });
    } else {
        uint16_t* kc = a.bf16(o[4], "k_pool", {P, H, SV_KV_PAGE, D});
        uint16_t* vc = a.bf16(o[5], "v_pool", {P, H, SV_KV_PAGE, D});
        const int32_t d32 = size32(D, "D");
        enqueue("sv_kv_append_paged", [&] {
            return sv_kv_append_paged(kp, vp, ks, vs, n32, off, b32, h32, d32, rp, pos32, r32, kc, vc, p32, tab, m32, len,
                                      flags, a.stream());
        });
    }
    Py_RETURN_NONE;
    END_HANDLE_TH_ERRORS
}

// (k_pool, v_pool, page_table, k_blk, v_blk, path, n_acc, length)
PyObject* kv_commit_q4(PyObject*, PyObject* const* o, Py_ssize_t n) {
    HANDLE_TH_ERRORS
    want(n, 8);
    const at::Tensor& blk = first(o[3], "k_blk", 5);
    const Args a{blk.device()};
    const c10::cuda::CUDAGuard guard(a.device);
    const int64_t L = blk.size(0), B = blk.size(1), H = blk.size(2), R = blk.size(3);
    const int64_t P = dims_of(o[0], "k_pool", 4).size(1), max_pages = dims_of(o[2], "page_table", 2).size(1);
    void* kp = a.get(o[0], "k_pool", at::kByte, {L, P, H, SV_KV_Q4_BYTES});
    void* vp = a.get(o[1], "v_pool", at::kByte, {L, P, H, SV_KV_Q4_BYTES});
    const int32_t* tab = a.ints(o[2], "page_table", {B, max_pages});
    const uint16_t* kb = a.bf16(o[3], "k_blk", {L, B, H, R, 128});
    const uint16_t* vb = a.bf16(o[4], "v_blk", {L, B, H, R, 128});
    const int32_t* path = a.ints(o[5], "path", {B, R});
    const int32_t* acc = a.ints(o[6], "n_acc", {B});
    int32_t* len = a.as<int32_t>(o[7], "length", at::kInt, {B});
    enqueue("sv_kv_commit_q4", [&] {
        return sv_kv_commit_q4(kp, vp, size32(P, "num_pages"), tab, size32(max_pages, "max_pages"), kb, vb, size32(L, "L"),
                               size32(B, "B"), size32(H, "Hkv"), size32(R, "R"), path, acc, len, a.stream());
    });
    Py_RETURN_NONE;
    END_HANDLE_TH_ERRORS
}

// An output: the one given, or a new tensor.
struct Output {
    void* ptr = nullptr;
    THPObjectPtr ref;
};
Output output(const Args& a, PyObject* o, const char* name, at::ScalarType type, at::IntArrayRef shape) {
    if (o != Py_None) {
        void* p = a.get(o, name, type, shape);
        Py_INCREF(o);
        return {p, THPObjectPtr(o)};
    }
    at::Tensor t = a.empty(shape, type);
    void* p = t.data_ptr();
    THPObjectPtr r(THPVariable_Wrap(std::move(t)));
    if (!r) throw python_error();
    return {p, std::move(r)};
}

// A tensor of its own over part of another's memory.
Output half_of(const at::Tensor& both, at::IntArrayRef shape, int64_t offset) {
    at::Tensor t = at::detail::make_tensor<c10::TensorImpl>(c10::Storage(both.storage()), both.key_set(), both.dtype());
    t.unsafeGetTensorImpl()->set_storage_offset(offset);
    t.unsafeGetTensorImpl()->set_sizes_contiguous(shape);
    void* p = t.data_ptr();
    THPObjectPtr r(THPVariable_Wrap(std::move(t)));
    if (!r) throw python_error();
    return {p, std::move(r)};
}

// (k_pool, v_pool, page_table, start, length, n, k_out, v_out) -> (k_out, v_out)
PyObject* kv_gather_q4(PyObject*, PyObject* const* o, Py_ssize_t n) {
    HANDLE_TH_ERRORS
    want(n, 8);
    const at::Tensor& pool = first(o[0], "k_pool", 4);
    const Args a{pool.device()};
    const c10::cuda::CUDAGuard guard(a.device);
    const int64_t L = pool.size(0), P = pool.size(1), H = pool.size(2), count = whole(o[5]);
    const at::Tensor& table = dims_of(o[2], "page_table", 2);
    const int64_t B = table.size(0), max_pages = table.size(1);
    const int32_t n32 = size32(count, "n");
    const void* kp = a.get(o[0], "k_pool", at::kByte, {L, P, H, SV_KV_Q4_BYTES});
    const void* vp = a.get(o[1], "v_pool", at::kByte, {L, P, H, SV_KV_Q4_BYTES});
    const int32_t* tab = a.ints(o[2], "page_table", {B, max_pages});
    const int32_t* start = a.ints(o[3], "start", {B});
    const int32_t* len = a.ints(o[4], "length", {B});
    const std::array<int64_t, 5> shape{L, B, H, count, 128};
    Output k, v;
    if (o[6] == Py_None && o[7] == Py_None) {   // both from one allocation
        const at::Tensor both = a.empty({2, L, B, H, count, 128}, at::kBFloat16);
        k = half_of(both, shape, 0);
        v = half_of(both, shape, both.numel() / 2);
    } else {
        k = output(a, o[6], "k_out", at::kBFloat16, shape);
        v = output(a, o[7], "v_out", at::kBFloat16, shape);
    }
    enqueue("sv_kv_gather_q4", [&] {
        return sv_kv_gather_q4(kp, vp, size32(P, "num_pages"), tab, size32(max_pages, "max_pages"), size32(L, "L"),
                               size32(B, "B"), size32(H, "Hkv"), start, len, n32, static_cast<uint16_t*>(k.ptr),
                               static_cast<uint16_t*>(v.ptr), a.stream());
    });
    return PyTuple_Pack(2, k.ref.get(), v.ref.get());
    END_HANDLE_TH_ERRORS
}

// (q, k_pool, v_pool, page_table, length, k_blk, v_blk, parent, scale, out, ws, cache_ready) -> out
PyObject* verify_attn_q4(PyObject*, PyObject* const* o, Py_ssize_t n) {
    HANDLE_TH_ERRORS
    want(n, 12);
    const at::Tensor& q = first(o[0], "q", 4);
    const Args a{q.device()};
    const c10::cuda::CUDAGuard guard(a.device);
    const int64_t B = q.size(0), R = q.size(1), Hq = q.size(2), D = q.size(3);
    const at::Tensor& pool = dims_of(o[1], "k_pool", 3);
    const int64_t P = pool.size(0), H = pool.size(1), max_pages = dims_of(o[3], "page_table", 2).size(1);
    const uint16_t* qp = a.bf16(o[0], "q", {B, R, Hq, D});
    const void* kp = a.get(o[1], "k_pool", at::kByte, {P, H, SV_KV_Q4_BYTES});
    const void* vp = a.get(o[2], "v_pool", at::kByte, {P, H, SV_KV_Q4_BYTES});
    const int32_t* tab = a.ints(o[3], "page_table", {B, max_pages});
    const int32_t* len = a.ints(o[4], "length", {B});
    const uint16_t* kb = a.bf16(o[5], "k_blk", {B, H, R, D});
    const uint16_t* vb = a.bf16(o[6], "v_blk", {B, H, R, D});
    const int32_t* par = a.ints(o[7], "parent", {B, R});
    const float scale = o[8] == Py_None ? static_cast<float>(1.0 / std::sqrt(static_cast<double>(D)))
                                        : static_cast<float>(number(o[8]));
    const uint32_t flags = truth(o[11]) ? SV_ATTN_CACHE_READY : 0u;
    const sv_attn_shape shape{size32(B, "B"), size32(R, "R"), size32(Hq, "Hq"), size32(H, "Hkv"), size32(D, "D"),
                              size32(max_pages * SV_KV_PAGE, "the page table's positions")};
    const size_t bytes = sv_verify_attn_q4_workspace(&shape);
    at::Tensor ws;
    if (bytes > 0 && o[10] != Py_None) {
        ws = tensor(o[10], "ws");
        TORCH_CHECK_VALUE(ws.device() == a.device && ws.is_contiguous() && ws.nbytes() >= bytes,
                          "ws must be contiguous, on ", a.device, " and hold ", bytes, " bytes");
    } else if (bytes > 0) {
        // This call's own until both of its launches are enqueued: a thread that makes a
        // call on the same stream can come between them.
        ws = a.empty({static_cast<int64_t>(bytes)}, at::kByte);
    }
    Output out = output(a, o[9], "out", at::kBFloat16, {B, R, Hq, D});
    enqueue("sv_verify_attn_q4", [&] {
        return sv_verify_attn_q4(&shape, qp, kp, vp, size32(P, "num_pages"), tab, size32(max_pages, "max_pages"), len, kb, vb,
                                 par, scale, static_cast<uint16_t*>(out.ptr), ws.defined() ? ws.data_ptr() : nullptr, bytes,
                                 flags, a.stream());
    });
    return out.ref.release();
    END_HANDLE_TH_ERRORS
}

// (logits, tok, parent, hist, hist_len, prompt_len, repetition, frequency, presence, bias_off, bias_tok, bias_val, mask,
//  mask_value, out, argmax, write_logits, write_argmax) -> (out or None, argmax or None)
PyObject* logits_process(PyObject*, PyObject* const* o, Py_ssize_t n) {
    HANDLE_TH_ERRORS
    want(n, 18);
    const at::Tensor& x = first(o[0], "logits", 3);
    const Args a{x.device()};
    const c10::cuda::CUDAGuard guard(a.device);
    const int64_t B = x.size(0), R = x.size(1), V = x.size(2), S = (V + SV_ARGMAX_SLAB - 1) / SV_ARGMAX_SLAB;
    const float* lp = a.floats(o[0], "logits", {B, R, V});
    int64_t cap = 0, nb = 0;
    if (o[3] != Py_None) {
        TORCH_CHECK_VALUE(o[4] != Py_None, "hist needs hist_len");
        cap = dims_of(o[3], "hist", 2).size(1);
    }
    if (o[9] != Py_None) {
        TORCH_CHECK_VALUE(o[10] != Py_None && o[11] != Py_None, "bias_off needs bias_tok and bias_val");
        nb = dims_of(o[10], "bias_tok", 1).size(0);
    }
    const int32_t* tok = a.ints(o[1], "tok", {B, R});
    const int32_t* par = a.ints(o[2], "parent", {B, R});
    const int32_t* hist = a.ints(o[3], "hist", {B, cap});
    const int32_t* hl = a.ints(o[4], "hist_len", {B});
    const int32_t* pl = a.ints(o[5], "prompt_len", {B});
    const float* rep = a.floats(o[6], "repetition", {B});
    const float* freq = a.floats(o[7], "frequency", {B});
    const float* pres = a.floats(o[8], "presence", {B});
    const int32_t* boff = a.ints(o[9], "bias_off", {B + 1});
    const int32_t* btok = a.ints(o[10], "bias_tok", {nb});
    const float* bval = a.floats(o[11], "bias_val", {nb});
    const auto* mask = reinterpret_cast<const uint32_t*>(a.ints(o[12], "mask", {B, R, (V + 31) / 32}));
    const auto mask_value = static_cast<float>(number(o[13]));
    Output out, keys;
    if (truth(o[16])) out = output(a, o[14], "out", at::kFloat, {B, R, V});
    if (o[15] != Py_None || truth(o[17])) keys = output(a, o[15], "argmax", at::kLong, {B * R, S});
    enqueue("sv_logits_process", [&] {
        return sv_logits_process(lp, size32(B, "B"), size32(R, "R"), size32(V, "V"), cap ? hist : nullptr, size32(cap, "hist's capacity"),
                                 hl, pl, tok, par, rep, freq, pres, boff, btok, bval, size32(nb, "the number of biases"), mask,
                                 mask_value, static_cast<float*>(out.ptr), static_cast<uint64_t*>(keys.ptr),
                                 keys.ptr ? static_cast<size_t>(B * R * S) * 8 : 0, a.stream());
    });
    return PyTuple_Pack(2, out.ref ? out.ref.get() : Py_None, keys.ref ? keys.ref.get() : Py_None);
    END_HANDLE_TH_ERRORS
}

// set_check(f): f(fn, status) raises what a status of the C ABI stands for
PyObject* set_check(PyObject*, PyObject* f) {
    Py_INCREF(f);
    Py_XDECREF(g_check);
    g_check = f;
    Py_RETURN_NONE;
}

#define SV_FAST(name) {#name, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(name)), METH_FASTCALL, nullptr}
PyMethodDef g_methods[] = {SV_FAST(kv_append),      SV_FAST(kv_commit_q4),   SV_FAST(kv_gather_q4),
                           SV_FAST(verify_attn_q4), SV_FAST(logits_process), {"set_check", set_check, METH_O, nullptr},
                           {nullptr, nullptr, 0, nullptr}};
PyModuleDef g_module = {PyModuleDef_HEAD_INIT, "sv_calls", nullptr, -1, g_methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

extern "C" __attribute__((visibility("default"))) PyObject* PyInit_sv_calls() { return PyModule_Create(&g_module); }
