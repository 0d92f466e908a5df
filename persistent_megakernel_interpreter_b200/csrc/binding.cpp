// The binding of the calls that a decode loop makes between steps (beam selection, cache
// reordering, the 8-bit cache): argument checks and marshalling only, as in the
// ctypes binding, but in compiled code. Their kernels take 1 to 6 us where little is to
// be moved, and checking eight tensors in Python and passing them through ctypes takes
// as long again (measured: 7.0 us a call against 3.5).
//
// Each call returns the library's mk_status; a tensor of the wrong type, device or
// size raises AssertionError before the library is called.
#define PY_SSIZE_T_CLEAN
#include <Python.h>

#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/autograd/python_variable.h>

#include <exception>
#include <stdexcept>

#include "mk.h"

namespace {

// A Python error is set.
struct Refused {};

[[noreturn]] void refuse(const char* name, const char* why) {
    PyErr_Format(PyExc_AssertionError, "%s: %s", name, why);
    throw Refused{};
}

const at::Tensor& tensor(PyObject* o, const char* name) {
    if (!THPVariable_Check(o)) refuse(name, "a tensor is wanted");
    return THPVariable_Unpack(o);
}

void check(const at::Tensor& t, const char* name, c10::ScalarType type, int device) {
    if (t.scalar_type() != type) refuse(name, "a tensor of another type is wanted");
    if (!t.is_cuda() || t.get_device() != device) refuse(name, "a tensor on the calling thread's current CUDA device is wanted");
}

// The address of a contiguous tensor of at least n elements on the device.
template <class T>
T* at_least(PyObject* o, const char* name, c10::ScalarType type, int64_t n, int device) {
    const at::Tensor& t = tensor(o, name);
    check(t, name, type, device);
    if (t.numel() < n || !t.is_contiguous()) refuse(name, "a contiguous tensor with more elements is wanted");
    return static_cast<T*>(t.data_ptr());
}
template <class T>
T* at_least_or_null(PyObject* o, const char* name, c10::ScalarType type, int64_t n, int device) {
    return o == Py_None ? nullptr : at_least<T>(o, name, type, n, device);
}

long number(PyObject* o, const char* name) {
    const long v = PyLong_AsLong(o);
    if (v == -1 && PyErr_Occurred()) throw Refused{};
    if (v > INT32_MAX || v < INT32_MIN) refuse(name, "the number is out of range");
    return v;
}

// The given torch.cuda.Stream, or the device's current one.
void* stream_of(PyObject* o, int device) {
    if (o == Py_None) return c10::cuda::getCurrentCUDAStream((c10::DeviceIndex)device).stream();
    PyObject* raw = PyObject_GetAttrString(o, "cuda_stream");
    if (!raw) throw Refused{};
    void* s = PyLong_AsVoidPtr(raw);
    Py_DECREF(raw);
    if (!s && PyErr_Occurred()) throw Refused{};
    return s;
}

// The calling thread's current device, where everything has to be; asked for only when there is a CUDA tensor.
int device_of(const at::Tensor& t, const char* name) {
    if (!t.is_cuda()) refuse(name, "a tensor on the calling thread's current CUDA device is wanted");
    return (int)c10::cuda::current_device();
}

const mk_qcache* qcache_of(PyObject* address, PyObject* device, int current) {
    const void* p = PyLong_AsVoidPtr(address);
    if (!p && PyErr_Occurred()) throw Refused{};
    if (number(device, "cache") != current) refuse("cache", "it is not on the calling thread's current CUDA device");
    return static_cast<const mk_qcache*>(p);
}

// The library's call without the interpreter's lock: a launch may wait for the GPU, and the GPU for a host
// function of another thread.
template <class F>
mk_status unlocked(F&& call) {
    PyThreadState* state = PyEval_SaveThread();
    const mk_status st = call();
    PyEval_RestoreThread(state);
    return st;
}

template <class F>
PyObject* guarded(Py_ssize_t n, Py_ssize_t wanted, F&& body) {
    if (n != wanted) {
        PyErr_Format(PyExc_TypeError, "%zd arguments are wanted, got %zd", wanted, n);
        return nullptr;
    }
    try {
        return PyLong_FromLong((long)body());
    } catch (const Refused&) {
    } catch (const std::exception& e) {
        PyErr_SetString(PyExc_RuntimeError, e.what());
    } catch (...) {
        PyErr_SetString(PyExc_RuntimeError, "unknown error");
    }
    return nullptr;
}

constexpr c10::ScalarType kI32 = c10::ScalarType::Int, kF32 = c10::ScalarType::Float, kBf16 = c10::ScalarType::BFloat16,
                          kU8 = c10::ScalarType::Byte;

// logits, scores, next_tokens, parents, next_scores, finished, eos, next_finished, positions, stream[, status: a tensor
// or a device address]
PyObject* beam_select(PyObject*, PyObject* const* a, Py_ssize_t n) {
    return guarded(n, n == 11 ? 11 : 10, [&] {
        const at::Tensor &logits = tensor(a[0], "logits"), &scores = tensor(a[1], "scores"), &tokens = tensor(a[2], "next_tokens");
        const int device = device_of(logits, "logits");
        check(logits, "logits", kF32, device);
        if (logits.dim() != 2 || scores.dim() != 2 || tokens.dim() != 2)
            refuse("logits, scores, next_tokens", "two dimensions are wanted");
        const int64_t rows = logits.size(0), vocab = logits.size(1), batch = scores.size(0), beams = scores.size(1);
        const int64_t n_in = batch * beams, n_out = tokens.size(1), n_all = batch * n_out;
        if (rows != n_in) refuse("logits", "a row for each beam is wanted");
        if (tokens.size(0) != batch) refuse("next_tokens", "a row for each sequence is wanted");
        if (vocab > 1 && logits.stride(1) != 1) refuse("logits", "rows of consecutive elements are wanted");
        if (rows > INT32_MAX || vocab > INT32_MAX || n_out > INT32_MAX) refuse("logits", "it is too large");
        const float* sc = at_least<float>(a[1], "scores", kF32, n_in, device);
        const int32_t* fin = at_least_or_null<int32_t>(a[5], "finished", kI32, n_in, device);
        const int32_t eos = (int32_t)number(a[6], "eos");
        int32_t* tok = at_least<int32_t>(a[2], "next_tokens", kI32, n_all, device);
        int32_t* par = at_least<int32_t>(a[3], "parents", kI32, n_all, device);
        float* out = at_least<float>(a[4], "next_scores", kF32, n_all, device);
        int32_t* next_fin = at_least_or_null<int32_t>(a[7], "next_finished", kI32, n_all, device);
        int32_t* pos = at_least_or_null<int32_t>(a[8], "positions", kI32, n_in, device);
        void* stream = stream_of(a[9], device);
        const int32_t* status = nullptr;
        if (n == 11 && PyLong_Check(a[10])) {
            status = static_cast<const int32_t*>(PyLong_AsVoidPtr(a[10]));
            if (!status) refuse("status", "an address is wanted");
        } else if (n == 11) {
            status = at_least_or_null<int32_t>(a[10], "status", kI32, 1, device);
        }
        const float* x = static_cast<const float*>(logits.data_ptr());
        const int64_t stride = rows > 1 ? logits.stride(0) : vocab;
        return unlocked([&] {
            if (status)
                return mk_beam_select_checked(x, stride, (int)batch, (int)beams, (int)vocab, (int)n_out, sc, fin, eos, tok, par, out,
                                              next_fin, pos, status, stream);
            return mk_beam_select(x, stride, (int)batch, (int)beams, (int)vocab, (int)n_out, sc, fin, eos, tok, par, out, next_fin, pos,
                                  stream);
        });
    });
}

// k_cache, v_cache, parents, lengths, starts, stream
PyObject* cache_reorder(PyObject*, PyObject* const* a, Py_ssize_t n) {
    return guarded(n, 6, [&] {
        const at::Tensor &k = tensor(a[0], "k_cache"), &v = tensor(a[1], "v_cache");
        const int device = device_of(k, "k_cache");
        if (k.dim() != 5 || v.sizes() != k.sizes()) refuse("k_cache, v_cache", "[layers][rows][heads][max_seq][dim] of one shape is wanted");
        for (int i = 0; i < 5; ++i)
            if (k.size(i) > INT32_MAX) refuse("k_cache", "it is too large");
        mk_config cfg{};
        cfg.n_layers = (int32_t)k.size(0);
        cfg.max_batch = (int32_t)k.size(1);
        cfg.n_kv_heads = (int32_t)k.size(2);
        cfg.max_seq = (int32_t)k.size(3);
        cfg.head_dim = (int32_t)k.size(4);
        const int64_t rows = tensor(a[2], "parents").numel();
        if (rows > cfg.max_batch) refuse("parents", "it has more rows than the cache");
        void* kp = at_least<void>(a[0], "k_cache", kBf16, 0, device);
        void* vp = at_least<void>(a[1], "v_cache", kBf16, 0, device);
        const int32_t* par = at_least<int32_t>(a[2], "parents", kI32, rows, device);
        const int32_t* len = at_least<int32_t>(a[3], "lengths", kI32, rows, device);
        const int32_t* from = at_least_or_null<int32_t>(a[4], "starts", kI32, rows, device);
        void* stream = stream_of(a[5], device);
        return unlocked([&] { return mk_cache_reorder(&cfg, kp, vp, (int)rows, par, len, from, stream); });
    });
}

// cache, its device, k, v, positions, counts, first_layer, stream
PyObject* qcache_append(PyObject*, PyObject* const* a, Py_ssize_t n) {
    return guarded(n, 8, [&] {
        const at::Tensor &k = tensor(a[2], "k"), &v = tensor(a[3], "v");
        const int device = device_of(k, "k");
        const mk_qcache* c = qcache_of(a[0], a[1], device);
        check(k, "k", kBf16, device);
        check(v, "v", kBf16, device);
        if (k.dim() != 5 || v.sizes() != k.sizes() || k.size(2) != c->n_kv_heads || k.size(4) != c->head_dim || k.stride(4) != 1 ||
            v.stride(4) != 1)
            refuse("k, v", "[layers][rows][heads][tokens][dim] of one shape and the cache's heads is wanted");
        int64_t strides[4];
        for (int i = 0; i < 4; ++i) {
            // the stride of a dimension of one is any number
            strides[i] = k.size(i) > 1 ? k.stride(i) : 0;
            if (k.size(i) > 1 && v.stride(i) != k.stride(i)) refuse("k, v", "the same strides are wanted");
            if (k.size(i) > INT32_MAX) refuse("k", "it is too large");
        }
        const int first = (int)number(a[6], "first_layer");
        const int32_t* pos = at_least<int32_t>(a[4], "positions", kI32, k.size(1), device);
        const int32_t* cnt = at_least_or_null<int32_t>(a[5], "counts", kI32, k.size(1), device);
        void* stream = stream_of(a[7], device);
        const void *kp = k.data_ptr(), *vp = v.data_ptr();
        const int layers = (int)k.size(0), rows = (int)k.size(1), tokens = (int)k.size(3);
        return unlocked([&] { return mk_qcache_append(c, first, layers, rows, tokens, kp, vp, strides, pos, cnt, stream); });
    });
}

// cache, its device, parents, lengths, starts, stream
PyObject* qcache_reorder(PyObject*, PyObject* const* a, Py_ssize_t n) {
    return guarded(n, 6, [&] {
        const at::Tensor& parents = tensor(a[2], "parents");
        const int device = device_of(parents, "parents");
        const mk_qcache* c = qcache_of(a[0], a[1], device);
        const int64_t rows = parents.numel();
        if (rows > c->max_batch) refuse("parents", "it has more rows than the cache");
        const int32_t* par = at_least<int32_t>(a[2], "parents", kI32, rows, device);
        const int32_t* len = at_least<int32_t>(a[3], "lengths", kI32, rows, device);
        const int32_t* from = at_least_or_null<int32_t>(a[4], "starts", kI32, rows, device);
        void* stream = stream_of(a[5], device);
        return unlocked([&] { return mk_qcache_reorder(c, (int)rows, par, len, from, stream); });
    });
}

// cache, its device, layer, q, positions, out, max_ctx, workspace, stream[, lengths]
PyObject* qcache_attention(PyObject*, PyObject* const* a, Py_ssize_t n) {
    return guarded(n, n == 10 ? 10 : 9, [&] {
        const at::Tensor& q = tensor(a[3], "q");
        const int device = device_of(q, "q");
        const mk_qcache* c = qcache_of(a[0], a[1], device);
        if (q.dim() != 3 || q.size(2) != c->head_dim) refuse("q", "[rows][n_heads][the cache's dims] is wanted");
        const int64_t rows = q.size(0), heads = q.size(1), all = q.numel();
        if (rows > INT32_MAX || heads > INT32_MAX) refuse("q", "it is too large");
        const int layer = (int)number(a[2], "layer"), max_ctx = (int)number(a[6], "max_ctx");
        const float* qp = at_least<float>(a[3], "q", kF32, all, device);
        const int32_t* pos = at_least<int32_t>(a[4], "positions", kI32, rows, device);
        float* out = at_least<float>(a[5], "out", kF32, all, device);
        void* work = at_least_or_null<void>(a[7], "workspace", kU8, 1, device);
        const size_t size = work ? (size_t)THPVariable_Unpack(a[7]).numel() : 0;
        void* stream = stream_of(a[8], device);
        const int32_t* len = n == 10 ? at_least_or_null<int32_t>(a[9], "lengths", kI32, rows, device) : nullptr;
        return unlocked([&] {
            if (len)
                return mk_qcache_attention_prefix(c, layer, (int)rows, (int)heads, max_ctx, qp, pos, len, out, work, size, stream);
            return mk_qcache_attention(c, layer, (int)rows, (int)heads, max_ctx, qp, pos, out, work, size, stream);
        });
    });
}

// cache, rows, n_heads, max_ctx: the bytes of workspace an attention call needs
PyObject* qcache_attention_workspace(PyObject*, PyObject* const* a, Py_ssize_t n) {
    return guarded(n, 4, [&] {
        const void* c = PyLong_AsVoidPtr(a[0]);
        if (!c && PyErr_Occurred()) throw Refused{};
        return mk_qcache_attention_workspace(static_cast<const mk_qcache*>(c), (int)number(a[1], "rows"), (int)number(a[2], "n_heads"),
                                             (int)number(a[3], "max_ctx"));
    });
}

PyMethodDef methods[] = {
    {"beam_select", (PyCFunction)(void*)beam_select, METH_FASTCALL, nullptr},
    {"cache_reorder", (PyCFunction)(void*)cache_reorder, METH_FASTCALL, nullptr},
    {"qcache_append", (PyCFunction)(void*)qcache_append, METH_FASTCALL, nullptr},
    {"qcache_reorder", (PyCFunction)(void*)qcache_reorder, METH_FASTCALL, nullptr},
    {"qcache_attention", (PyCFunction)(void*)qcache_attention, METH_FASTCALL, nullptr},
    {"qcache_attention_workspace", (PyCFunction)(void*)qcache_attention_workspace, METH_FASTCALL, nullptr},
    {nullptr, nullptr, 0, nullptr},
};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_call", "Checked calls into libmk.so.", -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__call() { return PyModule_Create(&module); }
