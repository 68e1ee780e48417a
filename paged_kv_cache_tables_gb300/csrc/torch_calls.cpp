// The Python side of the entry points that a serving loop calls once per layer
// or step: argument checks and marshalling of torch tensors, nothing else (the
// module _torch_calls, loaded by _binding.py).
//
// A decode step's kernels take a few microseconds, less than checking eight
// tensors and filling in twenty arguments from Python (8 to 11 us for one call
// on the host cores of a GB300 machine; 2.8 us from here).  Every function takes
// its arguments by position, returns the C entry point's status, and raises
// TypeError or ValueError for tensors that do not fit together.
#include <Python.h>

#include <ATen/core/Tensor.h>
#include <c10/cuda/CUDACachingAllocator.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/autograd/python_variable.h>

#include <cmath>
#include <cstdio>
#include <initializer_list>
#include <string>

#include "pkv.h"

namespace {

// A Python exception on its way to the interpreter.
struct Refused {
    PyObject *type;       // nullptr: already set
    std::string message;
};

[[noreturn]] void refuse(PyObject *type, const std::string &message) { throw Refused{type, message}; }

std::string shape_text(at::IntArrayRef s) {
    std::string r = "(";
    for (size_t i = 0; i < s.size(); ++i) r += (i ? ", " : "") + std::to_string(s[i]);
    return r + (s.size() == 1 ? ",)" : ")");
}

const at::Tensor &tensor(PyObject *o, const char *name) {
    if (!THPVariable_Check(o)) refuse(PyExc_TypeError, std::string(name) + " must be a CUDA tensor");
    return THPVariable_Unpack(o);
}

// The call's device: that of its leading tensor.
int device_of(const at::Tensor &t, const char *name) {
    if (!t.is_cuda()) refuse(PyExc_TypeError, std::string(name) + " must be a CUDA tensor");
    return t.get_device();
}

void check(const at::Tensor &t, const char *name, at::ScalarType type, at::IntArrayRef shape, int device) {
    if (t.scalar_type() != type)
        refuse(PyExc_TypeError, std::string(name) + " must be " + c10::toString(type) + ", got " + c10::toString(t.scalar_type()));
    if (t.sizes() != shape)
        refuse(PyExc_ValueError, std::string(name) + " must have shape " + shape_text(shape) + ", got " + shape_text(t.sizes()));
    if (!t.is_cuda() || t.get_device() != device)
        refuse(PyExc_ValueError, std::string(name) + " must be a CUDA tensor on the device of the others");
}

// Address of a contiguous tensor of this type, shape and device.
void *ptr(PyObject *o, const char *name, at::ScalarType type, at::IntArrayRef shape, int device) {
    const at::Tensor &t = tensor(o, name);
    check(t, name, type, shape, device);
    if (!t.is_contiguous()) refuse(PyExc_ValueError, std::string(name) + " must be contiguous");
    return t.data_ptr();
}

void *ptr_or_null(PyObject *o, const char *name, at::ScalarType type, at::IntArrayRef shape, int device) {
    return o == Py_None ? nullptr : ptr(o, name, type, shape, device);
}

// [T, heads, d] rows whose heads are contiguous within a token (a slice of a
// fused projection's rows will do): address, and elements between tokens.
struct Rows {
    void *p;
    int64_t stride;
};

Rows rows(PyObject *o, const char *name, at::ScalarType type, at::IntArrayRef shape, int device) {
    const at::Tensor &t = tensor(o, name);
    check(t, name, type, shape, device);
    const auto st = t.strides();
    if (shape[0] && (st[2] != 1 || (shape[1] > 1 && st[1] != shape[2])))
        refuse(PyExc_ValueError, std::string(name) + " must hold each token's heads contiguously");
    return {t.data_ptr(), shape[0] > 1 ? st[0] : shape[1] * shape[2]};
}

int dtype_code(at::ScalarType t, const char *name) {
    if (t == at::kHalf) return PKV_DTYPE_F16;
    if (t == at::kBFloat16) return PKV_DTYPE_BF16;
    if (t == at::kFloat) return PKV_DTYPE_F32;
    refuse(PyExc_TypeError, std::string(name) + " must be float16, bfloat16 or float32, got " + c10::toString(t));
}

at::IntArrayRef dims(const at::Tensor &t, const char *name, size_t n) {
    if (t.sizes().size() != n) refuse(PyExc_ValueError, std::string(name) + " must have " + std::to_string(n) + " dims");
    return t.sizes();
}

int size_arg(int64_t n, const char *name) {
    if (n > INT32_MAX) refuse(PyExc_ValueError, std::string(name) + " is too large");
    return (int)n;
}

int int_arg(PyObject *o, const char *name) {
    const long long v = PyLong_AsLongLong(o);   // takes what has __index__
    if (v == -1 && PyErr_Occurred()) throw Refused{nullptr, ""};
    if (v > INT32_MAX || v < INT32_MIN) refuse(PyExc_ValueError, std::string(name) + " does not fit 32 bits");
    return (int)v;
}

float float_arg(PyObject *o) {
    const double v = PyFloat_AsDouble(o);
    if (v == -1.0 && PyErr_Occurred()) throw Refused{nullptr, ""};
    return (float)v;
}

bool bool_arg(PyObject *o) {
    const int v = PyObject_IsTrue(o);
    if (v < 0) throw Refused{nullptr, ""};
    return v != 0;
}

// The stream to run on: the device's current one, or a torch stream given.
void *stream_arg(PyObject *o, int device) {
    if (o == Py_None) return c10::cuda::getCurrentCUDAStream((c10::DeviceIndex)device).stream();
    auto number = [&](const char *name) {
        PyObject *a = PyObject_GetAttrString(o, name);
        if (!a) throw Refused{nullptr, ""};
        const long long v = PyLong_AsLongLong(a);
        Py_DECREF(a);
        if (v == -1 && PyErr_Occurred()) throw Refused{nullptr, ""};
        return v;
    };
    if (number("device_index") != device)
        refuse(PyExc_ValueError, "the stream belongs to another device than the tensors");
    return reinterpret_cast<void *>((uintptr_t)number("cuda_stream"));
}

// Torch's memory for what is launched on a stream of the current device before
// this goes: what takes it next there runs behind that.
struct StreamMemory {
    void *p = nullptr;
    StreamMemory() = default;
    StreamMemory(const StreamMemory &) = delete;
    void *get(size_t bytes, void *stream) {
        return p = c10::cuda::CUDACachingAllocator::raw_alloc_with_stream(bytes, static_cast<cudaStream_t>(stream));
    }
    ~StreamMemory() {
        if (p) c10::cuda::CUDACachingAllocator::raw_delete(p);
    }
};

// The interpreter is free for other threads while this lives: a launch waits
// when the stream's queue is full.  Nothing of Python's may be used meanwhile.
class OtherThreads {
    PyThreadState *state_ = PyEval_SaveThread();

  public:
    OtherThreads() = default;
    OtherThreads(const OtherThreads &) = delete;
    ~OtherThreads() { PyEval_RestoreThread(state_); }
};

int *status_arg(PyObject *o, int device) {
    return static_cast<int *>(ptr_or_null(o, "dev_status", at::kInt, {1}, device));
}

using Args = PyObject *const *;

// Runs `body` (which returns a status) with C++ exceptions turned into Python's.
template <typename F>
PyObject *guarded(const char *name, Py_ssize_t n, Py_ssize_t wanted, F body) {
    if (n != wanted) {
        PyErr_Format(PyExc_TypeError, "%s takes %zd arguments, got %zd", name, wanted, n);
        return nullptr;
    }
    try {
        return PyLong_FromLong(body());
    } catch (const Refused &r) {
        if (r.type) PyErr_SetString(r.type, r.message.c_str());
    } catch (const std::exception &e) {
        PyErr_SetString(PyExc_RuntimeError, e.what());
    } catch (...) {
        PyErr_SetString(PyExc_RuntimeError, "unknown C++ exception");
    }
    return nullptr;
}

// What the two attention calls share.
struct Attention {
    int device;
    at::IntArrayRef q_shape, cache;
    at::ScalarType type, out_type;
    void *out, *q, *k, *v;
    int Hq, d, NB, Hkv, bs;
    Attention(PyObject *o_out, PyObject *o_q, PyObject *o_k, PyObject *o_v) {
        const at::Tensor &tq = tensor(o_q, "q"), &tout = tensor(o_out, "out"), &tk = tensor(o_k, "k_cache");
        device = device_of(tq, "q");
        q_shape = dims(tq, "q", 3);
        cache = dims(tk, "k_cache", 4);
        type = tq.scalar_type();
        out_type = tout.scalar_type();
        if (cache[3] != q_shape[2]) refuse(PyExc_ValueError, "q and the caches must have one head_dim");
        out = ptr(o_out, "out", out_type, q_shape, device);
        q = ptr(o_q, "q", type, q_shape, device);
        k = ptr(o_k, "k_cache", type, cache, device);
        v = ptr(o_v, "v_cache", type, cache, device);
        Hq = size_arg(q_shape[1], "q");
        d = size_arg(q_shape[2], "q");
        NB = size_arg(cache[0], "k_cache");
        Hkv = size_arg(cache[1], "k_cache");
        bs = size_arg(cache[2], "k_cache");
    }
    float scale(PyObject *o) const { return o == Py_None ? (float)(1.0 / std::sqrt((double)d)) : float_arg(o); }
};

// (out, q, k_cache, v_cache, block_tables, context_lens, window, num_sinks, scale, dev_status, stream)
PyObject *window_decode(PyObject *, Args a, Py_ssize_t n) {
    return guarded("window_decode", n, 11, [&] {
        const Attention t(a[0], a[1], a[2], a[3]);
        const int64_t S = t.q_shape[0], MB = dims(tensor(a[4], "block_tables"), "block_tables", 2)[1];
        void *tables = ptr(a[4], "block_tables", at::kInt, {S, MB}, t.device);
        void *ctx = ptr(a[5], "context_lens", at::kInt, {S}, t.device);
        const int max_blocks = size_arg(MB, "block_tables"), seqs = size_arg(S, "q");
        const int window = int_arg(a[6], "window"), sinks = int_arg(a[7], "num_sinks");
        const float scale = t.scale(a[8]);
        const int type = dtype_code(t.type, "q"), out_type = dtype_code(t.out_type, "out");
        int *status = status_arg(a[9], t.device);
        void *stream = stream_arg(a[10], t.device);
        OtherThreads run;
        c10::cuda::OptionalCUDAGuard guard(c10::Device(c10::kCUDA, (c10::DeviceIndex)t.device));
        return pkv_paged_window_decode_attention(t.out, t.q, t.k, t.v, static_cast<int32_t *>(tables), max_blocks,
                                                 static_cast<int32_t *>(ctx), seqs, t.NB, t.Hq, t.Hkv, t.d, t.bs, window,
                                                 sinks, scale, type, out_type, status, stream);
    });
}

// (out, q, cu_seqlens, max_q_len, k_cache, v_cache, block_tables, context_lens, window, num_sinks, scale, dev_status, stream)
PyObject *window_prefill(PyObject *, Args a, Py_ssize_t n) {
    return guarded("window_prefill", n, 13, [&] {
        const Attention t(a[0], a[1], a[4], a[5]);
        const auto tb = dims(tensor(a[6], "block_tables"), "block_tables", 2);
        const int64_t S = tb[0], MB = tb[1];
        void *cu = ptr(a[2], "cu_seqlens", at::kInt, {S + 1}, t.device);
        void *tables = ptr(a[6], "block_tables", at::kInt, {S, MB}, t.device);
        void *ctx = ptr(a[7], "context_lens", at::kInt, {S}, t.device);
        const int max_blocks = size_arg(MB, "block_tables"), seqs = size_arg(S, "block_tables");
        const int max_q = int_arg(a[3], "max_q_len"), total_q = size_arg(t.q_shape[0], "q");
        const int window = int_arg(a[8], "window"), sinks = int_arg(a[9], "num_sinks");
        const float scale = t.scale(a[10]);
        const int type = dtype_code(t.type, "q"), out_type = dtype_code(t.out_type, "out");
        int *status = status_arg(a[11], t.device);
        void *stream = stream_arg(a[12], t.device);
        OtherThreads run;
        c10::cuda::OptionalCUDAGuard guard(c10::Device(c10::kCUDA, (c10::DeviceIndex)t.device));
        return pkv_paged_window_prefill_attention(t.out, t.q, static_cast<int32_t *>(cu), seqs, max_q, total_q, t.k, t.v,
                                                  static_cast<int32_t *>(tables), max_blocks, static_cast<int32_t *>(ctx),
                                                  t.NB, t.Hq, t.Hkv, t.d, t.bs, window, sinks, scale, type, out_type,
                                                  status, stream);
    });
}

// What the two rotation calls share.
struct Rotation {
    int device;
    int64_t T, Hq, Hkv, d, pairs;
    at::ScalarType type, weight_type = at::kFloat;
    Rows q, k, q_out;
    const int32_t *positions;
    const int64_t *freqs;
    void *q_weight, *k_weight;
    int T_arg, Hq_arg, Hkv_arg, d_arg, rotary_dim, code, weight_code;   // as the C entry points take them
    Rotation(PyObject *o_q_out, PyObject *o_q, PyObject *o_k, PyObject *o_pos, PyObject *o_freqs, PyObject *o_wq,
             PyObject *o_wk) {
        const at::Tensor &tq = tensor(o_q, "q"), &tf = tensor(o_freqs, "freqs");
        device = device_of(tq, "q");
        const auto qs = dims(tq, "q", 3);
        T = qs[0], Hq = qs[1], d = qs[2];
        Hkv = dims(tensor(o_k, "k"), "k", 3)[1];
        type = tq.scalar_type();
        pairs = dims(tf, "freqs", 1)[0];
        q = rows(o_q, "q", type, {T, Hq, d}, device);
        k = rows(o_k, "k", type, {T, Hkv, d}, device);
        q_out = rows(o_q_out, "q_out", type, {T, Hq, d}, device);
        positions = static_cast<int32_t *>(ptr(o_pos, "positions", at::kInt, {T}, device));
        freqs = static_cast<int64_t *>(ptr(o_freqs, "freqs", at::kLong, {pairs}, device));
        if (o_wq != Py_None || o_wk != Py_None)
            weight_type = tensor(o_wq != Py_None ? o_wq : o_wk, "the weights").scalar_type();
        q_weight = ptr_or_null(o_wq, "q_weight", weight_type, {d}, device);
        k_weight = ptr_or_null(o_wk, "k_weight", weight_type, {d}, device);
        T_arg = size_arg(T, "q"), Hq_arg = size_arg(Hq, "q"), Hkv_arg = size_arg(Hkv, "k"), d_arg = size_arg(d, "q");
        rotary_dim = size_arg(2 * pairs, "freqs");
        code = dtype_code(type, "q"), weight_code = dtype_code(weight_type, "the weights");
    }
};

// (q_out, k_out, q, k, positions, freqs, interleaved, mscale, q_weight, k_weight, eps, stream)
PyObject *qk_rope(PyObject *, Args a, Py_ssize_t n) {
    return guarded("qk_rope", n, 12, [&] {
        const Rotation t(a[0], a[2], a[3], a[4], a[5], a[8], a[9]);
        const Rows k_out = rows(a[1], "k_out", t.type, {t.T, t.Hkv, t.d}, t.device);
        const bool interleaved = bool_arg(a[6]);
        const float mscale = float_arg(a[7]), eps = float_arg(a[10]);
        void *stream = stream_arg(a[11], t.device);
        OtherThreads run;
        c10::cuda::OptionalCUDAGuard guard(c10::Device(c10::kCUDA, (c10::DeviceIndex)t.device));
        return pkv_qk_rope(t.q_out.p, t.q_out.stride, k_out.p, k_out.stride, t.q.p, t.q.stride, t.k.p, t.k.stride,
                           t.positions, t.freqs, t.rotary_dim, interleaved, mscale, t.q_weight, t.k_weight, t.weight_code,
                           eps, t.T_arg, t.Hq_arg, t.Hkv_arg, t.d_arg, t.code, stream);
    });
}

// (q_out, q, k, v, positions, slot_mapping, freqs, k_cache, v_cache, interleaved, mscale, q_weight, k_weight, eps,
//  dev_status, stream)
PyObject *qk_rope_append(PyObject *, Args a, Py_ssize_t n) {
    return guarded("qk_rope_append", n, 16, [&] {
        const Rotation t(a[0], a[1], a[2], a[4], a[6], a[11], a[12]);
        const Rows v = rows(a[3], "v", t.type, {t.T, t.Hkv, t.d}, t.device);
        void *slots = ptr(a[5], "slot_mapping", at::kLong, {t.T}, t.device);
        const auto cs = dims(tensor(a[7], "k_cache"), "k_cache", 4);
        const int64_t NB = cs[0], bs = cs[2];
        void *kc = ptr(a[7], "k_cache", t.type, {NB, t.Hkv, bs, t.d}, t.device);
        void *vc = ptr(a[8], "v_cache", t.type, {NB, t.Hkv, bs, t.d}, t.device);
        const bool interleaved = bool_arg(a[9]);
        const float mscale = float_arg(a[10]), eps = float_arg(a[13]);
        const int blocks = size_arg(NB, "k_cache"), block_size = size_arg(bs, "k_cache");
        int *status = status_arg(a[14], t.device);
        void *stream = stream_arg(a[15], t.device);
        OtherThreads run;
        c10::cuda::OptionalCUDAGuard guard(c10::Device(c10::kCUDA, (c10::DeviceIndex)t.device));
        return pkv_qk_rope_append(t.q_out.p, t.q_out.stride, t.q.p, t.q.stride, t.k.p, t.k.stride, v.p, v.stride, t.positions,
                                  static_cast<int64_t *>(slots), t.freqs, t.rotary_dim, interleaved, mscale, t.q_weight,
                                  t.k_weight, t.weight_code, eps, t.T_arg, kc, vc, blocks, block_size, t.Hq_arg, t.Hkv_arg,
                                  t.d_arg, t.code, status, stream);
    });
}

// (seq_lens, new_lens, block_tables, free_list, free_count, num_blocks, context_lens, cu_seqlens, slot_mapping,
//  token_pos, free_count_out, dev_status, stream)
PyObject *step_tables(PyObject *, Args a, Py_ssize_t n) {
    return guarded("step_tables", n, 13, [&] {
        const int dev = device_of(tensor(a[0], "seq_lens"), "seq_lens");
        const auto tb = dims(tensor(a[2], "block_tables"), "block_tables", 2);
        const int64_t S = tb[0], MB = tb[1];
        const int64_t capacity = dims(tensor(a[3], "free_list"), "free_list", 1)[0];
        const int64_t T = dims(tensor(a[8], "slot_mapping"), "slot_mapping", 1)[0];
        auto i32 = [&](int i, const char *name, at::IntArrayRef shape) {
            return static_cast<int32_t *>(ptr(a[i], name, at::kInt, shape, dev));
        };
        int32_t *count = i32(4, "free_count", {1});
        int32_t *count_out = a[10] == Py_None ? count : i32(10, "free_count_out", {1});
        int32_t *lens = i32(0, "seq_lens", {S}), *fresh = i32(1, "new_lens", {S}), *tables = i32(2, "block_tables", {S, MB});
        int32_t *list = i32(3, "free_list", {capacity}), *ctx = i32(6, "context_lens", {S}), *cu = i32(7, "cu_seqlens", {S + 1});
        int64_t *slots = static_cast<int64_t *>(ptr(a[8], "slot_mapping", at::kLong, {T}, dev));
        int32_t *pos = i32(9, "token_pos", {T});
        const int seqs = size_arg(S, "block_tables"), max_blocks = size_arg(MB, "block_tables");
        const int room = size_arg(capacity, "free_list"), tokens = size_arg(T, "slot_mapping");
        const int blocks = int_arg(a[5], "num_blocks");
        int *status = status_arg(a[11], dev);
        void *stream = stream_arg(a[12], dev);
        OtherThreads run;
        c10::cuda::OptionalCUDAGuard guard(c10::Device(c10::kCUDA, (c10::DeviceIndex)dev));
        return pkv_step_tables(lens, fresh, seqs, tables, max_blocks, list, room, count, count_out, blocks, 16, ctx, cu, slots,
                               pos, tokens, status, stream);
    });
}

// (block_tables, seq_lens, free_list, free_count, num_blocks, finished, window, num_sinks, workspace, dev_status, stream)
PyObject *release_blocks(PyObject *, Args a, Py_ssize_t n) {
    return guarded("release_blocks", n, 11, [&] {
        const int dev = device_of(tensor(a[0], "block_tables"), "block_tables");
        const auto tb = dims(tensor(a[0], "block_tables"), "block_tables", 2);
        const int64_t S = tb[0], MB = tb[1];
        const int64_t capacity = dims(tensor(a[2], "free_list"), "free_list", 1)[0];
        auto i32 = [&](int i, const char *name, at::IntArrayRef shape) {
            return static_cast<int32_t *>(ptr(a[i], name, at::kInt, shape, dev));
        };
        int32_t *tables = i32(0, "block_tables", {S, MB}), *lens = i32(1, "seq_lens", {S});
        int32_t *list = i32(2, "free_list", {capacity}), *count = i32(3, "free_count", {1});
        int32_t *finished = a[5] == Py_None ? nullptr : i32(5, "finished", {S});
        void *work = nullptr;
        size_t nwork = 0;
        if (a[8] != Py_None) {
            nwork = (size_t)tensor(a[8], "workspace").numel();
            work = ptr(a[8], "workspace", at::kByte, {(int64_t)nwork}, dev);
        }
        const int seqs = size_arg(S, "block_tables"), max_blocks = size_arg(MB, "block_tables");
        const int room = size_arg(capacity, "free_list"), blocks = int_arg(a[4], "num_blocks");
        const int window = int_arg(a[6], "window"), sinks = int_arg(a[7], "num_sinks");
        int *status = status_arg(a[9], dev);
        void *stream = stream_arg(a[10], dev);
        const bool take = a[8] == Py_None;
        OtherThreads run;
        c10::cuda::OptionalCUDAGuard guard(c10::Device(c10::kCUDA, (c10::DeviceIndex)dev));
        // without a workspace of the caller's: memory of the stream that the call runs on
        StreamMemory own;
        if (take && (nwork = pkv_release_workspace_size(seqs)) > 0) work = own.get(nwork, stream);
        return pkv_release_blocks(tables, max_blocks, lens, finished, seqs, window, sinks, list, room, count, blocks, 16, work,
                                  nwork, status, stream);
    });
}

#define PKV_METHOD(f) {#f, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(f)), METH_FASTCALL, nullptr}
PyMethodDef methods[] = {PKV_METHOD(window_decode),  PKV_METHOD(window_prefill), PKV_METHOD(qk_rope),
                         PKV_METHOD(qk_rope_append), PKV_METHOD(step_tables),    PKV_METHOD(release_blocks),
                         {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_torch_calls", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__torch_calls() { return PyModule_Create(&module); }
