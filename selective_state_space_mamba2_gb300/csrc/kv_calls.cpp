// Argument marshalling of the attention-side calls (kv_*) as a CPython module, `_kv_calls`.
//
// A decode step makes these calls between kernels of a few microseconds; checking a dozen tensors
// and filling a ctypes structure takes the interpreter 15 to 35 us a call, several times the
// kernel, and here 4 to 9.  No numeric step runs in this file: it checks shapes, types and strides,
// allocates outputs that the caller did not give, and calls the C ABI of ssd.h.  An argument that
// is refused raises ValueError; a status other than SSD_OK comes back as a Python int, which the
// binding raises as SSDError.
#include <ATen/ATen.h>
#include <ATen/cuda/EmptyTensor.h>
#include <Python.h>
#include <c10/cuda/CUDACachingAllocator.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/autograd/python_variable.h>

#include <climits>
#include <cmath>
#include <stdexcept>
#include <string>

#include "ssd.h"

namespace {

using at::ScalarType;

struct PythonError {};  // an exception is set already

// An owned reference.
struct Held {
    PyObject *o = nullptr;
    Held() = default;
    Held(const Held &) = delete;
    Held &operator=(const Held &) = delete;
    ~Held() { Py_XDECREF(o); }
};

[[noreturn]] void refuse(const std::string &what) { throw std::invalid_argument(what); }

const char *type_name(ScalarType t) {
    return t == at::kInt ? "int32" : t == at::kFloat ? "float32" : t == at::kBFloat16 ? "bfloat16" : c10::toString(t);
}

std::string shape_text(at::IntArrayRef s) {
    std::string o = "[";
    for (size_t i = 0; i < s.size(); ++i) o += (i ? ", " : "") + std::to_string(s[i]);
    return o + "]";
}

// The device of a call is that of its first tensor; every other one has to be there too.
thread_local int call_device = -1;

void on_call_device(int index, const char *name) {
    if (call_device < 0) call_device = index;
    if (index != call_device)
        refuse(std::string(name) + " is on cuda:" + std::to_string(index) + ", other arguments are on cuda:" +
               std::to_string(call_device));
}

const at::Tensor &tensor(PyObject *o, const char *name) {
    if (!THPVariable_Check(o)) refuse(std::string(name) + (o == Py_None ? " is required" : " must be a CUDA tensor"));
    const at::Tensor &t = THPVariable_Unpack(o);
    if (!t.is_cuda()) refuse(std::string(name) + " must be a CUDA tensor");
    on_call_device(t.get_device(), name);
    return t;
}

int64_t integer(PyObject *o) {
    const long long v = PyLong_AsLongLong(o);
    if (v == -1 && PyErr_Occurred()) throw PythonError{};
    return v;
}

int32_t int32(PyObject *o, const char *name) {
    const int64_t v = integer(o);
    if (v < INT_MIN || v > INT_MAX) refuse(std::string(name) + " must fit 32 bits");
    return (int32_t)v;
}

int32_t size32(int64_t v, const char *name) {
    if (v > INT_MAX) refuse(std::string(name) + " must fit 32 bits");
    return (int32_t)v;
}

float real(PyObject *o) {
    const double v = PyFloat_AsDouble(o);
    if (v == -1.0 && PyErr_Occurred()) throw PythonError{};
    return (float)v;
}

bool truth(PyObject *o) {
    const int v = PyObject_IsTrue(o);
    if (v < 0) throw PythonError{};
    return v == 1;
}

int32_t dtype_code(const at::Tensor &t, const char *name) {
    const ScalarType s = t.scalar_type();
    if (s == at::kBFloat16) return SSD_BF16;
    if (s == at::kFloat) return SSD_F32;
    refuse(std::string(name) + " must be bfloat16 or float32, got " + type_name(s));
}

// Pointer of a dense device tensor of that shape and type.
void *dense(PyObject *o, const char *name, at::IntArrayRef shape, ScalarType type) {
    const at::Tensor &t = tensor(o, name);
    if (t.scalar_type() != type || t.sizes() != shape)
        refuse(std::string(name) + " must be " + type_name(type) + " of shape " + shape_text(shape));
    if (!t.is_contiguous()) refuse(std::string(name) + " must be contiguous");
    return t.data_ptr();
}

const int32_t *ints(PyObject *o, const char *name, int64_t n) {
    const int64_t shape[1] = {n};
    return static_cast<const int32_t *>(dense(o, name, shape, at::kInt));
}

// Dense int32 [rows, cols] (cols: whatever it has).
const int32_t *table(PyObject *o, const char *name, int64_t rows, int64_t &cols) {
    const at::Tensor &t = tensor(o, name);
    if (t.dim() != 2 || t.size(0) != rows || t.scalar_type() != at::kInt)
        refuse(std::string(name) + " must be int32 [" + std::to_string(rows) + ", columns]");
    if (!t.is_contiguous()) refuse(std::string(name) + " must be contiguous");
    cols = t.size(1);
    return static_cast<const int32_t *>(t.data_ptr());
}

struct Rows {
    void *p;
    int64_t stride;  // elements from token to token
};

// [T, heads, D] whose tokens are dense rows.
Rows rows(PyObject *o, const char *name, int64_t T, int64_t H, int64_t D, ScalarType type) {
    const at::Tensor &t = tensor(o, name);
    const int64_t shape[3] = {T, H, D};
    if (t.scalar_type() != type || t.sizes() != at::IntArrayRef(shape))
        refuse(std::string(name) + " must be " + type_name(type) + " of shape " + shape_text(shape));
    if (T > 0 && ((t.stride(2) != 1 && D > 1) || (t.stride(1) != D && H > 1)))
        refuse("the rows of " + std::string(name) + " must be dense");
    return {t.data_ptr(), T > 1 ? t.stride(0) : H * D};
}

struct Pages {
    void *k, *v;
    int32_t blocks, block_size;
    int64_t stride;
};

// k_cache and v_cache: [num_blocks, block_size, H, D], blocks dense, the same block stride.
Pages pages(PyObject *ko, PyObject *vo, int64_t H, int64_t D, ScalarType type) {
    const at::Tensor &k = tensor(ko, "k_cache"), &v = tensor(vo, "v_cache");
    if (k.dim() != 4 || k.scalar_type() != type || v.scalar_type() != type || k.sizes() != v.sizes() || k.size(2) != H ||
        k.size(3) != D)
        refuse(std::string("k_cache and v_cache must be ") + type_name(type) + " [num_blocks, block_size, " +
               std::to_string(H) + ", " + std::to_string(D) + "]");
    const int64_t nb = k.size(0), bs = k.size(1);
    for (const at::Tensor *t : {&k, &v})
        if ((t->stride(3) != 1 && D > 1) || (t->stride(2) != D && H > 1) || (t->stride(1) != H * D && bs > 1))
            refuse("the blocks of k_cache and v_cache must be dense");
    if (nb > 1 && k.stride(0) != v.stride(0)) refuse("k_cache and v_cache must have the same block stride");
    return {k.data_ptr(), v.data_ptr(), size32(nb, "num_blocks"), size32(bs, "block_size"),
            nb > 1 ? k.stride(0) : bs * H * D};
}

// The kernels or 32 bits into it.
uint32_t *error_word(PyObject *o) {
    if (o == Py_None) return nullptr;
    const at::Tensor &t = tensor(o, "err_word");
    if ((t.scalar_type() != at::kInt && t.scalar_type() != at::kUInt32) || t.numel() < 1)
        refuse("err_word must be int32 of one element");
    return static_cast<uint32_t *>(t.data_ptr());
}

// The caller's stream (a torch stream or its pointer as a number), or the current one of the device.
ssd_stream_t stream_of(PyObject *o, const at::Tensor &like) {
    if (o == Py_None)
        return reinterpret_cast<ssd_stream_t>(c10::cuda::getCurrentCUDAStream(like.get_device()).stream());
    if (PyObject_HasAttrString(o, "device_index")) {
        PyObject *index = PyObject_GetAttrString(o, "device_index");
        const long i = index ? PyLong_AsLong(index) : -1;
        Py_XDECREF(index);
        if (PyErr_Occurred()) throw PythonError{};
        on_call_device((int)i, "stream");
    }
    PyObject *p = PyObject_HasAttrString(o, "cuda_stream") ? PyObject_GetAttrString(o, "cuda_stream") : PyNumber_Index(o);
    if (!p) throw PythonError{};
    const unsigned long long v = PyLong_AsUnsignedLongLong(p);
    Py_DECREF(p);
    if (PyErr_Occurred()) throw PythonError{};
    return reinterpret_cast<ssd_stream_t>(v);
}

// Memory of the call's stream, on which it is written: memory of the current one, where that is another, could still have
// work of that stream to come, of whoever had it before.  What the current stream may do with it later is waited
// for before it is handed out again.
at::Tensor empty(at::IntArrayRef shape, ScalarType type, const at::Tensor &like, ssd_stream_t s) {
    const auto dev = like.get_device();
    const c10::cuda::CUDAStream now = c10::cuda::getCurrentCUDAStream(dev);
    if (reinterpret_cast<cudaStream_t>(s) == now.stream())
        return at::detail::empty_cuda(shape, type, like.device(), std::nullopt);
    const c10::cuda::CUDAStreamGuard guard(c10::cuda::getStreamFromExternal(reinterpret_cast<cudaStream_t>(s), dev));
    at::Tensor t = at::detail::empty_cuda(shape, type, like.device(), std::nullopt);
    c10::cuda::CUDACachingAllocator::recordStream(t.storage().data_ptr(), now);
    return t;
}

// A dense int32 tensor of n entries in `room`'s memory, from entry `at` on.
at::Tensor piece_of(const at::Tensor &room, int64_t n, int64_t at) {
    at::Tensor t = at::detail::make_tensor<c10::TensorImpl>(c10::Storage(room.storage()), room.key_set(), room.dtype());
    t.unsafeGetTensorImpl()->set_storage_offset(at);
    t.unsafeGetTensorImpl()->set_sizes_contiguous({n});
    return t;
}

PyObject *status(ssd_status_t s) { return PyLong_FromLong((long)s); }

PyObject *block_tables(PyObject *const *a, PyObject *) {
    const at::Tensor &ctx = tensor(a[0], "context_lens");
    const c10::cuda::CUDAGuard guard(ctx.device());
    const int64_t S = ctx.numel();
    kv_tables_args p = {};
    p.num_reqs = size32(S, "requests");
    p.context_lens = ints(a[0], "context_lens", S);
    p.new_lens = ints(a[1], "new_lens", S);
    p.reserved_lens = ints(a[2], "reserved_lens", S);
    int64_t cols = 0;
    p.block_table = const_cast<int32_t *>(table(a[3], "block_table", S, cols));
    p.table_cols = size32(cols, "block_table columns");
    const int64_t ring = tensor(a[4], "free_ring").numel();
    p.free_ring = ints(a[4], "free_ring", ring);
    p.free_capacity = size32(ring, "free_ring");
    p.ring_in = ints(a[5], "ring_state", 2);
    p.block_size = int32(a[6], "block_size");
    p.num_blocks = int32(a[7], "num_blocks");
    p.max_tokens = int32(a[8], "max_tokens");
    p.null_block_id = int32(a[9], "null_block_id");
    if (p.max_tokens < 0) refuse("max_tokens must not be negative");
    static const char *const keys[7] = {"cu_seqlens", "seq_lens", "reserved_lens", "ring_state", "slots", "positions",
                                        "token_req"};
    static PyObject *names[7] = {};  // made once, as attribute names are (under the interpreter's lock)
    for (int i = 0; i < 7 && !names[i]; ++i)
        if (!(names[i] = PyUnicode_InternFromString(keys[i]))) throw PythonError{};
    const int64_t sizes[7] = {S + 1, S, S, 2, p.max_tokens, p.max_tokens, p.max_tokens};
    int32_t *ptr[7] = {};
    p.err_word = error_word(a[11]);
    const ssd_stream_t stream = stream_of(a[12], ctx);
    PyObject *out = a[10];
    Held given[7];  // a mapping may make its values on access: they live until the call is queued
    at::Tensor room;
    if (out == Py_None) {
        // one allocation, each output at a 64-byte boundary of it
        int64_t at[7], all = 0;
        for (int i = 0; i < 7; ++i) at[i] = all, all += (sizes[i] + 15) / 16 * 16;
        room = empty(all, at::kInt, ctx, stream);
        out = PyDict_New();
        if (!out) throw PythonError{};
        for (int i = 0; i < 7; ++i) {
            ptr[i] = static_cast<int32_t *>(room.data_ptr()) + at[i];
            PyObject *w = THPVariable_Wrap(piece_of(room, sizes[i], at[i]));
            const int bad = w ? PyDict_SetItem(out, names[i], w) : -1;
            Py_XDECREF(w);
            if (bad) {
                Py_DECREF(out);
                throw PythonError{};
            }
        }
    } else {
        for (int i = 0; i < 7; ++i) {
            PyObject *t = given[i].o = PyObject_GetItem(out, names[i]);
            if (!t) {
                if (i < 6 || !PyErr_ExceptionMatches(PyExc_KeyError)) throw PythonError{};
                PyErr_Clear();  // token_req may be left out
                continue;
            }
            if (i < 6 || t != Py_None) ptr[i] = const_cast<int32_t *>(ints(t, keys[i], sizes[i]));
        }
        Py_INCREF(out);
    }
    p.cu_seqlens = ptr[0], p.seq_lens = ptr[1], p.reserved_out = ptr[2], p.ring_out = ptr[3];
    p.slots = ptr[4], p.positions = ptr[5], p.token_req = ptr[6];
    const ssd_status_t s = kv_block_tables(&p, stream);
    if (s == SSD_OK) return out;
    Py_DECREF(out);
    return status(s);
}

PyObject *norm_rope(PyObject *const *a, PyObject *) {
    const at::Tensor &q = tensor(a[0], "q"), &k = tensor(a[1], "k");
    const c10::cuda::CUDAGuard guard(q.device());
    if (q.dim() != 3 || k.dim() != 3) refuse("q and k must be [T, heads, D]");
    const int64_t T = q.size(0), H = q.size(1), D = q.size(2), G = k.size(1);
    const ScalarType type = q.scalar_type();
    kv_qk_args p = {};
    p.dtype = dtype_code(q, "q");
    p.total_tokens = size32(T, "tokens"), p.nheads = size32(H, "heads"), p.kv_heads = size32(G, "heads");
    p.headdim = size32(D, "headdim");
    const Rows rq = rows(a[0], "q", T, H, D, type), rk = rows(a[1], "k", T, G, D, type);
    p.q = rq.p, p.q_stride = rq.stride, p.k = rk.p, p.k_stride = rk.stride;
    if (a[3] != Py_None) {
        const at::Tensor &cs = tensor(a[3], "cos_sin");
        if (cs.dim() != 2) refuse("cos_sin must be float32 [max_position, rotary_dim]");
        p.max_position = size32(cs.size(0), "positions"), p.rotary_dim = size32(cs.size(1), "rotary_dim");
        p.cos_sin = static_cast<const float *>(dense(a[3], "cos_sin", cs.sizes(), at::kFloat));
        p.positions = ints(a[2], "positions", T);
    }
    const int64_t wide[1] = {D};
    if (a[4] != Py_None) p.q_weight = static_cast<const float *>(dense(a[4], "q_weight", wide, at::kFloat));
    if (a[5] != Py_None) p.k_weight = static_cast<const float *>(dense(a[5], "k_weight", wide, at::kFloat));
    p.eps = real(a[6]);
    p.interleaved = truth(a[7]);
    if (a[9] != Py_None || a[10] != Py_None || a[11] != Py_None) {
        const Pages c = pages(a[9], a[10], G, D, type);
        p.k_cache = c.k, p.v_cache = c.v, p.num_blocks = c.blocks, p.block_size = c.block_size;
        p.cache_block_stride = c.stride;
        const Rows rv = rows(a[8], "v", T, G, D, type);
        p.v = rv.p, p.v_stride = rv.stride;
        p.slots = ints(a[11], "slots", T);
    }
    p.err_word = error_word(a[14]);
    const ssd_stream_t stream = stream_of(a[15], q);
    const int64_t qs[3] = {T, H, D}, ks[3] = {T, G, D};
    at::Tensor q_new, k_new;
    if (a[12] == Py_None) {
        q_new = empty(qs, type, q, stream);
        p.q_out = q_new.data_ptr();
    } else {
        p.q_out = dense(a[12], "q_out", qs, type);
    }
    if (a[13] == Py_None) {
        k_new = empty(ks, type, q, stream);
        p.k_out = k_new.data_ptr();
    } else {
        p.k_out = dense(a[13], "k_out", ks, type);
    }
    const ssd_status_t s = kv_qk_norm_rope(&p, stream);
    if (s != SSD_OK) return status(s);
    PyObject *qo = a[12] == Py_None ? THPVariable_Wrap(std::move(q_new)) : Py_NewRef(a[12]);
    PyObject *ko = a[13] == Py_None ? THPVariable_Wrap(std::move(k_new)) : Py_NewRef(a[13]);
    PyObject *r = qo && ko ? PyTuple_Pack(2, qo, ko) : nullptr;
    Py_XDECREF(qo);
    Py_XDECREF(ko);
    return r;
}

PyObject *tree_attention(PyObject *const *a, PyObject *) {
    const at::Tensor &q = tensor(a[0], "q"), &k = tensor(a[1], "k_new");
    const c10::cuda::CUDAGuard guard(q.device());
    if (q.dim() != 3 || k.dim() != 3) refuse("q and k_new must be [T, heads, D]");
    const int64_t T = q.size(0), H = q.size(1), D = q.size(2), G = k.size(1);
    const ScalarType type = q.scalar_type();
    kv_attention_args p = {};
    p.dtype = dtype_code(q, "q");
    p.total_tokens = size32(T, "tokens"), p.nheads = size32(H, "heads"), p.kv_heads = size32(G, "heads");
    p.headdim = size32(D, "headdim");
    const Rows rq = rows(a[0], "q", T, H, D, type), rk = rows(a[1], "k_new", T, G, D, type),
               rv = rows(a[2], "v_new", T, G, D, type);
    p.q = rq.p, p.q_stride = rq.stride, p.k_new = rk.p, p.k_stride = rk.stride, p.v_new = rv.p, p.v_stride = rv.stride;
    const Pages c = pages(a[3], a[4], G, D, type);
    p.k_cache = c.k, p.v_cache = c.v, p.num_blocks = c.blocks, p.block_size = c.block_size;
    p.cache_block_stride = c.stride;
    const int64_t S = tensor(a[5], "cu_seqlens").numel() - 1;
    if (S < 0) refuse("cu_seqlens must have an entry more than there are requests");
    p.num_seqs = size32(S, "requests");
    p.cu_seqlens = ints(a[5], "cu_seqlens", S + 1);
    p.context_lens = ints(a[6], "context_lens", S);
    int64_t cols = 0;
    p.block_table = table(a[7], "block_table", S, cols);
    p.table_cols = size32(cols, "block_table columns");
    p.max_new_tokens = int32(a[8], "max_new_tokens");
    if (a[9] != Py_None) {
        int64_t words = 0;
        p.tree_mask = reinterpret_cast<const uint32_t *>(table(a[9], "tree_mask", T, words));
        if (T > 0 && words == 0) refuse("tree_mask must have a word at least");  // it has no pointer: a chain
        p.mask_words = size32(words, "tree_mask words");
    }
    p.scale = a[10] == Py_None ? (float)(1.0 / std::sqrt((double)D)) : real(a[10]);
    p.err_word = error_word(a[15]);
    const ssd_stream_t stream = stream_of(a[16], q);
    const int64_t shape[3] = {T, H, D}, lse_shape[2] = {T, H};
    at::Tensor out, lse, room;
    if (a[11] == Py_None) {
        out = empty(shape, type, q, stream);
        p.out = out.data_ptr();
    } else {
        p.out = dense(a[11], "out", shape, type);
    }
    const bool with_lse = a[12] != Py_None || truth(a[13]);
    if (a[12] != Py_None) {
        p.lse = static_cast<float *>(dense(a[12], "lse", lse_shape, at::kFloat));
    } else if (with_lse) {
        lse = empty(lse_shape, at::kFloat, q, stream);
        p.lse = static_cast<float *>(lse.data_ptr());
    }
    p.wait_limit_cycles = integer(a[17]);
    if (a[14] == Py_None) {
        room = empty((int64_t)kv_tree_attention_workspace_size(&p), at::kByte, q, stream);
    } else {
        room = tensor(a[14], "workspace");
        if (!room.is_contiguous()) refuse("workspace must be contiguous");
    }
    const ssd_status_t s = kv_tree_attention(&p, room.data_ptr(), (size_t)room.nbytes(), stream);
    if (s != SSD_OK) return status(s);
    PyObject *oo = a[11] == Py_None ? THPVariable_Wrap(std::move(out)) : Py_NewRef(a[11]);
    if (!with_lse || !oo) return oo;
    PyObject *lo = a[12] == Py_None ? THPVariable_Wrap(std::move(lse)) : Py_NewRef(a[12]);
    PyObject *r = lo ? PyTuple_Pack(2, oo, lo) : nullptr;
    Py_DECREF(oo);
    Py_XDECREF(lo);
    return r;
}

PyObject *commit_tokens(PyObject *const *a, PyObject *) {
    const at::Tensor &k = tensor(a[0], "k_new");
    const c10::cuda::CUDAGuard guard(k.device());
    if (k.dim() != 3) refuse("k_new must be [T, heads, D]");
    const int64_t T = k.size(0), H = k.size(1), D = k.size(2);
    const ScalarType type = k.scalar_type();
    kv_commit_args p = {};
    p.dtype = dtype_code(k, "k_new");
    p.total_tokens = size32(T, "tokens"), p.kv_heads = size32(H, "heads"), p.headdim = size32(D, "headdim");
    const Rows rk = rows(a[0], "k_new", T, H, D, type), rv = rows(a[1], "v_new", T, H, D, type);
    p.k_new = rk.p, p.k_stride = rk.stride, p.v_new = rv.p, p.v_stride = rv.stride;
    const Pages c = pages(a[2], a[3], H, D, type);
    p.k_cache = c.k, p.v_cache = c.v, p.num_blocks = c.blocks, p.block_size = c.block_size;
    p.cache_block_stride = c.stride;
    const int64_t slots = tensor(a[4], "slots").numel();
    p.slots = ints(a[4], "slots", slots);
    if (slots < T) refuse("slots must have an entry for each of the " + std::to_string(T) + " tokens");
    int64_t S = 0;
    if (a[5] != Py_None) {
        S = tensor(a[5], "cu_seqlens").numel() - 1;
        if (S < 0) refuse("cu_seqlens must have an entry more than there are requests");
        p.cu_seqlens = ints(a[5], "cu_seqlens", S + 1);
    } else if (a[6] != Py_None || a[7] != Py_None) {
        refuse("cu_seqlens is required");
    }
    p.num_seqs = size32(S, "requests");
    if (a[7] != Py_None) {
        int64_t width = 0;
        p.path = table(a[7], "path", S, width);
        if (width == 0) refuse("path must have a column at least");
        p.max_path = size32(width, "path columns");
        p.path_lens = ints(a[8], "path_lens", S);
    }
    p.err_word = error_word(a[10]);
    const ssd_stream_t stream = stream_of(a[11], k);
    at::Tensor made;
    PyObject *out = a[9];
    if (a[6] != Py_None) {
        p.context_lens = ints(a[6], "context_lens", S);
        if (out == Py_None) {
            made = empty(S, at::kInt, k, stream);
            p.context_out = static_cast<int32_t *>(made.data_ptr());
        } else {
            p.context_out = const_cast<int32_t *>(ints(out, "context_out", S));
        }
    }
    const ssd_status_t s = kv_commit_tokens(&p, stream);
    if (s != SSD_OK) return status(s);
    if (made.defined()) return THPVariable_Wrap(std::move(made));
    return Py_NewRef(out);
}

// The device that a call with tensors on the devices of these two indices runs on (the check that tensor() makes, for
// machines without a second one).
PyObject *device_of_call(PyObject *const *a, PyObject *) {
    on_call_device(int32(a[0], "index"), "first");
    on_call_device(int32(a[1], "index"), "second");
    return PyLong_FromLong(call_device);
}

template <PyObject *(*Fn)(PyObject *const *, PyObject *), Py_ssize_t kArgs>
PyObject *guarded(PyObject *self, PyObject *const *args, Py_ssize_t n) {
    if (n != kArgs) {
        PyErr_Format(PyExc_TypeError, "%zd arguments expected, got %zd", kArgs, n);
        return nullptr;
    }
    call_device = -1;
    try {
        return Fn(args, self);
    } catch (const PythonError &) {
    } catch (const std::invalid_argument &e) {
        PyErr_SetString(PyExc_ValueError, e.what());
    } catch (const std::exception &e) {
        PyErr_SetString(PyExc_RuntimeError, e.what());
    }
    return nullptr;
}

#define KV_METHOD(name, fn, n) \
    {name, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(guarded<fn, n>)), METH_FASTCALL, nullptr}
PyMethodDef methods[] = {KV_METHOD("block_tables", block_tables, 13), KV_METHOD("norm_rope", norm_rope, 16),
                         KV_METHOD("tree_attention", tree_attention, 18), KV_METHOD("commit_tokens", commit_tokens, 12),
                         KV_METHOD("device_of_call", device_of_call, 2),
                         {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_kv_calls", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__kv_calls() { return PyModule_Create(&module); }
