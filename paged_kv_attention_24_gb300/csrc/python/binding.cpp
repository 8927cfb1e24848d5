// Native argument marshalling for the calls of a step whose kernels are short: a
// decode step runs them once per forward, and checking a dozen tensors and
// filling ctypes arguments from Python took two to four times as long as the
// launches themselves (tables 10.9, groups 16, shared decode 22 us a call).
// It does what the ctypes binding does for the other calls (contiguous tensors
// of the right type on one device, raw pointers, the current stream) and nothing
// else; the calls go through the same C ABI.  Every function returns None or the
// call's non-zero status, which the Python side turns into MsglError.
#include <Python.h>

#include <ATen/cuda/EmptyTensor.h>
#include <c10/cuda/CUDACachingAllocator.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/autograd/python_variable.h>

#include <initializer_list>
#include <stdexcept>
#include <vector>

#include "../../../include/msgl_attn.h"

namespace {

struct Refused {};   // a Python error is set

[[noreturn]] void refuse(const char *fmt, const char *name, const char *more = "") {
    PyErr_Format(PyExc_ValueError, fmt, name, more);
    throw Refused{};
}

const at::Tensor &tensor(PyObject *o, const char *name) {
    if (!THPVariable_Check(o)) refuse("%s must be a CUDA tensor", name);
    return THPVariable_Unpack(o);
}

// A contiguous tensor of the type on cuda:dev (dev = -1: on any, which it then sets).
const at::Tensor &checked(PyObject *o, const char *name, at::ScalarType type, int &dev) {
    const at::Tensor &t = tensor(o, name);
    if (!t.is_cuda()) refuse("%s must be a CUDA tensor", name);
    if (t.scalar_type() != type)
        refuse("%s must be torch.%s", name, type == at::kInt ? "int32" : type == at::kLong ? "int64" : type == at::kFloat ? "float32" : "bfloat16");
    if (dev < 0) dev = t.get_device();
    if (t.get_device() != dev) refuse("%s must be on the same CUDA device as the other tensors", name);
    if (!t.is_contiguous()) refuse("%s must be contiguous", name);
    return t;
}

int32_t *i32(const at::Tensor &t) { return static_cast<int32_t *>(t.data_ptr()); }

long long integer(PyObject *o) {
    const long long v = PyLong_AsLongLong(o);   // takes whatever has __index__
    if (v == -1 && PyErr_Occurred()) throw Refused{};
    return v;
}

int32_t integer32(PyObject *o, const char *name) {
    const long long v = integer(o);
    if (v < INT32_MIN || v > INT32_MAX) refuse("%s does not fit 32 bits", name);
    return (int32_t)v;
}

int32_t size32(int64_t v, const char *name) {
    if (v > INT32_MAX) refuse("%s has a size that does not fit 32 bits", name);
    return (int32_t)v;
}

uint32_t *status_ptr(PyObject *o, int dev) {
    if (o == Py_None) return nullptr;
    const at::Tensor &t = checked(o, "status", at::kInt, dev);
    if (t.numel() < 1) refuse("%s must have an entry", "status");
    return static_cast<uint32_t *>(t.data_ptr());
}

// The device's current stream, or the one given (as the integer of its handle).
c10::cuda::CUDAStream stream_of(PyObject *o, int dev) {
    if (o == Py_None) return c10::cuda::getCurrentCUDAStream(dev);
    void *p = PyLong_AsVoidPtr(o);
    if (!p && PyErr_Occurred()) throw Refused{};
    return c10::cuda::getStreamFromExternal(static_cast<cudaStream_t>(p), dev);
}

// A new tensor in `stream`'s order.  When the caller named a stream other than the current one, the
// tensor's memory also waits for the current one before it is used again.
at::Tensor fresh(at::IntArrayRef sizes, at::ScalarType type, int dev, const c10::cuda::CUDAStream &stream) {
    const c10::cuda::CUDAStream current = c10::cuda::getCurrentCUDAStream((c10::DeviceIndex)dev);
    const c10::Device device(c10::kCUDA, (c10::DeviceIndex)dev);
    if (current == stream) return at::detail::empty_cuda(sizes, type, device, c10::nullopt);
    c10::cuda::setCurrentCUDAStream(stream);
    struct Back {
        c10::cuda::CUDAStream s;
        ~Back() { c10::cuda::setCurrentCUDAStream(s); }
    } back{current};
    at::Tensor t = at::detail::empty_cuda(sizes, type, device, c10::nullopt);
    c10::cuda::CUDACachingAllocator::recordStream(t.storage().data_ptr(), current);
    return t;
}

// Row i of a contiguous [rows, n] tensor as a tensor of its own over the same memory (an allocation
// costs about 0.9 us, this 0.2).
at::Tensor row_of(const at::Tensor &t, int64_t i) {
    auto impl = c10::make_intrusive<at::TensorImpl>(c10::Storage(t.storage()), t.key_set(), t.dtype());
    impl->set_sizes_contiguous({t.size(1)});
    impl->set_storage_offset(i * t.size(1));
    return at::Tensor(std::move(impl));
}

msgl_stream_t raw(const c10::cuda::CUDAStream &s) { return reinterpret_cast<msgl_stream_t>(s.stream()); }

PyObject *done(msgl_status rc) {
    if (rc == MSGL_OK) Py_RETURN_NONE;
    return PyLong_FromLong(rc);
}

bool arity(Py_ssize_t n, Py_ssize_t want) {
    if (n == want) return true;
    PyErr_Format(PyExc_TypeError, "expected %zd arguments, got %zd", want, n);
    return false;
}

// Other Python threads run while the allocator and the launches may block (a full launch queue).
struct NoGil {
    PyThreadState *state = PyEval_SaveThread();
    ~NoGil() { PyEval_RestoreThread(state); }
};

// Runs f; C++ exceptions (an allocation that fails) become Python ones.
template <class F>
PyObject *guarded(F f) {
    try {
        return f();
    } catch (const Refused &) {
    } catch (const c10::OutOfMemoryError &e) {
        PyObject *torch = PyImport_ImportModule("torch");
        PyObject *type = torch ? PyObject_GetAttrString(torch, "OutOfMemoryError") : nullptr;
        PyErr_Clear();
        PyErr_SetString(type ? type : PyExc_MemoryError, e.what_without_backtrace());
        Py_XDECREF(type);
        Py_XDECREF(torch);
    } catch (const std::exception &e) {
        PyErr_SetString(PyExc_RuntimeError, e.what());
    }
    return nullptr;
}

// (req_table, cached_lens, new_lens | None, free_pages, num_slots, page_size, req_rows | None, page_table,
//  seq_lens, cu_ext, positions, out_loc, pages_taken, status | None, stream | None)
PyObject *step_tables(PyObject *, PyObject *const *a, Py_ssize_t n) {
    if (!arity(n, 15)) return nullptr;
    return guarded([&]() -> PyObject * {
        int dev = -1;
        const at::Tensor &cached = checked(a[1], "cached_lens", at::kInt, dev);
        const at::Tensor &table = checked(a[0], "req_table", at::kInt, dev);
        const at::Tensor &free_pages = checked(a[3], "free_pages", at::kInt, dev);
        const at::Tensor &pages = checked(a[7], "page_table", at::kInt, dev);
        const at::Tensor &seq = checked(a[8], "seq_lens", at::kInt, dev);
        const at::Tensor &cu = checked(a[9], "cu_ext", at::kInt, dev);
        const at::Tensor &pos = checked(a[10], "positions", at::kInt, dev);
        const at::Tensor &loc = checked(a[11], "out_loc", at::kInt, dev);
        const at::Tensor &taken = checked(a[12], "pages_taken", at::kInt, dev);
        const int32_t B = size32(cached.numel(), "cached_lens");
        const int32_t *added = nullptr, *rows = nullptr;
        if (a[2] != Py_None) {
            const at::Tensor &t = checked(a[2], "new_lens", at::kInt, dev);
            if (t.numel() != B) refuse("%s must have one entry per request", "new_lens");
            added = i32(t);
        }
        if (a[6] != Py_None) {
            const at::Tensor &t = checked(a[6], "req_rows", at::kInt, dev);
            if (t.numel() != B) refuse("%s must have one entry per request", "req_rows");
            rows = i32(t);
        }
        if (table.dim() != 2) refuse("%s must be [rows, width]", "req_table");
        if (pages.dim() != 2 || pages.size(0) != B || seq.numel() != B || cu.numel() != (int64_t)B + 1 ||
            loc.numel() != pos.numel() || taken.numel() != 1)
            refuse("%s must hold [B, width], [B], [B + 1], [T], [T] and [1] entries", "out");
        const int32_t W = size32(table.size(1), "req_table"), w = size32(pages.size(1), "page_table");
        msgl_step_out out;
        out.page_ids = i32(pages);
        out.stride = out.width = w;
        out.seq_lens = i32(seq);
        out.cu_ext = i32(cu);
        out.positions = i32(pos);
        out.out_loc = i32(loc);
        out.pages_taken = i32(taken);
        out.total_tokens = size32(pos.numel(), "positions");
        const int64_t slots = integer(a[4]);
        const int32_t ps = integer32(a[5], "page_size");
        uint32_t *status = status_ptr(a[13], dev);
        c10::cuda::CUDAGuard guard((c10::DeviceIndex)dev);
        const c10::cuda::CUDAStream stream = stream_of(a[14], dev);
        const int32_t num_rows = size32(table.size(0), "req_table"), num_free = size32(free_pages.numel(), "free_pages");
        msgl_status rc;
        {
            NoGil no_gil;
            rc = msgl_step_tables(slots, ps, i32(table), num_rows, W, W, rows, i32(cached), added, B, i32(free_pages),
                                  num_free, &out, status, raw(stream));
        }
        return done(rc);
    });
}

// (page_table, seq_lens, page_size, max_seq_len, min_shared, group_start | None, shared_lens | None,
//  status | None, stream | None) -> (group_start, shared_lens) or the status
PyObject *shared_prefixes(PyObject *, PyObject *const *a, Py_ssize_t n) {
    if (!arity(n, 9)) return nullptr;
    return guarded([&]() -> PyObject * {
        int dev = -1;
        const at::Tensor &seq = checked(a[1], "seq_lens", at::kInt, dev);
        const at::Tensor &pages = checked(a[0], "page_table", at::kInt, dev);
        const int32_t B = size32(seq.numel(), "seq_lens");
        const int32_t ps = integer32(a[2], "page_size"), max_seq = integer32(a[3], "max_seq_len"),
                      min_shared = integer32(a[4], "min_shared");
        c10::cuda::CUDAGuard guard((c10::DeviceIndex)dev);
        const c10::cuda::CUDAStream stream = stream_of(a[8], dev);
        at::Tensor first, shared;
        if (a[5] != Py_None) first = checked(a[5], "group_start", at::kInt, dev);
        if (a[6] != Py_None) shared = checked(a[6], "shared_lens", at::kInt, dev);
        if (pages.dim() != 2 || pages.size(0) != B || (first.defined() && first.numel() != B) ||
            (shared.defined() && shared.numel() != B))
            refuse("%s must be [B, width]; seq_lens, group_start and shared_lens [B]", "page_table");
        uint32_t *status = status_ptr(a[7], dev);
        msgl_page_table pt;
        pt.page_ids = i32(pages);
        pt.stride = pt.width = size32(pages.size(1), "page_table");
        msgl_status rc;
        {
            NoGil no_gil;
            if (!first.defined() && !shared.defined()) {
                const at::Tensor both = fresh({2, B}, at::kInt, dev, stream);
                first = row_of(both, 0);
                shared = row_of(both, 1);
            }
            if (!first.defined()) first = fresh({B}, at::kInt, dev, stream);
            if (!shared.defined()) shared = fresh({B}, at::kInt, dev, stream);
            rc = msgl_shared_prefixes(&pt, i32(seq), B, ps, max_seq, min_shared, i32(first), i32(shared), status,
                                      raw(stream));
        }
        if (rc != MSGL_OK) return done(rc);
        PyObject *x = THPVariable_Wrap(first), *y = THPVariable_Wrap(shared);
        PyObject *r = x && y ? PyTuple_Pack(2, x, y) : nullptr;
        Py_XDECREF(x);
        Py_XDECREF(y);
        return r;
    });
}

// (k_pool, v_pool, page_size, q, page_table, seq_lens, group_start, shared_lens, max_seq_len, scale, out | None,
//  lse | None, workspace | None, status | None, stream | None, sharing) -> (out, lse) or the status
PyObject *attn_decode_shared(PyObject *, PyObject *const *a, Py_ssize_t n) {
    if (!arity(n, 16)) return nullptr;
    return guarded([&]() -> PyObject * {
        int dev = -1;
        const at::Tensor &q = checked(a[3], "q", at::kBFloat16, dev);
        const at::Tensor &k = checked(a[0], "k_pool", at::kBFloat16, dev);
        const at::Tensor &v = checked(a[1], "v_pool", at::kBFloat16, dev);
        const at::Tensor &pages = checked(a[4], "page_table", at::kInt, dev);
        const at::Tensor &seq = checked(a[5], "seq_lens", at::kInt, dev);
        const at::Tensor &first = checked(a[6], "group_start", at::kInt, dev);
        const at::Tensor &shared = checked(a[7], "shared_lens", at::kInt, dev);
        if (q.dim() != 3) refuse("%s must be [B, Hq, D]", "q");
        if (k.dim() != 3 || v.sizes() != k.sizes()) refuse("%s and v_pool must both be [num_slots, Hkv, D]", "k_pool");
        const int32_t B = size32(q.size(0), "q"), hq = size32(q.size(1), "q");
        if (q.size(2) != k.size(2)) refuse("%s and the pool must have the same head_dim", "q");
        if (pages.dim() != 2 || pages.size(0) != B || seq.numel() != B || first.numel() != B || shared.numel() != B)
            refuse("%s must be [B, width]; seq_lens, group_start and shared_lens [B]", "page_table");
        const int32_t ps = integer32(a[2], "page_size"), max_seq = integer32(a[8], "max_seq_len"),
                      sharing = integer32(a[15], "sharing");
        const double scale = PyFloat_AsDouble(a[9]);
        if (scale == -1.0 && PyErr_Occurred()) throw Refused{};
        uint32_t *status = status_ptr(a[13], dev);
        msgl_kv_pool pool;
        pool.k_pool = k.data_ptr();
        pool.v_pool = v.data_ptr();
        pool.num_slots = k.size(0);
        pool.page_size = ps;
        pool.num_kv_heads = size32(k.size(1), "k_pool");
        pool.head_dim = size32(k.size(2), "k_pool");
        msgl_page_table pt;
        pt.page_ids = i32(pages);
        pt.stride = pt.width = size32(pages.size(1), "page_table");

        c10::cuda::CUDAGuard guard((c10::DeviceIndex)dev);
        const c10::cuda::CUDAStream stream = stream_of(a[14], dev);
        at::Tensor out, lse;
        if (a[10] != Py_None) out = checked(a[10], "out", at::kBFloat16, dev);
        if (a[11] != Py_None) lse = checked(a[11], "lse", at::kFloat, dev);
        if (out.defined() && out.sizes() != q.sizes()) refuse("%s must be [B, Hq, D]", "out");
        if (lse.defined() && (lse.dim() != 2 || lse.size(0) != B || lse.size(1) != hq)) refuse("%s must be [B, Hq]", "lse");
        void *ws = nullptr;
        size_t ws_bytes = 0;
        if (a[12] != Py_None) {
            const at::Tensor &t = tensor(a[12], "workspace");
            if (!t.is_cuda() || t.get_device() != dev || !t.is_contiguous())
                refuse("%s must be contiguous and on q's device", "workspace");
            ws = t.data_ptr();
            ws_bytes = t.nbytes();
        }
        const bool own_scratch = a[12] == Py_None;
        msgl_status rc;
        {
            NoGil no_gil;
            if (!out.defined()) out = fresh(q.sizes(), at::kBFloat16, dev, stream);
            if (!lse.defined()) lse = fresh({q.size(0), q.size(1)}, at::kFloat, dev, stream);
            // Scratch, when the caller brings none: from the caching allocator in the stream's order, and
            // back to it once the kernels are queued (its next user on the stream comes behind them).
            struct Scratch {
                void *p = nullptr;
                ~Scratch() {
                    if (p) c10::cuda::CUDACachingAllocator::raw_delete(p);
                }
            } scratch;
            if (own_scratch) {
                ws_bytes = msgl_decode_shared_workspace_size(B, hq, pool.num_kv_heads, pool.head_dim, max_seq);
                if (ws_bytes)
                    ws = scratch.p = c10::cuda::CUDACachingAllocator::raw_alloc_with_stream(ws_bytes, stream.stream());
            }
            rc = msgl_attn_decode_shared(&pool, &pt, q.data_ptr(), hq, i32(first), i32(shared), i32(seq), B, max_seq,
                                         sharing, (float)scale, out.data_ptr(), static_cast<float *>(lse.data_ptr()), ws,
                                         ws_bytes, status, raw(stream));
        }
        if (rc != MSGL_OK) return done(rc);
        PyObject *x = THPVariable_Wrap(out), *y = THPVariable_Wrap(lse);
        PyObject *r = x && y ? PyTuple_Pack(2, x, y) : nullptr;
        Py_XDECREF(x);
        Py_XDECREF(y);
        return r;
    });
}

// A tensor [T, H, D] of bf16 whose heads stand one behind the other; its tokens may be further apart.
const at::Tensor &token_rows(PyObject *o, const char *name, int &dev, int64_t &stride) {
    const at::Tensor &t = tensor(o, name);
    if (!t.is_cuda()) refuse("%s must be a CUDA tensor", name);
    if (t.scalar_type() != at::kBFloat16) refuse("%s must be torch.bfloat16", name);
    if (dev < 0) dev = t.get_device();
    if (t.get_device() != dev) refuse("%s must be on the same CUDA device as the other tensors", name);
    if (t.dim() != 3) refuse("%s must be [T, heads, D]", name);
    if (t.numel() > 0 && ((t.size(2) > 1 && t.stride(2) != 1) || (t.size(1) > 1 && t.stride(1) != t.size(2))))
        refuse("%s must have contiguous heads (only tokens may be strided)", name);
    stride = t.size(0) > 1 ? t.stride(0) : t.size(1) * t.size(2);
    return t;
}

double number(PyObject *o) {
    const double v = PyFloat_AsDouble(o);
    if (v == -1.0 && PyErr_Occurred()) throw Refused{};
    return v;
}

const char *bytes_of(PyObject *o, const char *name, Py_ssize_t size) {
    char *p;
    Py_ssize_t n;
    if (PyBytes_AsStringAndSize(o, &p, &n)) throw Refused{};
    if (n != size) refuse("%s has the wrong size", name);
    return p;
}

// An optional array of n int32 entries; NULL when it is None.
int32_t *entries(PyObject *o, const char *name, int64_t n, int &dev) {
    if (o == Py_None) return nullptr;
    const at::Tensor &t = checked(o, name, at::kInt, dev);
    if (t.numel() != n) refuse("%s does not have the right number of entries", name);
    return i32(t);
}

PyObject *tuple_of(std::initializer_list<at::Tensor> ts) {
    PyObject *r = PyTuple_New((Py_ssize_t)ts.size());
    Py_ssize_t i = 0;
    for (const at::Tensor &t : ts) {
        PyObject *x = r ? THPVariable_Wrap(t) : nullptr;
        if (!x) {
            Py_XDECREF(r);
            return nullptr;
        }
        PyTuple_SET_ITEM(r, i++, x);
    }
    return r;
}

// (k_pool, v_pool, page_size, q, k, v, positions, out_loc, turns, axes, adjacent, factor, q_out | None,
//  q_norm | None, k_norm | None, eps, status | None, stream | None) -> q_out or the status
PyObject *rope_store_kv(PyObject *, PyObject *const *a, Py_ssize_t n) {
    if (!arity(n, 18)) return nullptr;
    return guarded([&]() -> PyObject * {
        int dev = -1;
        msgl_new_tokens tok{};
        const at::Tensor &q = token_rows(a[3], "q", dev, tok.q_stride);
        const at::Tensor &k = token_rows(a[4], "k", dev, tok.k_stride);
        const at::Tensor &v = token_rows(a[5], "v", dev, tok.v_stride);
        const at::Tensor &k_pool = checked(a[0], "k_pool", at::kBFloat16, dev);
        const at::Tensor &v_pool = checked(a[1], "v_pool", at::kBFloat16, dev);
        const at::Tensor &loc = checked(a[7], "out_loc", at::kInt, dev);
        if (k_pool.dim() != 3 || v_pool.sizes() != k_pool.sizes())
            refuse("%s and v_pool must both be [num_slots, Hkv, D]", "k_pool");
        const int64_t T = q.size(0), D = k_pool.size(2);
        if (k.size(0) != T || v.size(0) != T || loc.numel() != T) refuse("%s, k, v and out_loc must have T tokens", "q");
        if (q.size(2) != D || k.size(2) != D || v.size(2) != D || k.size(1) != k_pool.size(1) || v.size(1) != k_pool.size(1))
            refuse("%s and the pool must have the same head_dim, and k and v its heads", "q");
        const at::Tensor &pos = tensor(a[6], "positions");
        if (!pos.is_cuda() || pos.get_device() != dev || pos.scalar_type() != at::kInt)
            refuse("%s must be torch.int32 on the same CUDA device as the other tensors", "positions");
        if (pos.dim() < 1 || pos.dim() > 2 || pos.size(-1) != T || (T > 1 && pos.stride(-1) != 1))
            refuse("%s must be [T] or [axes, T] with contiguous rows", "positions");
        msgl_rope rope{};
        rope.num_pairs = size32(PyBytes_Check(a[9]) ? PyBytes_GET_SIZE(a[9]) : -1, "axes");
        rope.axes = reinterpret_cast<const uint8_t *>(bytes_of(a[9], "axes", rope.num_pairs));
        const at::Tensor &turns = checked(a[8], "rope.turns", at::kLong, dev);
        if (turns.numel() != rope.num_pairs) refuse("%s must have an entry for each of rope.axes", "rope.turns");
        rope.turns = static_cast<const uint64_t *>(turns.data_ptr());
        rope.num_axes = pos.dim() == 2 ? size32(pos.size(0), "positions") : 1;
        rope.adjacent = (int32_t)integer(a[10]);
        rope.factor = (float)number(a[11]);
        const void *norm[2] = {};
        for (int i = 0; i < 2; ++i) {
            if (a[13 + i] == Py_None) continue;
            const at::Tensor &t = checked(a[13 + i], i ? "k_norm" : "q_norm", at::kBFloat16, dev);
            if (t.numel() != D) refuse("%s must be [D]", i ? "k_norm" : "q_norm");
            norm[i] = t.data_ptr();
        }
        const float eps = (float)number(a[15]);
        msgl_kv_pool pool;
        pool.k_pool = k_pool.data_ptr();
        pool.v_pool = v_pool.data_ptr();
        pool.num_slots = k_pool.size(0);
        pool.page_size = integer32(a[2], "page_size");
        pool.num_kv_heads = size32(k_pool.size(1), "k_pool");
        pool.head_dim = size32(D, "k_pool");
        uint32_t *status = status_ptr(a[16], dev);
        c10::cuda::CUDAGuard guard((c10::DeviceIndex)dev);
        const c10::cuda::CUDAStream stream = stream_of(a[17], dev);
        at::Tensor out;
        if (a[12] != Py_None) {
            out = token_rows(a[12], "q_out", dev, tok.out_stride);
            if (out.sizes() != q.sizes()) refuse("%s must be [T, Hq, D]", "q_out");
        }
        tok.q = q.data_ptr();
        tok.k = k.data_ptr();
        tok.v = v.data_ptr();
        tok.positions = i32(pos);
        tok.axis_stride = pos.dim() == 2 && pos.size(0) > 1 ? pos.stride(0) : T;
        tok.out_loc = i32(loc);
        tok.n_tokens = size32(T, "q");
        tok.num_q_heads = size32(q.size(1), "q");
        msgl_status rc;
        {
            NoGil no_gil;
            if (!out.defined()) {
                out = fresh(q.sizes(), at::kBFloat16, dev, stream);
                tok.out_stride = q.size(1) * q.size(2);
            }
            tok.q_out = out.data_ptr();
            rc = msgl_rope_store_kv(&pool, &tok, &rope, norm[0], norm[1], eps, status, raw(stream));
        }
        if (rc != MSGL_OK) return done(rc);
        return THPVariable_Wrap(out);
    });
}

// (target, draft | None, tokens, cu_ext, accept_u, sample_u, cached_lens | None, accepted | None, out_tokens | None,
//  kv_lens | None, status | None, stream | None) -> (accepted, out_tokens, kv_lens) or the status
PyObject *verify_drafts(PyObject *, PyObject *const *a, Py_ssize_t n) {
    if (!arity(n, 12)) return nullptr;
    return guarded([&]() -> PyObject * {
        int dev = -1;
        const at::Tensor &tokens = checked(a[2], "tokens", at::kInt, dev);
        const at::Tensor &cu = checked(a[3], "cu_ext", at::kInt, dev);
        const at::Tensor &au = checked(a[4], "accept_u", at::kFloat, dev);
        const at::Tensor &su = checked(a[5], "sample_u", at::kFloat, dev);
        const int64_t T = tokens.numel();
        msgl_draft_batch d{};
        auto probs = [&](PyObject *o, const char *name, int64_t &stride) -> const at::Tensor & {
            const at::Tensor &t = tensor(o, name);
            if (!t.is_cuda() || t.get_device() != dev) refuse("%s must be on the same CUDA device as tokens", name);
            if (t.scalar_type() != at::kFloat && t.scalar_type() != at::kBFloat16)
                refuse("%s must be torch.float32 or torch.bfloat16", name);
            if (t.dim() != 2 || t.size(0) != T) refuse("%s must be [T, vocab]", name);
            if (t.size(1) > 1 && t.numel() > 0 && t.stride(1) != 1) refuse("%s must have contiguous rows", name);
            stride = t.size(0) > 1 ? t.stride(0) : t.size(1);
            return t;
        };
        const at::Tensor &p = probs(a[0], "target_probs", d.target_stride);
        d.vocab = size32(p.size(1), "target_probs");
        d.is_bf16 = p.scalar_type() == at::kBFloat16;
        d.target = p.data_ptr();
        if (a[1] != Py_None) {
            const at::Tensor &q = probs(a[1], "draft_probs", d.draft_stride);
            if (q.scalar_type() != p.scalar_type() || q.size(1) != p.size(1))
                refuse("%s must have the type and vocab of target_probs", "draft_probs");
            d.draft = q.data_ptr();
        }
        const int64_t B = su.numel();
        if (cu.numel() != B + 1) refuse("%s must be [B + 1] for the [B] entries of sample_u", "cu_ext");
        if (au.numel() != T) refuse("%s must be [T]", "accept_u");
        d.cached_lens = entries(a[6], "cached_lens", B, dev);
        d.tokens = i32(tokens);
        d.cu_ext = i32(cu);
        d.accept_u = static_cast<const float *>(au.data_ptr());
        d.sample_u = static_cast<const float *>(su.data_ptr());
        d.num_reqs = size32(B, "sample_u");
        d.total_tokens = size32(T, "tokens");
        uint32_t *status = status_ptr(a[10], dev);
        c10::cuda::CUDAGuard guard((c10::DeviceIndex)dev);
        const c10::cuda::CUDAStream stream = stream_of(a[11], dev);
        at::Tensor accepted, out, lens;
        const bool given = a[7] != Py_None;
        if (given) {
            accepted = checked(a[7], "accepted", at::kInt, dev);
            out = checked(a[8], "out_tokens", at::kInt, dev);
            lens = checked(a[9], "kv_lens", at::kInt, dev);
            if (accepted.numel() != B || out.numel() != T || lens.numel() != B)
                refuse("%s must hold [B], [T] and [B] entries", "out");
        }
        msgl_status rc;
        {
            NoGil no_gil;
            if (!given) {
                const at::Tensor both = fresh({2, B}, at::kInt, dev, stream);
                accepted = row_of(both, 0);
                lens = row_of(both, 1);
                out = fresh({T}, at::kInt, dev, stream);
                // (rows outside all requests are not written)
                if (T && cudaMemsetAsync(out.data_ptr(), 0xff, 4 * (size_t)T, stream.stream()) != cudaSuccess)
                    throw std::runtime_error(cudaGetErrorString(cudaGetLastError()));
            }
            d.accepted = i32(accepted);
            d.out_tokens = i32(out);
            d.kv_lens = i32(lens);
            rc = msgl_verify_drafts(&d, status, raw(stream));
        }
        if (rc != MSGL_OK) return done(rc);
        if (given) Py_RETURN_NONE;
        return tuple_of({accepted, out, lens});
    });
}

struct Table {
    int32_t *at, rows, width;
};
Table table_of(PyObject *o, const char *name, int &dev) {
    const at::Tensor &t = checked(o, name, at::kInt, dev);
    if (t.dim() != 2) refuse("%s must be [rows, width]", name);
    return Table{i32(t), size32(t.size(0), name), size32(t.size(1), name)};
}

// (req_table, parent_rows, child_rows, lens, free_pages, num_slots, page_size, src | None, dst | None, tokens | None,
//  pages_taken | None, status | None, stream | None) -> (src, dst, tokens, pages_taken), None when they were given, or
//  the status
PyObject *fork_requests(PyObject *, PyObject *const *a, Py_ssize_t n) {
    if (!arity(n, 13)) return nullptr;
    return guarded([&]() -> PyObject * {
        int dev = -1;
        const Table table = table_of(a[0], "req_table", dev);
        const at::Tensor &parents = checked(a[1], "parent_rows", at::kInt, dev);
        const int64_t N = parents.numel();
        if (a[2] == Py_None || a[3] == Py_None) refuse("%s and lens must be CUDA tensors", "child_rows");
        const int32_t *children = entries(a[2], "child_rows", N, dev), *lens = entries(a[3], "lens", N, dev);
        const at::Tensor &free_pages = checked(a[4], "free_pages", at::kInt, dev);
        const int64_t slots = integer(a[5]);
        const int32_t ps = integer32(a[6], "page_size");
        uint32_t *status = status_ptr(a[11], dev);
        c10::cuda::CUDAGuard guard((c10::DeviceIndex)dev);
        const c10::cuda::CUDAStream stream = stream_of(a[12], dev);
        const int32_t forks = size32(N, "parent_rows"), num_free = size32(free_pages.numel(), "free_pages");
        msgl_fork_out out{};
        at::Tensor src, dst, tokens, taken;
        const bool given = a[7] != Py_None;
        if (given) {
            src = checked(a[7], "src", at::kInt, dev);
            dst = checked(a[8], "dst", at::kInt, dev);
            tokens = checked(a[9], "tokens", at::kInt, dev);
            taken = checked(a[10], "pages_taken", at::kInt, dev);
            if (src.numel() != N || dst.numel() != N || tokens.numel() != N || taken.numel() != 1)
                refuse("%s must hold [N], [N], [N] and [1] entries", "out");
        }
        msgl_status rc;
        {
            NoGil no_gil;
            if (!given) {
                const at::Tensor all = fresh({3, N}, at::kInt, dev, stream);
                src = row_of(all, 0);
                dst = row_of(all, 1);
                tokens = row_of(all, 2);
                taken = fresh({1}, at::kInt, dev, stream);
            }
            out.copy_src = i32(src);
            out.copy_dst = i32(dst);
            out.copy_tokens = i32(tokens);
            out.pages_taken = i32(taken);
            rc = msgl_fork_requests(slots, ps, table.at, table.rows, table.width, table.width, i32(parents), children, lens,
                                    forks, i32(free_pages), num_free, &out, status, raw(stream));
        }
        if (rc != MSGL_OK) return done(rc);
        if (given) Py_RETURN_NONE;
        return tuple_of({src, dst, tokens, taken});
    });
}

// (pools: sequence of objects with k, v and page_size, src, dst, tokens | None, count | None, status | None,
//  stream | None)
PyObject *copy_pages(PyObject *, PyObject *const *a, Py_ssize_t n) {
    if (!arity(n, 7)) return nullptr;
    return guarded([&]() -> PyObject * {
        struct Ref {
            PyObject *p;
            explicit Ref(PyObject *o) : p(o) {
                if (!p) throw Refused{};
            }
            Ref(const Ref &) = delete;
            ~Ref() { Py_DECREF(p); }
        };
        static PyObject *const names[3] = {PyUnicode_InternFromString("k"), PyUnicode_InternFromString("v"),
                                           PyUnicode_InternFromString("page_size")};
        int dev = -1;
        const at::Tensor &src = checked(a[1], "src", at::kInt, dev);
        const at::Tensor &dst = checked(a[2], "dst", at::kInt, dev);
        const int64_t N = src.numel();
        if (dst.numel() != N) refuse("%s must have an entry for each of src", "dst");
        const int32_t *tokens = entries(a[3], "tokens", N, dev), *count = entries(a[4], "count", 1, dev);
        // (a tuple of the caller's pools: what looks up their attributes may be Python code that changes a list)
        const Ref fast(PySequence_Fast(a[0], "pools must be a sequence of KVPool")), seq(PySequence_Tuple(fast.p));
        const Py_ssize_t pools = PyTuple_GET_SIZE(seq.p);
        std::vector<msgl_kv_pool> c((size_t)pools);
        for (Py_ssize_t i = 0; i < pools; ++i) {
            PyObject *pool = PyTuple_GET_ITEM(seq.p, i);
            const Ref ko(PyObject_GetAttr(pool, names[0])), vo(PyObject_GetAttr(pool, names[1])),
                po(PyObject_GetAttr(pool, names[2]));
            const at::Tensor &k = checked(ko.p, "k_pool", at::kBFloat16, dev), &v = checked(vo.p, "v_pool", at::kBFloat16, dev);
            if (k.dim() != 3 || v.sizes() != k.sizes()) refuse("%s and v_pool must both be [num_slots, Hkv, D]", "k_pool");
            c[i].k_pool = k.data_ptr();
            c[i].v_pool = v.data_ptr();
            c[i].num_slots = k.size(0);
            c[i].page_size = integer32(po.p, "page_size");
            c[i].num_kv_heads = size32(k.size(1), "k_pool");
            c[i].head_dim = size32(k.size(2), "k_pool");
        }
        uint32_t *status = status_ptr(a[5], dev);
        c10::cuda::CUDAGuard guard((c10::DeviceIndex)dev);
        const c10::cuda::CUDAStream stream = stream_of(a[6], dev);
        const int32_t pairs = size32(N, "src"), num_pools = size32(pools, "pools");
        msgl_status rc;
        {
            NoGil no_gil;
            rc = msgl_copy_pages(c.data(), num_pools, i32(src), i32(dst), tokens, pairs, count, status, raw(stream));
        }
        return done(rc);
    });
}

// The workspace that the caller brings, or scratch in `stream`'s order for the length of a call (its next user on
// the stream comes behind the call's kernels).
struct Workspace {
    void *p = nullptr, *own = nullptr;
    size_t bytes = 0;
    bool brought = false;
    Workspace(PyObject *o, int dev) {
        if (o == Py_None) return;
        const at::Tensor &t = tensor(o, "workspace");
        if (!t.is_cuda() || t.get_device() != dev || !t.is_contiguous())
            refuse("%s must be contiguous and on the other tensors' device", "workspace");
        p = t.data_ptr();
        bytes = t.nbytes();
        brought = true;
    }
    Workspace(const Workspace &) = delete;
    void need(size_t n, const c10::cuda::CUDAStream &stream) {
        if (brought || !n) return;
        p = own = c10::cuda::CUDACachingAllocator::raw_alloc_with_stream(n, stream.stream());
        bytes = n;
    }
    ~Workspace() {
        if (own) c10::cuda::CUDACachingAllocator::raw_delete(own);
    }
};

// The arguments that free_pages and compact_pages begin with: (req_table, lens, num_slots, page_size, req_rows | None,
// held | None).
struct PageMap {
    Table table;
    const int32_t *lens, *rows;
    const uint8_t *held;
    int64_t slots, pages;
    int32_t reqs, ps;
};
PageMap page_map(PyObject *const *a, int &dev) {
    PageMap m{};
    m.table = table_of(a[0], "req_table", dev);
    const at::Tensor &lens = checked(a[1], "lens", at::kInt, dev);
    m.lens = i32(lens);
    m.reqs = size32(lens.numel(), "lens");
    m.slots = integer(a[2]);
    m.ps = integer32(a[3], "page_size");
    m.rows = entries(a[4], "req_rows", m.reqs, dev);
    // (the sizes below need a page size that divides; the C call says what else is wrong with it)
    if (m.ps <= 0 || m.slots < 0 || m.slots % m.ps != 0 || m.slots / m.ps > INT32_MAX)
        refuse("%s must be a non-negative multiple of page_size, of less than 2^31 pages", "num_slots");
    m.pages = m.slots / m.ps;
    if (a[5] != Py_None) {
        const at::Tensor &t = tensor(a[5], "held");
        if (!t.is_cuda() || t.get_device() != dev || !t.is_contiguous())
            refuse("%s must be contiguous and on req_table's device", "held");
        if (t.scalar_type() != at::kByte && t.scalar_type() != at::kBool) refuse("%s must be torch.uint8 or torch.bool", "held");
        if (t.numel() != m.pages) refuse("%s must have an entry for every page", "held");
        m.held = static_cast<const uint8_t *>(t.data_ptr());
    }
    return m;
}

// (.. , pages | None, num_free | None, workspace | None, status | None, stream | None) -> (pages, num_free), None when they were given,
// or the status
PyObject *free_pages(PyObject *, PyObject *const *a, Py_ssize_t n) {
    if (!arity(n, 11)) return nullptr;
    return guarded([&]() -> PyObject * {
        int dev = -1;
        const PageMap m = page_map(a, dev);
        uint32_t *status = status_ptr(a[9], dev);
        c10::cuda::CUDAGuard guard((c10::DeviceIndex)dev);
        const c10::cuda::CUDAStream stream = stream_of(a[10], dev);
        Workspace ws(a[8], dev);
        at::Tensor pages, count;
        const bool given = a[6] != Py_None;
        if (given) {
            pages = checked(a[6], "pages", at::kInt, dev);
            count = checked(a[7], "num_free", at::kInt, dev);
            if (pages.numel() != m.pages || count.numel() != 1) refuse("%s must hold [num_pages] and [1] entries", "out");
        }
        msgl_status rc;
        {
            NoGil no_gil;
            if (!given) {
                pages = fresh({m.pages}, at::kInt, dev, stream);
                count = fresh({1}, at::kInt, dev, stream);
            }
            ws.need(msgl_page_map_workspace_size(m.slots, m.ps), stream);
            rc = msgl_free_pages(m.slots, m.ps, m.table.at, m.table.rows, m.table.width, m.table.width, m.rows, m.lens,
                                 m.reqs, m.held, i32(pages), i32(count), ws.p, ws.bytes, status, raw(stream));
        }
        if (rc != MSGL_OK) return done(rc);
        if (given) Py_RETURN_NONE;
        return tuple_of({pages, count});
    });
}

// (.. , table_out, remap | None, src | None, dst | None, num_moves | None, num_used | None, workspace | None,
//  status | None, stream | None) -> (remap, src, dst, num_moves, num_used), None when they were given, or the status
PyObject *compact_pages(PyObject *, PyObject *const *a, Py_ssize_t n) {
    if (!arity(n, 15)) return nullptr;
    return guarded([&]() -> PyObject * {
        int dev = -1;
        const PageMap m = page_map(a, dev);
        const Table to = table_of(a[6], "out.page_table", dev);
        if (to.rows != m.table.rows || to.width != m.table.width) refuse("%s must have req_table's size", "out.page_table");
        uint32_t *status = status_ptr(a[13], dev);
        c10::cuda::CUDAGuard guard((c10::DeviceIndex)dev);
        const c10::cuda::CUDAStream stream = stream_of(a[14], dev);
        Workspace ws(a[12], dev);
        at::Tensor remap, src, dst, moves, used;
        const bool given = a[7] != Py_None;
        if (given) {
            remap = checked(a[7], "remap", at::kInt, dev);
            src = checked(a[8], "src", at::kInt, dev);
            dst = checked(a[9], "dst", at::kInt, dev);
            moves = checked(a[10], "num_moves", at::kInt, dev);
            used = checked(a[11], "num_used", at::kInt, dev);
            if (remap.numel() != m.pages || src.numel() != m.pages / 2 || dst.numel() != m.pages / 2 || moves.numel() != 1 ||
                used.numel() != 1)
                refuse("%s must hold [num_pages], twice [num_pages // 2], and [1] and [1] entries", "out");
        }
        msgl_compact_out out{};
        msgl_status rc;
        {
            NoGil no_gil;
            if (!given) {
                remap = fresh({m.pages}, at::kInt, dev, stream);
                const at::Tensor both = fresh({2, m.pages / 2}, at::kInt, dev, stream);
                src = row_of(both, 0);
                dst = row_of(both, 1);
                const at::Tensor counts = fresh({2, 1}, at::kInt, dev, stream);
                moves = row_of(counts, 0);
                used = row_of(counts, 1);
            }
            out.page_ids = to.at;
            out.stride = to.width;
            out.remap = i32(remap);
            out.src = i32(src);
            out.dst = i32(dst);
            out.num_moves = i32(moves);
            out.num_used = i32(used);
            ws.need(msgl_page_map_workspace_size(m.slots, m.ps), stream);
            rc = msgl_compact_pages(m.slots, m.ps, m.table.at, m.table.rows, m.table.width, m.table.width, m.rows, m.lens,
                                    m.reqs, m.held, &out, ws.p, ws.bytes, status, raw(stream));
        }
        if (rc != MSGL_OK) return done(rc);
        if (given) Py_RETURN_NONE;
        return tuple_of({remap, src, dst, moves, used});
    });
}

PyMethodDef methods[] = {
    {"rope_store_kv", (PyCFunction)(void (*)(void))rope_store_kv, METH_FASTCALL, nullptr},
    {"verify_drafts", (PyCFunction)(void (*)(void))verify_drafts, METH_FASTCALL, nullptr},
    {"fork_requests", (PyCFunction)(void (*)(void))fork_requests, METH_FASTCALL, nullptr},
    {"copy_pages", (PyCFunction)(void (*)(void))copy_pages, METH_FASTCALL, nullptr},
    {"free_pages", (PyCFunction)(void (*)(void))free_pages, METH_FASTCALL, nullptr},
    {"compact_pages", (PyCFunction)(void (*)(void))compact_pages, METH_FASTCALL, nullptr},
    {"step_tables", (PyCFunction)(void (*)(void))step_tables, METH_FASTCALL, nullptr},
    {"shared_prefixes", (PyCFunction)(void (*)(void))shared_prefixes, METH_FASTCALL, nullptr},
    {"attn_decode_shared", (PyCFunction)(void (*)(void))attn_decode_shared, METH_FASTCALL, nullptr},
    {nullptr, nullptr, 0, nullptr},
};

PyModuleDef module = {PyModuleDef_HEAD_INIT, "_msgl_binding", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__msgl_binding(void) { return PyModule_Create(&module); }
