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
        refuse("%s must be torch.%s", name, type == at::kInt ? "int32" : type == at::kFloat ? "float32" : "bfloat16");
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

PyMethodDef methods[] = {
    {"step_tables", (PyCFunction)(void (*)(void))step_tables, METH_FASTCALL, nullptr},
    {"shared_prefixes", (PyCFunction)(void (*)(void))shared_prefixes, METH_FASTCALL, nullptr},
    {"attn_decode_shared", (PyCFunction)(void (*)(void))attn_decode_shared, METH_FASTCALL, nullptr},
    {nullptr, nullptr, 0, nullptr},
};

PyModuleDef module = {PyModuleDef_HEAD_INIT, "_msgl_binding", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__msgl_binding(void) { return PyModule_Create(&module); }
