// streaming_binding.cpp -- the torch side of the streaming calls (attn.py:
// cache_plan, cache_append, cached, norm_residual): looks at the tensors,
// allocates what the call returns and calls the C entry point.
//
// A streaming step is many small calls.  With the marshalling in Python one took
// 9 us (append) to 22 us (attention) on the host, launches included, more than
// its kernels; with this module 4 to 9.  The entry points are given as
// addresses, so that the library stays the one that attn.load() opened (release
// or debug build).
#define PY_SSIZE_T_CLEAN
#include <Python.h>

#include <ATen/ATen.h>
#include <ATen/core/LegacyTypeDispatch.h>
#include <ATen/cuda/EmptyTensor.h>
#include <c10/cuda/CUDACachingAllocator.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include <algorithm>
#include <optional>

#include "vggt_attn.h"

namespace {

using at::ScalarType;

const at::Tensor &tensor(PyObject *o, const char *name)
{
    TORCH_CHECK_TYPE(THPVariable_Check(o), name, ": expected a CUDA tensor");
    return THPVariable_Unpack(o);
}

std::optional<at::Tensor> maybe(PyObject *o, const char *name)
{
    if (o == Py_None)
        return std::nullopt;
    return tensor(o, name);
}

int64_t integer(PyObject *o)
{
    const long long v = PyLong_AsLongLong(o);
    if (v == -1 && PyErr_Occurred())
        throw python_error();
    return v;
}

int32_t int32(PyObject *o, const char *name)
{
    const int64_t v = integer(o);
    TORCH_CHECK_VALUE(v >= INT32_MIN && v <= INT32_MAX, name, ": outside the 32-bit range");
    return static_cast<int32_t>(v);
}

double number(PyObject *o)
{
    const double v = PyFloat_AsDouble(o);
    if (v == -1.0 && PyErr_Occurred())
        throw python_error();
    return v;
}

bool truth(PyObject *o)
{
    const int v = PyObject_IsTrue(o);
    if (v < 0)
        throw python_error();
    return v != 0;
}

template <typename F>
F *entry(PyObject *address)
{
    return reinterpret_cast<F *>(static_cast<uintptr_t>(integer(address)));
}

// The device and the stream of a call.  Buffers of a call on another stream
// than torch's current one are allocated on that stream: memory that was freed
// on the current stream may still be in use on it.  What is returned is freed
// only after the work of the current stream that reads it.
struct Call {
    at::AutoDispatchBelowADInplaceOrView below_autograd;  // results are plain tensors: no view or gradient to track
    c10::cuda::CUDAGuard device;
    c10::cuda::CUDAStream current;
    std::optional<c10::cuda::CUDAStream> other;

    Call(const at::Tensor &first, const char *name, PyObject *stream)
        : device(index_of(first, name)), current(c10::cuda::getCurrentCUDAStream())
    {
        if (stream == Py_None)
            return;
        int64_t raw;
        if (PyLong_Check(stream)) {
            raw = integer(stream);
        } else {
            PyObject *attr = PyObject_GetAttrString(stream, "cuda_stream");
            if (!attr)
                throw python_error();
            raw = PyLong_AsLongLong(attr);
            Py_DECREF(attr);
            if (raw == -1 && PyErr_Occurred())
                throw python_error();
        }
        if (reinterpret_cast<cudaStream_t>(raw) != current.stream())
            other = c10::cuda::getStreamFromExternal(reinterpret_cast<cudaStream_t>(raw), current.device_index());
    }

    static c10::Device index_of(const at::Tensor &first, const char *name)
    {
        TORCH_CHECK_VALUE(first.is_cuda(), name, ": tensor must live on a CUDA device");
        return first.device();
    }

    void *stream() const { return other ? other->stream() : current.stream(); }

    at::Tensor empty(at::IntArrayRef shape, ScalarType type, bool returned = true) const
    {
        if (!other)
            return at::detail::empty_cuda(shape, type, current.device(), std::nullopt);
        at::Tensor t;
        {
            const c10::cuda::CUDAStreamGuard guard(*other);
            t = at::detail::empty_cuda(shape, type, current.device(), std::nullopt);
        }
        if (returned)
            c10::cuda::CUDACachingAllocator::recordStream(t.storage().data_ptr(), current);
        return t;
    }

    // The address of a tensor of the call.
    void *use(const at::Tensor &t, ScalarType type, const char *name, bool contiguous = true) const
    {
        TORCH_CHECK_VALUE(t.is_cuda(), name, ": tensor must live on a CUDA device");
        TORCH_CHECK_VALUE(t.device() == current.device(), name, ": tensor on ", t.device(), ", the call runs on ",
                          current.device());
        TORCH_CHECK_VALUE(t.scalar_type() == type, name, ": expected dtype ", type, ", got ", t.scalar_type());
        TORCH_CHECK_VALUE(!contiguous || t.is_contiguous(), name, ": tensor must be contiguous");
        return t.data_ptr();
    }

    void *use(const std::optional<at::Tensor> &t, ScalarType type, const char *name, bool contiguous = true) const
    {
        return t ? use(*t, type, name, contiguous) : nullptr;
    }
};

// Of the same sizes, with elements at the same places: a dimension of one element has no stride of its own.
bool alike(const at::Tensor &a, const at::Tensor &b)
{
    if (a.sizes() != b.sizes())
        return false;
    for (int64_t d = 0; d < a.dim(); ++d)
        if (a.size(d) > 1 && a.stride(d) != b.stride(d))
            return false;
    return true;
}

vggt_cache page_layout(const at::Tensor &k, const at::Tensor &v, int64_t n_heads, int64_t n_seqs, int64_t max_pages)
{
    TORCH_CHECK_VALUE(k.dim() == 4 && alike(k, v) && (k.stride(3) == 1 || k.size(3) == 1),
                      "k_pages, v_pages: [n_pages, n_kv_heads, page_size, head_dim] of the same strides, the last one 1");
    for (int64_t n : {k.size(0), k.size(1), k.size(2), k.size(3), n_heads, n_seqs, max_pages})
        TORCH_CHECK_VALUE(n <= INT32_MAX, "a size outside the 32-bit range");
    vggt_cache c;
    c.n_seqs = static_cast<int32_t>(n_seqs);
    c.n_heads = static_cast<int32_t>(n_heads);
    c.n_kv_heads = static_cast<int32_t>(k.size(1));
    c.head_dim = static_cast<int32_t>(k.size(3));
    c.page_size = static_cast<int32_t>(k.size(2));
    c.n_pages = static_cast<int32_t>(k.size(0));
    c.max_pages = static_cast<int32_t>(max_pages);
    // a single page or head has no stride of its own: any valid one does
    c.page_stride = k.size(0) == 1 ? 64 : k.stride(0);
    c.head_stride = k.size(1) == 1 ? 64 : k.stride(1);
    c.token_stride = k.stride(2);
    return c;
}

struct RowStrides {
    int64_t row, head;
};

RowStrides row_strides(const at::Tensor &x, const char *name)
{
    TORCH_CHECK_VALUE(x.stride(2) == 1 || x.size(2) == 1, name, ": the last dimension must be contiguous");
    RowStrides s{x.stride(0), x.size(1) > 1 ? x.stride(1) : 64};
    if (x.size(0) <= 1)
        s.row = std::max<int64_t>(64, s.head * x.size(1));
    return s;
}

// (status, results...), or the status alone.
template <typename... T>
PyObject *results(vggt_status status, T &&...values)
{
    PyObject *items[] = {PyLong_FromLong(status), values...};
    constexpr Py_ssize_t n = sizeof...(T) + 1;
    PyObject *out = PyTuple_New(n);
    for (Py_ssize_t i = 0; i < n; ++i) {
        if (!items[i] || !out) {
            Py_XDECREF(out);
            return nullptr;
        }
        PyTuple_SET_ITEM(out, i, items[i]);
    }
    return out;
}

PyObject *wrap(const at::Tensor &t)
{
    return THPVariable_Wrap(t);
}

PyObject *none()
{
    Py_INCREF(Py_None);
    return Py_None;
}

void expect_args(Py_ssize_t n, Py_ssize_t want)
{
    TORCH_CHECK_TYPE(n == want, "expected ", want, " arguments, got ", n);
}

// entry, cached_lens, new_lens, free_pages, n_free, block_table, page_size, n_rows, n_pages, stream, step, state
//
// step (or None): where cu_rows and the slots go, [n_seqs + 1 + n_rows] at least.  state (or None): the counts and
// kv_lens are copied there behind the kernel, [2 + n_seqs]; cached_lens and n_free may lie in it.
PyObject *plan(PyObject *, PyObject *const *a, Py_ssize_t n)
{
    HANDLE_TH_ERRORS
    expect_args(n, 12);
    const at::Tensor &cached = tensor(a[1], "cached_lens"), &fresh = tensor(a[2], "new_lens");
    const at::Tensor &free = tensor(a[3], "free_pages"), &n_free = tensor(a[4], "n_free");
    const at::Tensor &table = tensor(a[5], "block_table");
    TORCH_CHECK_VALUE(table.dim() == 2 && cached.numel() == table.size(0) && fresh.numel() == table.size(0) &&
                          n_free.numel() == 1,
                      "one cached length, new length and row of block_table per sequence, one n_free");
    TORCH_CHECK_VALUE(table.size(0) <= INT32_MAX && table.size(1) <= INT32_MAX && free.numel() <= INT32_MAX,
                      "a size outside the 32-bit range");
    const int64_t seqs = table.size(0);
    const int32_t rows = int32(a[7], "n_rows");
    const int64_t step_size = seqs + 1 + std::max(rows, 0);
    std::optional<at::Tensor> step = maybe(a[10], "step"), state = maybe(a[11], "state");
    TORCH_CHECK_VALUE((!step || step->numel() >= step_size) && (!state || state->numel() == 2 + seqs),
                      "step: [n_seqs + 1 + n_rows] at least, state: [2 + n_seqs]");
    const Call call(table, "block_table", a[9]);
    vggt_cache c{};
    c.n_seqs = static_cast<int32_t>(seqs);
    c.n_heads = c.n_kv_heads = 1;
    c.head_dim = 64;
    c.page_size = int32(a[6], "page_size");
    c.n_pages = int32(a[8], "n_pages");
    c.max_pages = static_cast<int32_t>(table.size(1));
    c.page_stride = c.head_stride = c.token_stride = 64;
    auto *in_cached = static_cast<const int32_t *>(call.use(cached, at::kInt, "cached_lens"));
    auto *in_fresh = static_cast<const int32_t *>(call.use(fresh, at::kInt, "new_lens"));
    auto *in_free = static_cast<const int32_t *>(call.use(free, at::kInt, "free_pages"));
    auto *in_n_free = static_cast<const int32_t *>(call.use(n_free, at::kInt, "n_free"));
    auto *in_table = static_cast<int32_t *>(call.use(table, at::kInt, "block_table"));
    // counts, lengths and the step in one buffer: every part starts on 4 bytes, which is all that is asked
    const at::Tensor out = call.empty({2 + seqs + (step ? 0 : step_size)}, at::kInt);
    int32_t *counts = out.mutable_data_ptr<int32_t>(), *lens = counts + 2;
    int32_t *offsets = step ? static_cast<int32_t *>(call.use(step, at::kInt, "step")) : lens + seqs;
    if (state)
        call.use(state, at::kInt, "state");
    const vggt_status status = entry<decltype(vggt_cache_plan)>(a[0])(
        c, in_cached, in_fresh, in_free, static_cast<int32_t>(free.numel()), in_n_free, in_table, rows, offsets, lens,
        offsets + seqs + 1, counts, call.stream());
    if (status != VGGT_OK)
        return results(status);
    if (state) {
        // not by the kernel: it reads the old values while it writes the new ones
        const c10::cuda::CUDAStreamGuard guard(call.other.value_or(call.current));
        state->copy_(out.as_strided({2 + seqs}, {1}, 0));
    }
    const at::Tensor &in = step ? *step : out;
    const int64_t first = step ? step->storage_offset() : 2 + seqs;
    auto part = [](const at::Tensor &t, int64_t at, int64_t size) { return wrap(t.as_strided({size}, {1}, at)); };
    return results(status, part(in, first, seqs + 1), part(out, 2, seqs), part(in, first + seqs + 1, rows),
                   part(out, 0, 2));
    END_HANDLE_TH_ERRORS
}

// entry, k, v, slots, k_pages, v_pages, stream
PyObject *append(PyObject *, PyObject *const *a, Py_ssize_t n)
{
    HANDLE_TH_ERRORS
    expect_args(n, 7);
    const at::Tensor &k = tensor(a[1], "k"), &v = tensor(a[2], "v"), &slots = tensor(a[3], "slots");
    const at::Tensor &k_pages = tensor(a[4], "k_pages"), &v_pages = tensor(a[5], "v_pages");
    TORCH_CHECK_VALUE(k.dim() == 3 && alike(k, v) && slots.dim() == 1 && slots.size(0) == k.size(0),
                      "k, v: [n_rows, n_kv_heads, head_dim] of the same strides, one slot per row");
    const vggt_cache c = page_layout(k_pages, v_pages, k.size(1), 1, 1);
    TORCH_CHECK_VALUE(k.size(1) == c.n_kv_heads && k.size(2) == c.head_dim && k.size(0) <= INT32_MAX,
                      "k, v: the heads and head_dim of the pages");
    const Call call(k_pages, "k_pages", a[6]);
    const RowStrides s = row_strides(k, "k, v");
    const vggt_status status = entry<decltype(vggt_cache_append)>(a[0])(
        c, call.use(k, at::kBFloat16, "k", false), call.use(v, at::kBFloat16, "v", false), s.row, s.head,
        static_cast<const int32_t *>(call.use(slots, at::kInt, "slots")), static_cast<int32_t>(k.size(0)),
        call.use(k_pages, at::kBFloat16, "k_pages", false), call.use(v_pages, at::kBFloat16, "v_pages", false),
        call.stream());
    return PyLong_FromLong(status);
    END_HANDLE_TH_ERRORS
}

// entry, entry of the workspace size, q, k_pages, v_pages, block_table, cu_rows, kv_lens, causal_unit, scale,
// want_lse, workspace, o, stream
PyObject *attend(PyObject *, PyObject *const *a, Py_ssize_t n)
{
    HANDLE_TH_ERRORS
    expect_args(n, 14);
    const at::Tensor &q = tensor(a[2], "q"), &k_pages = tensor(a[3], "k_pages"), &v_pages = tensor(a[4], "v_pages");
    const at::Tensor &table = tensor(a[5], "block_table"), &cu_rows = tensor(a[6], "cu_rows");
    const at::Tensor &kv_lens = tensor(a[7], "kv_lens");
    TORCH_CHECK_VALUE(q.dim() == 3 && k_pages.dim() == 4 && q.size(2) == k_pages.size(3) && q.size(0) <= INT32_MAX,
                      "q: [n_rows, n_heads, head_dim]");
    TORCH_CHECK_VALUE(table.dim() == 2 && kv_lens.numel() == table.size(0) && cu_rows.numel() == table.size(0) + 1,
                      "one row of block_table and one length per sequence, one row offset more");
    std::optional<at::Tensor> workspace = maybe(a[11], "workspace"), o = maybe(a[12], "o"), lse;
    TORCH_CHECK_VALUE(!o || o->sizes() == q.sizes(), "o: the shape of q");
    const vggt_cache c = page_layout(k_pages, v_pages, q.size(1), table.size(0), table.size(1));
    const Call call(q, "q", a[13]);
    const RowStrides s = row_strides(q, "q");
    const int32_t rows = static_cast<int32_t>(q.size(0));
    void *in_q = call.use(q, at::kBFloat16, "q", false);
    void *in_k = call.use(k_pages, at::kBFloat16, "k_pages", false);
    void *in_v = call.use(v_pages, at::kBFloat16, "v_pages", false);
    auto *in_table = static_cast<const int32_t *>(call.use(table, at::kInt, "block_table"));
    auto *in_cu = static_cast<const int32_t *>(call.use(cu_rows, at::kInt, "cu_rows"));
    auto *in_kv = static_cast<const int32_t *>(call.use(kv_lens, at::kInt, "kv_lens"));
    if (!o)
        o = call.empty(q.sizes(), at::kBFloat16);
    void *out_o = call.use(o, at::kBFloat16, "o");
    if (truth(a[10]))
        lse = call.empty({q.size(0), q.size(1)}, at::kFloat);
    size_t bytes;
    if (workspace) {
        bytes = workspace->nbytes();
    } else if ((bytes = entry<decltype(vggt_attn_cached_workspace_bytes)>(a[1])(c, rows)) > 0) {
        workspace = call.empty({static_cast<int64_t>(bytes)}, at::kByte, false);
    }
    void *ws = workspace ? call.use(*workspace, workspace->scalar_type(), "workspace") : nullptr;
    const vggt_status status = entry<decltype(vggt_attn_cached)>(a[0])(
        c, in_q, s.row, s.head, in_k, in_v, in_table, in_cu, in_kv, rows, int32(a[8], "causal_unit"), out_o,
        lse ? lse->mutable_data_ptr<float>() : nullptr, ws, bytes, static_cast<float>(number(a[9])), call.stream());
    if (status != VGGT_OK)
        return results(status);
    return results(status, a[12] == Py_None ? wrap(*o) : (Py_INCREF(a[12]), a[12]), lse ? wrap(*lse) : none());
    END_HANDLE_TH_ERRORS
}

// entry, x, y, kind, eps, scale, gate, rows_per_gate, post_norm, post_weight, post_bias, weight, bias, want_h,
// inplace, stream
PyObject *norm(PyObject *, PyObject *const *a, Py_ssize_t n)
{
    HANDLE_TH_ERRORS
    expect_args(n, 16);
    const at::Tensor &x = tensor(a[1], "x");
    const std::optional<at::Tensor> y = maybe(a[2], "y"), gate = maybe(a[6], "gate");
    TORCH_CHECK_VALUE(x.dim() == 2 && (!y || y->sizes() == x.sizes()), "x, y: [n_rows, n_cols]");
    const int64_t rows = x.size(0), cols = x.size(1);
    TORCH_CHECK_VALUE(cols <= INT32_MAX, "x: too many columns");
    const int32_t rows_per_gate = gate ? int32(a[7], "rows_per_gate") : 0;
    TORCH_CHECK_VALUE(!gate || (rows_per_gate >= 1 && gate->dim() == 2 &&
                                gate->size(0) == (rows + rows_per_gate - 1) / rows_per_gate && gate->size(1) == cols),
                      "gate: [ceil(n_rows / rows_per_gate), n_cols]");
    TORCH_CHECK_VALUE(x.scalar_type() == at::kFloat || x.scalar_type() == at::kBFloat16, "x: float32 or bfloat16");
    const Call call(x, "x", a[15]);
    auto factors = [&](PyObject *o, const char *name) -> const float * {
        const std::optional<at::Tensor> t = maybe(o, name);
        TORCH_CHECK_VALUE(!t || (t->dim() == 1 && t->size(0) == cols), name, ": [n_cols]");
        return static_cast<const float *>(call.use(t, at::kFloat, name));
    };
    auto stride = [&](const at::Tensor &t, const char *name) {
        TORCH_CHECK_VALUE(t.stride(1) == 1 || cols == 1, name, ": the last dimension must be contiguous");
        return rows > 1 ? t.stride(0) : cols;
    };
    vggt_norm p{};
    p.n_rows = rows;
    p.n_cols = static_cast<int32_t>(cols);
    p.kind = int32(a[3], "kind");
    p.x_fp32 = x.scalar_type() == at::kFloat;
    p.post_norm = truth(a[8]);
    p.rows_per_gate = rows_per_gate;
    p.eps = static_cast<float>(number(a[4]));
    p.x_stride = stride(x, "x");
    p.y_stride = y ? stride(*y, "y") : cols;
    p.out_stride = p.h_stride = cols;
    void *in_x = call.use(x, x.scalar_type(), "x", false);
    void *in_y = call.use(y, at::kBFloat16, "y", false);
    const float *post_w = factors(a[9], "post_weight"), *post_b = factors(a[10], "post_bias");
    const float *scale = factors(a[5], "scale"), *w = factors(a[11], "weight"), *b = factors(a[12], "bias");
    void *in_gate = call.use(gate, at::kBFloat16, "gate");
    std::optional<at::Tensor> out, h;
    void *out_x = nullptr;
    if (y && truth(a[14])) {
        p.out_stride = p.x_stride;
        out_x = in_x;
    } else if (y) {
        out = call.empty(x.sizes(), x.scalar_type());
        out_x = out->data_ptr();
    }
    if (truth(a[13]))
        h = call.empty(x.sizes(), at::kBFloat16);
    const vggt_status status = entry<decltype(vggt_norm_residual)>(a[0])(
        p, in_x, in_y, post_w, post_b, scale, in_gate, w, b, out_x, h ? h->data_ptr() : nullptr, call.stream());
    if (status != VGGT_OK)
        return results(status);
    return results(status, out ? wrap(*out) : (Py_INCREF(a[1]), a[1]), h ? wrap(*h) : none());
    END_HANDLE_TH_ERRORS
}

PyMethodDef methods[] = {
    {"plan", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(plan)), METH_FASTCALL, nullptr},
    {"append", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(append)), METH_FASTCALL, nullptr},
    {"attend", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(attend)), METH_FASTCALL, nullptr},
    {"norm", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(norm)), METH_FASTCALL, nullptr},
    {nullptr, nullptr, 0, nullptr}};

#ifndef VGGT_BUILT_FOR
#define VGGT_BUILT_FOR "built by hand"
#endif

PyModuleDef module = {PyModuleDef_HEAD_INIT, "_streaming", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

} // namespace

PyMODINIT_FUNC PyInit__streaming()
{
    PyObject *m = PyModule_Create(&module);
    // torch's and Python's versions; the build looks for them to see whether the module is theirs
    if (m && PyModule_AddStringConstant(m, "built_for", VGGT_BUILT_FOR) < 0) {
        Py_DECREF(m);
        return nullptr;
    }
    return m;
}
