// The calls of a step whose host cost shows (kv_plan_step, kv_append,
// paged_attention_decode_scored, paged_attention_prefill_scored) on torch tensors:
// argument marshalling only, like the ctypes binding, but without its 10-20 us of
// interpreter time around kernels of 6-12 us.  A call checks its tensors, takes
// the current stream, allocates its results and goes through the C ABI.
//
// Each function returns its results, or the call's kv_status as an int when that
// is not KV_OK; wrong tensors raise ValueError.
#include <Python.h>

#include <ATen/core/Tensor.h>
#include <ATen/ops/empty.h>
#include <ATen/ops/empty_like.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/autograd/python_variable.h>

#include <stdexcept>
#include <string>

#include "pagedkv.h"

namespace {

// A wrong argument: becomes a Python ValueError.
struct BadArgument : std::runtime_error {
    using std::runtime_error::runtime_error;
};
// A Python exception is already set.
struct PythonError {};

const at::Tensor& tensor(PyObject* o, const char* name) {
    if (!THPVariable_Check(o)) throw BadArgument(std::string(name) + " must be a CUDA tensor");
    return THPVariable_Unpack(o);
}

std::string text(c10::IntArrayRef s) {
    std::string t = "[";
    for (size_t i = 0; i < s.size(); ++i) t += (i ? ", " : "") + std::to_string(s[i]);
    return t + "]";
}

// Device pointer of a dense CUDA tensor of `type` on `device`.
void* address(const at::Tensor& t, const char* name, at::ScalarType type, int device) {
    if (!t.is_cuda()) throw BadArgument(std::string(name) + " must be a CUDA tensor");
    if (!t.is_contiguous()) throw BadArgument(std::string(name) + " must be contiguous");
    if (t.scalar_type() != type)
        throw BadArgument(std::string(name) + " must be " + c10::toString(type) + ", got " +
                          c10::toString(t.scalar_type()));
    if (t.get_device() != device)
        throw BadArgument("tensors on different devices: " + std::string(name) + " on cuda:" +
                          std::to_string(t.get_device()) + ", not cuda:" + std::to_string(device));
    return t.data_ptr();
}

void shape(const at::Tensor& t, const char* name, c10::IntArrayRef want) {
    if (t.sizes() != want)
        throw BadArgument(std::string(name) + " must be " + text(want) + ", got " + text(t.sizes()));
}

// The same for an optional vector of n elements (None: null).
void* vector(PyObject* o, const char* name, at::ScalarType type, int64_t n, int device) {
    if (o == Py_None) return nullptr;
    const at::Tensor& t = tensor(o, name);
    shape(t, name, {n});
    return address(t, name, type, device);
}

long long integer(PyObject* o) {
    const long long v = PyLong_AsLongLong(o);
    if (v == -1 && PyErr_Occurred()) throw PythonError();
    return v;
}
int small(PyObject* o, const char* name) {
    const long long v = integer(o);
    if (v < -2147483647ll || v > 2147483647ll)
        throw BadArgument(std::string(name) + " is out of range");
    return (int)v;
}
double number(PyObject* o) {
    const double v = PyFloat_AsDouble(o);
    if (v == -1.0 && PyErr_Occurred()) throw PythonError();
    return v;
}
kv_pool_t handle(PyObject* o) { return reinterpret_cast<kv_pool_t>(PyLong_AsVoidPtr(o)); }

// A cudaStream_t given as an int, or None: the device's current stream.
void* stream_of(PyObject* o, int device) {
    if (o == Py_None) return c10::cuda::getCurrentCUDAStream((c10::DeviceIndex)device).stream();
    return reinterpret_cast<void*>((intptr_t)integer(o));
}

template <class F>
PyObject* guarded(F&& f) {
    try {
        return f();
    } catch (const PythonError&) {
    } catch (const BadArgument& e) {
        PyErr_SetString(PyExc_ValueError, e.what());
    } catch (const std::exception& e) {
        PyErr_SetString(PyExc_RuntimeError, e.what());
    }
    return nullptr;
}

void count(Py_ssize_t n, Py_ssize_t want) {
    if (n != want) {
        PyErr_Format(PyExc_TypeError, "%zd arguments, %zd expected", n, want);
        throw PythonError();
    }
}

// A tensor of n elements over `all`'s storage, from byte `from` on.
at::Tensor part(const at::Tensor& all, int64_t from, int64_t n, at::ScalarType type) {
    at::Tensor t = at::detail::make_tensor<c10::TensorImpl>(
        c10::Storage(all.storage()), all.key_set(), c10::scalarTypeToTypeMeta(type));
    t.unsafeGetTensorImpl()->set_storage_offset(from / (int64_t)c10::elementSize(type));
    t.unsafeGetTensorImpl()->set_sizes_contiguous({n});
    return t;
}

// plan_step(handle, context_lens, new_lens, block_tables, free_blocks, free_head,
//           num_tokens, stream) -> (cu_seqlens, seq_lens, slots, positions, head)
PyObject* plan_step(PyObject*, PyObject* const* a, Py_ssize_t n) {
    return guarded([&]() -> PyObject* {
        count(n, 8);
        const at::Tensor &ctx = tensor(a[1], "context_lens"), &fresh = tensor(a[2], "new_lens"),
                         &tables = tensor(a[3], "block_tables"), &blocks = tensor(a[4], "free_blocks"),
                         &head = tensor(a[5], "free_head");
        const int tokens = small(a[6], "num_tokens");
        const int device = ctx.is_cuda() ? (int)ctx.get_device() : -1;
        if (ctx.dim() != 1) throw BadArgument("context_lens must be one-dimensional");
        const int64_t b = ctx.size(0);
        shape(fresh, "new_lens", {b});
        shape(head, "free_head", {1});
        if (tables.dim() != 2 || tables.size(0) != b)
            throw BadArgument("block_tables must be [" + std::to_string(b) + ", max_blocks]");
        if (b > 2147483646 || tables.size(1) > 2147483647 || blocks.numel() > 2147483647 || tokens < 0)
            throw BadArgument("a size is out of range");
        const auto* pc = static_cast<int32_t*>(address(ctx, "context_lens", at::kInt, device));
        const auto* pn = static_cast<int32_t*>(address(fresh, "new_lens", at::kInt, device));
        auto* pt = static_cast<int32_t*>(address(tables, "block_tables", at::kInt, device));
        const auto* pf = static_cast<int32_t*>(address(blocks, "free_blocks", at::kInt, device));
        const auto* ph = static_cast<int32_t*>(address(head, "free_head", at::kInt, device));
        // The five results lie in one allocation, each on a 256-byte boundary: an
        // at::empty costs more than the rest of the call (8.5 -> 6.5 us a call).
        const auto room = [](int64_t bytes) { return (bytes + 255) / 256 * 256; };
        const int64_t at_lens = room(4 * (b + 1)), at_pos = at_lens + room(4 * b),
                      at_slots = at_pos + room(4 * (int64_t)tokens),
                      at_head = at_slots + room(8 * (int64_t)tokens);
        const at::Tensor all = at::empty({at_head + 4}, ctx.options().dtype(at::kByte));
        at::Tensor cu = part(all, 0, b + 1, at::kInt), lens = part(all, at_lens, b, at::kInt);
        at::Tensor pos = part(all, at_pos, tokens, at::kInt), slots = part(all, at_slots, tokens, at::kLong);
        at::Tensor out = part(all, at_head, 1, at::kInt);
        const kv_status st = kv_plan_step(
            handle(a[0]), pc, pn, (int)b, pt, (int)tables.size(1), pf, (int)blocks.numel(), ph,
            static_cast<int32_t*>(out.data_ptr()), static_cast<int32_t*>(cu.data_ptr()),
            static_cast<int32_t*>(lens.data_ptr()), static_cast<int64_t*>(slots.data_ptr()),
            static_cast<int32_t*>(pos.data_ptr()), tokens, stream_of(a[7], device));
        if (st != KV_OK) return PyLong_FromLong(st);
        PyObject* r = PyTuple_New(5);
        if (!r) throw PythonError();
        at::Tensor* t[5] = {&cu, &lens, &slots, &pos, &out};
        for (int i = 0; i < 5; ++i) {
            PyObject* o = THPVariable_Wrap(std::move(*t[i]));
            if (!o) {
                Py_DECREF(r);
                throw PythonError();
            }
            PyTuple_SET_ITEM(r, i, o);
        }
        return r;
    });
}

// append(handle, k_new, v_new, slot_mapping, row, stream) -> None; row: elements of
// a token's K or V; the caller has compared the rows' type with the pool's
PyObject* append(PyObject*, PyObject* const* a, Py_ssize_t n) {
    return guarded([&]() -> PyObject* {
        count(n, 6);
        const at::Tensor &k = tensor(a[1], "k_new"), &v = tensor(a[2], "v_new"),
                         &slots = tensor(a[3], "slot_mapping");
        const int device = k.is_cuda() ? (int)k.get_device() : -1;
        if (slots.dim() < 1 || slots.size(0) > 2147483647) throw BadArgument("slot_mapping must be [tokens]");
        const int64_t need = slots.size(0) * (int64_t)small(a[4], "row");
        if (k.numel() < need || v.numel() < need)
            throw BadArgument("k_new and v_new must hold a row for each of the " +
                              std::to_string(slots.size(0)) + " slots");
        const void* pk = address(k, "k_new", k.scalar_type(), device);
        const void* pv = address(v, "v_new", k.scalar_type(), device);
        const auto* ps = static_cast<int64_t*>(address(slots, "slot_mapping", at::kLong, device));
        const kv_status st = kv_append(handle(a[0]), pk, pv, ps, (int)slots.size(0), stream_of(a[5], device));
        if (st != KV_OK) return PyLong_FromLong(st);
        Py_RETURN_NONE;
    });
}

// out given, or a new tensor like q.
at::Tensor result(PyObject* o, const at::Tensor& q, const char* name) {
    if (o == Py_None) return at::empty_like(q);
    const at::Tensor& t = tensor(o, name);
    shape(t, name, q.sizes());
    return t;
}

// decode_scored(handle, q, block_tables, seq_lens, scale, num_kv_heads, softcap,
//               alibi_slopes, window, first_visible, out, workspace, stream) -> out
PyObject* decode_scored(PyObject*, PyObject* const* a, Py_ssize_t n) {
    return guarded([&]() -> PyObject* {
        count(n, 13);
        const at::Tensor &q = tensor(a[1], "q"), &tables = tensor(a[2], "block_tables"),
                         &lens = tensor(a[3], "seq_lens"), &ws = tensor(a[11], "workspace");
        const int device = q.is_cuda() ? (int)q.get_device() : -1;
        if (q.dim() != 3) throw BadArgument("q must be [batch, query heads, head_dim]");
        const int64_t b = q.size(0), hq = q.size(1);
        shape(lens, "seq_lens", {b});
        if (tables.dim() != 2 || tables.size(0) != b)
            throw BadArgument("block_tables must be [" + std::to_string(b) + ", max_blocks]");
        if (b > 2147483647 || hq > 2147483647 || tables.size(1) > 2147483647)
            throw BadArgument("a size is out of range");
        const void* pq = address(q, "q", q.scalar_type(), device);
        const auto* pt = static_cast<int32_t*>(address(tables, "block_tables", at::kInt, device));
        const auto* pl = static_cast<int32_t*>(address(lens, "seq_lens", at::kInt, device));
        void* pw = address(ws, "workspace", ws.scalar_type(), device);
        kv_score_mods mods = {};
        mods.softcap = (float)number(a[6]);
        mods.alibi_slopes = static_cast<float*>(vector(a[7], "alibi_slopes", at::kFloat, hq, device));
        mods.window = small(a[8], "window");
        mods.first_visible = static_cast<int32_t*>(vector(a[9], "first_visible", at::kInt, b, device));
        at::Tensor out = result(a[10], q, "out");
        void* po = address(out, "out", q.scalar_type(), device);
        const kv_status st = paged_attention_decode_scored(
            handle(a[0]), pq, po, pt, (int)tables.size(1), pl, (int)b, (int)hq, (float)number(a[4]),
            small(a[5], "num_kv_heads"), &mods, pw, ws.nbytes(), stream_of(a[12], device));
        if (st != KV_OK) return PyLong_FromLong(st);
        return THPVariable_Wrap(std::move(out));
    });
}

// prefill_scored(handle, q, cu_seqlens, max_query_len, block_tables, seq_lens, scale,
//                num_kv_heads, softcap, alibi_slopes, window, first_visible,
//                prefix_lens, out, stream) -> out
PyObject* prefill_scored(PyObject*, PyObject* const* a, Py_ssize_t n) {
    return guarded([&]() -> PyObject* {
        count(n, 15);
        const at::Tensor &q = tensor(a[1], "q"), &cu = tensor(a[2], "cu_seqlens"),
                         &tables = tensor(a[4], "block_tables"), &lens = tensor(a[5], "seq_lens");
        const int device = q.is_cuda() ? (int)q.get_device() : -1;
        if (q.dim() != 3) throw BadArgument("q must be [tokens, query heads, head_dim]");
        const int64_t t = q.size(0), hq = q.size(1), b = lens.numel();
        shape(cu, "cu_seqlens", {b + 1});
        if (tables.dim() != 2 || tables.size(0) != b)
            throw BadArgument("block_tables must be [" + std::to_string(b) + ", max_blocks]");
        if (t > 2147483647 || hq > 2147483647 || b > 2147483646 || tables.size(1) > 2147483647)
            throw BadArgument("a size is out of range");
        const void* pq = address(q, "q", q.scalar_type(), device);
        const auto* pc = static_cast<int32_t*>(address(cu, "cu_seqlens", at::kInt, device));
        const auto* pt = static_cast<int32_t*>(address(tables, "block_tables", at::kInt, device));
        const auto* pl = static_cast<int32_t*>(address(lens, "seq_lens", at::kInt, device));
        kv_score_mods mods = {};
        mods.softcap = (float)number(a[8]);
        mods.alibi_slopes = static_cast<float*>(vector(a[9], "alibi_slopes", at::kFloat, hq, device));
        mods.window = small(a[10], "window");
        mods.first_visible = static_cast<int32_t*>(vector(a[11], "first_visible", at::kInt, t, device));
        mods.prefix_lens = static_cast<int32_t*>(vector(a[12], "prefix_lens", at::kInt, b, device));
        at::Tensor out = result(a[13], q, "out");
        void* po = address(out, "out", q.scalar_type(), device);
        const kv_status st = paged_attention_prefill_scored(
            handle(a[0]), pq, po, pc, (int)t, small(a[3], "max_query_len"), pt, (int)tables.size(1), pl,
            (int)b, (int)hq, (float)number(a[6]), small(a[7], "num_kv_heads"), &mods,
            stream_of(a[14], device));
        if (st != KV_OK) return PyLong_FromLong(st);
        return THPVariable_Wrap(std::move(out));
    });
}

PyMethodDef methods[] = {
    {"plan_step", (PyCFunction)(void (*)(void))plan_step, METH_FASTCALL, nullptr},
    {"append", (PyCFunction)(void (*)(void))append, METH_FASTCALL, nullptr},
    {"decode_scored", (PyCFunction)(void (*)(void))decode_scored, METH_FASTCALL, nullptr},
    {"prefill_scored", (PyCFunction)(void (*)(void))prefill_scored, METH_FASTCALL, nullptr},
    {nullptr, nullptr, 0, nullptr}};

PyModuleDef module = {PyModuleDef_HEAD_INIT, "_pagedkv_binding", nullptr, -1, methods,
                      nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__pagedkv_binding() { return PyModule_Create(&module); }
