// pn_step_binding.cpp -- Python entry of the serving-step calls (include/pn.h,
// "4-bit cache"): checks, output allocation and the C call.
//
// A step makes these calls for every token, so what they cost on the host
// counts: through ctypes and Python checks a plan with its eight outputs took
// 42 us and a verification 17 us of host time on an Arm host, where the
// C calls themselves take 4 us (launch included).  pn.py keeps the signatures,
// defaults and documentation; each function here takes their arguments by
// position and returns (status, outputs...), status as in pn.h.
#include <Python.h>

#include <ATen/core/Tensor.h>
#include <ATen/EmptyTensor.h>
#include <c10/cuda/CUDACachingAllocator.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <c10/util/Exception.h>
#include <torch/csrc/autograd/python_variable.h>

#include <exception>

#include "../../include/pn.h"

namespace {

// A Python error has been set.
struct PythonError {};

[[noreturn]] void fail(PyObject* type, const char* format, const char* name, const char* what = "") {
    PyErr_Format(type, format, name, what);
    throw PythonError{};
}

const char* type_name(at::ScalarType t) {
    switch (t) {
        case at::kInt: return "torch.int32";
        case at::kLong: return "torch.int64";
        case at::kFloat: return "torch.float32";
        case at::kHalf: return "torch.float16";
        case at::kByte: return "torch.uint8";
        default: return "of another type";
    }
}

// The device of a call's tensors: the first one's, and the others have to be there too.
struct Device {
    int index = -1;
    const char* of = "";
    void take(const at::Tensor& t, const char* name) {
        if (index < 0) {
            index = t.get_device();
            of = name;
        } else if (t.get_device() != index) {
            fail(PyExc_ValueError, "%s must be on the device of %s", name, of);
        }
    }
};

const at::Tensor& cuda_tensor(Device& on, PyObject* o, const char* name) {
    if (!THPVariable_Check(o)) fail(PyExc_TypeError, "%s must be a CUDA tensor", name);
    const at::Tensor& t = THPVariable_Unpack(o);
    if (!t.is_cuda()) fail(PyExc_TypeError, "%s must be a CUDA tensor", name);
    on.take(t, name);
    return t;
}

const at::Tensor& dense(Device& on, PyObject* o, at::ScalarType type, const char* name) {
    const at::Tensor& t = cuda_tensor(on, o, name);
    if (t.scalar_type() != type) fail(PyExc_TypeError, "%s must be %s", name, type_name(type));
    if (!t.is_contiguous()) fail(PyExc_ValueError, "%s must be contiguous", name);
    return t;
}

// None, or a dense tensor of n entries.
const at::Tensor* optional(Device& on, PyObject* o, at::ScalarType type, int64_t n, const char* name, const char* shape) {
    if (o == Py_None) return nullptr;
    const at::Tensor& t = dense(on, o, type, name);
    if (t.numel() != n) fail(PyExc_ValueError, "%s must be %s", name, shape);
    return &t;
}

template <typename T>
T* data(const at::Tensor* t) {
    return t ? static_cast<T*>(t->data_ptr()) : nullptr;
}

int64_t whole(PyObject* o) {
    const long long v = PyLong_AsLongLong(o);
    if (v == -1 && PyErr_Occurred()) throw PythonError{};
    return v;
}
int number(PyObject* o, const char* name) {
    const int64_t v = whole(o);
    if (v < INT32_MIN || v > INT32_MAX) fail(PyExc_ValueError, "%s is out of range", name);
    return static_cast<int>(v);
}
float real(PyObject* o) {
    const double v = PyFloat_AsDouble(o);
    if (v == -1.0 && PyErr_Occurred()) throw PythonError{};
    return static_cast<float>(v);
}

// int32 rows of a page table.
const at::Tensor& page_table(Device& on, PyObject* o, int64_t batch) {
    const at::Tensor& t = cuda_tensor(on, o, "table");
    if (t.scalar_type() != at::kInt) fail(PyExc_TypeError, "%s must be a CUDA int32 tensor", "table");
    if (t.dim() != 2 || t.size(0) != batch || (t.size(1) > 1 && t.stride(1) != 1))
        fail(PyExc_ValueError, "%s must be [batch][pages per request] with contiguous rows", "table");
    if (t.size(1) > INT32_MAX) fail(PyExc_ValueError, "%s has too many columns", "table");
    return t;
}
int64_t table_stride(const at::Tensor& t) { return t.size(0) > 1 ? t.stride(0) : t.size(1); }

// [tokens][heads][dim] whose heads are contiguous within a token.
const at::Tensor& rows(Device& on, PyObject* o, const char* name, at::ScalarType a, at::ScalarType b, int64_t heads, int64_t dim) {
    const at::Tensor& t = cuda_tensor(on, o, name);
    if (t.scalar_type() != a && t.scalar_type() != b)
        fail(PyExc_TypeError, a == b ? "%s must be %s" : "%s must be torch.float32 or torch.float16", name, type_name(a));
    if (t.dim() != 3 || t.size(2) != dim || (heads >= 0 && t.size(1) != heads))
        fail(PyExc_ValueError, "%s must be [tokens][heads][head_dim]", name);
    if (t.numel() > 0 && (t.stride(2) != 1 || (t.size(1) > 1 && t.stride(1) != dim)))
        fail(PyExc_ValueError, "%s's heads must be contiguous within a token", name);
    return t;
}
// Elements between tokens (a lone token's stride may say anything).
int64_t row_stride(const at::Tensor& t) { return t.size(0) > 1 ? t.stride(0) : t.size(1) * t.size(2); }

struct Cache {
    const at::Tensor& t;
    int64_t pages;
    int page_size, heads, dim;
    Cache(Device& on, PyObject* o) : t(dense(on, o, at::kByte, "cache")) {
        if (t.dim() != 4 || t.size(3) % 17 || t.size(1) > 65536 || t.size(2) > 65536 || t.size(3) > 65536)
            fail(PyExc_ValueError, "%s must be uint8 [pages][kv_heads][page_size / 16][17 * head_dim]", "cache");
        pages = t.size(0);
        page_size = static_cast<int>(t.size(2)) * 16;
        heads = static_cast<int>(t.size(1));
        dim = static_cast<int>(t.size(3) / 17);
    }
};

// A new tensor on the current device (the guard's), as at::empty makes it for a CUDA
// device, without the dispatcher on the way.
at::Tensor fresh(at::IntArrayRef size, at::ScalarType type) {
    return at::detail::empty_generic(size, c10::cuda::CUDACachingAllocator::get(), c10::DispatchKeySet(c10::DispatchKey::CUDA), type, std::nullopt);
}

// `n` entries from byte `at` on of a tensor of ours: another tensor on the same
// memory (an allocation takes more than a microsecond).
at::Tensor part_of(const at::Tensor& t, int64_t at, int64_t n, at::ScalarType type) {
    const caffe2::TypeMeta meta = c10::scalarTypeToTypeMeta(type);
    auto impl = c10::make_intrusive<c10::TensorImpl>(c10::Storage(t.storage()), t.key_set(), meta);
    impl->set_storage_offset(at / static_cast<int64_t>(meta.itemsize()));
    impl->set_sizes_contiguous({n});
    return at::Tensor(std::move(impl));
}

pn_stream stream_of(const at::Tensor& t) {
    return reinterpret_cast<pn_stream>(c10::cuda::getCurrentCUDAStream(t.get_device()).stream());
}

// (status, outputs...): `out` are new references, null for None.
PyObject* answer(pn_status status, std::initializer_list<PyObject*> out) {
    PyObject* r = PyTuple_New(1 + static_cast<Py_ssize_t>(out.size()));
    Py_ssize_t i = 0;
    if (r) PyTuple_SET_ITEM(r, i++, PyLong_FromLong(status));
    for (PyObject* o : out) {
        if (!o) { Py_INCREF(Py_None); o = Py_None; }
        if (r) PyTuple_SET_ITEM(r, i++, o);
        else Py_DECREF(o);
    }
    return r;
}
PyObject* given_or(PyObject* given, const at::Tensor& made) {
    if (given != Py_None) { Py_INCREF(given); return given; }
    return THPVariable_Wrap(made);
}

// lens, add, held, table, free, ring, page_size, capacity, out (None or the eight tensors)
PyObject* kv_plan(PyObject* const* a) {
    Device on;
    const at::Tensor& lens = dense(on, a[0], at::kInt, "lens");
    const at::Tensor& add = dense(on, a[1], at::kInt, "add");
    const at::Tensor& held = dense(on, a[2], at::kInt, "held");
    const at::Tensor& free = dense(on, a[4], at::kInt, "free");
    const at::Tensor& ring = dense(on, a[5], at::kLong, "ring");
    const int64_t B = lens.numel();
    const at::Tensor& table = page_table(on, a[3], B);
    if (add.numel() != B || held.numel() != B || ring.numel() != 2)
        fail(PyExc_ValueError, "%s, add and held must have one entry per request and ring two", "lens");
    const int page_size = number(a[6], "page_size");
    const int64_t T = whole(a[7]);
    if (T < 0) fail(PyExc_ValueError, "%s must not be negative", "capacity");
    if (B > INT32_MAX) fail(PyExc_ValueError, "%s has too many entries", "lens");
    static const char* const names[8] = {"out.slots", "out.positions", "out.requests", "out.starts", "out.lens", "out.held", "out.ring", "out.refused"};
    const int64_t sizes[8] = {T, T, T, B + 1, B, B, 2, 1};
    at::Tensor o[8];
    PyObject* given[8];
    const bool have = a[8] != Py_None;
    if (have && (!PyTuple_Check(a[8]) || PyTuple_GET_SIZE(a[8]) != 8)) fail(PyExc_TypeError, "%s must be a KvPlan", "out");
    auto type_of = [](int i) { return i == 0 || i == 6 ? at::kLong : at::kInt; };
    for (int i = 0; i < 8; ++i) {
        given[i] = have ? PyTuple_GET_ITEM(a[8], i) : Py_None;
        if (!have) continue;
        o[i] = dense(on, given[i], type_of(i), names[i]);
        if (o[i].numel() != sizes[i]) fail(PyExc_ValueError, "%s has another size", names[i]);
    }
    const c10::cuda::CUDAGuard guard(lens.device());
    if (!have) {
        int64_t wide_at = 0, narrow_at = (T + 2) * 8;      // 64-bit outputs first
        const at::Tensor all = fresh({narrow_at + (2 * T + 3 * B + 2) * 4}, at::kByte);
        for (int i = 0; i < 8; ++i) {
            int64_t& from = type_of(i) == at::kLong ? wide_at : narrow_at;
            o[i] = part_of(all, from, sizes[i], type_of(i));
            from += sizes[i] * (type_of(i) == at::kLong ? 8 : 4);
        }
    }
    const pn_status st = pn_kv_plan(data<int32_t>(&lens), data<int32_t>(&add), data<int32_t>(&held), static_cast<int>(B), data<int32_t>(&table),
                                    table_stride(table), static_cast<int>(table.size(1)), data<int32_t>(&free), free.numel(),
                                    data<int64_t>(&ring), page_size, T, data<int64_t>(&o[0]), data<int32_t>(&o[1]), data<int32_t>(&o[2]),
                                    data<int32_t>(&o[3]), data<int32_t>(&o[4]), data<int32_t>(&o[5]), data<int64_t>(&o[6]), data<int32_t>(&o[7]),
                                    stream_of(lens));
    return answer(st, {given_or(given[0], o[0]), given_or(given[1], o[1]), given_or(given[2], o[2]), given_or(given[3], o[3]),
                       given_or(given[4], o[4]), given_or(given[5], o[5]), given_or(given[6], o[6]), given_or(given[7], o[7])});
}

// q, k, v, cache, slots, positions, cos, sin, q_weight, k_weight, eps, interleaved, q_out
PyObject* kv_append(PyObject* const* a) {
    Device on;
    const Cache c(on, a[3]);
    const at::Tensor& k = rows(on, a[1], "k", at::kFloat, at::kHalf, c.heads, c.dim);
    const at::ScalarType type = k.scalar_type();
    const at::Tensor& v = rows(on, a[2], "v", type, type, c.heads, c.dim);
    const at::Tensor* q = a[0] == Py_None ? nullptr : &rows(on, a[0], "q", type, type, -1, c.dim);
    const int64_t T = k.size(0), heads = q ? q->size(1) : 0;
    if (v.size(0) != T || (q && q->size(0) != T)) fail(PyExc_ValueError, "%s, k and v must have the same tokens", "q");
    if (heads > INT32_MAX) fail(PyExc_ValueError, "%s has too many heads", "q");
    const at::Tensor* slots = optional(on, a[4], at::kLong, T, "slots", "one entry per token");
    if (!slots) fail(PyExc_TypeError, "%s must be a CUDA tensor", "slots");
    const at::Tensor *cos = nullptr, *sin = nullptr, *positions = nullptr;
    int64_t pairs = 0, table_rows = 0;
    if (a[6] != Py_None || a[7] != Py_None) {
        cos = &dense(on, a[6], at::kFloat, "cos");
        sin = &dense(on, a[7], at::kFloat, "sin");
        if (cos->dim() != 2 || cos->sizes() != sin->sizes()) fail(PyExc_ValueError, "%s and sin must be [positions][rotated pairs]", "cos");
        table_rows = cos->size(0);
        pairs = cos->size(1);
        positions = optional(on, a[5], at::kInt, T, "positions", "one entry per token");
        if (!positions) fail(PyExc_TypeError, "%s must be a CUDA tensor", "positions");
        if (pairs > 65536) fail(PyExc_ValueError, "%s has too many columns", "cos");
    }
    const at::Tensor* qw = optional(on, a[8], at::kFloat, c.dim, "q_weight", "[head_dim]");
    const at::Tensor* kw = optional(on, a[9], at::kFloat, c.dim, "k_weight", "[head_dim]");
    const float eps = real(a[10]);
    const int interleaved = PyObject_IsTrue(a[11]);
    if (interleaved < 0) throw PythonError{};
    const at::Tensor* given = q ? optional(on, a[12], at::kHalf, T * heads * c.dim, "q_out", "[tokens][heads][head_dim]") : nullptr;
    const c10::cuda::CUDAGuard guard(k.device());
    at::Tensor out;
    if (q) out = given ? *given : fresh({T, heads, c.dim}, at::kHalf);
    const pn_status st = pn_kv_append(data<void>(q), q ? row_stride(*q) : 0, data<void>(&k), row_stride(k), data<void>(&v), row_stride(v),
                                      type == at::kFloat ? PN_DTYPE_F32 : PN_DTYPE_F16, T, static_cast<int>(heads), data<float>(qw),
                                      data<float>(kw), eps, data<float>(cos), data<float>(sin), table_rows, static_cast<int>(2 * pairs),
                                      interleaved, data<int32_t>(positions), data<int64_t>(slots), c.t.data_ptr(), c.pages, c.page_size,
                                      c.heads, c.dim, q ? data<uint16_t>(&out) : nullptr, stream_of(k));
    return answer(st, {q ? given_or(a[12], out) : nullptr});
}

// cache, slots, k, v (None, None: new ones)
PyObject* kv_read(PyObject* const* a) {
    Device on;
    const Cache c(on, a[0]);
    const at::Tensor& slots = dense(on, a[1], at::kLong, "slots");
    const int64_t T = slots.numel(), n = T * c.heads * c.dim;
    const at::Tensor* gk = optional(on, a[2], at::kFloat, n, "out", "two tensors [tokens][kv_heads][head_dim]");
    const at::Tensor* gv = optional(on, a[3], at::kFloat, n, "out", "two tensors [tokens][kv_heads][head_dim]");
    const c10::cuda::CUDAGuard guard(slots.device());
    const at::Tensor k = gk ? *gk : fresh({T, c.heads, c.dim}, at::kFloat);
    const at::Tensor v = gv ? *gv : fresh({T, c.heads, c.dim}, at::kFloat);
    const pn_status st = pn_kv_read(c.t.data_ptr(), c.pages, c.page_size, c.heads, c.dim, data<int64_t>(&slots), T, data<float>(&k),
                                    data<float>(&v), stream_of(slots));
    return answer(st, {given_or(a[2], k), given_or(a[3], v)});
}

// q, cache, table, lens, starts, max_queries, scale, window, sinks, out, lse, return_lse, workspace
PyObject* attention(PyObject* const* a) {
    Device on;
    const Cache c(on, a[1]);
    const at::Tensor& q = rows(on, a[0], "q", at::kHalf, at::kHalf, -1, c.dim);
    const int64_t T = q.size(0), heads = q.size(1);
    const at::Tensor& lens = dense(on, a[3], at::kInt, "lens");
    const at::Tensor& starts = dense(on, a[4], at::kInt, "starts");
    const int64_t B = lens.numel();
    const at::Tensor& table = page_table(on, a[2], B);
    if (starts.numel() != B + 1) fail(PyExc_ValueError, "%s must have one entry more than lens", "starts");
    if (B > INT32_MAX || heads > INT32_MAX) fail(PyExc_ValueError, "%s has too many entries", "lens or q");
    const int max_queries = number(a[5], "max_queries"), window = number(a[7], "window"), sinks = number(a[8], "sinks");
    const float scale = real(a[6]);
    const at::Tensor* given = optional(on, a[9], at::kHalf, T * heads * c.dim, "out", "[tokens][heads][head_dim]");
    const at::Tensor* lse = optional(on, a[10], at::kFloat, T * heads, "lse", "[tokens][heads]");
    const int want_lse = PyObject_IsTrue(a[11]);
    if (want_lse < 0) throw PythonError{};
    const at::Tensor& workspace = dense(on, a[12], at::kByte, "workspace");
    const c10::cuda::CUDAGuard guard(q.device());
    const at::Tensor out = given ? *given : fresh({T, heads, c.dim}, at::kHalf);
    at::Tensor made;
    if (!lse && want_lse) {
        made = fresh({T, heads}, at::kFloat);
        lse = &made;
    }
    const pn_status st = pn_attention(data<uint16_t>(&q), row_stride(q), T, static_cast<int>(heads), c.t.data_ptr(), c.pages, c.page_size,
                                      c.heads, c.dim, data<int32_t>(&table), table_stride(table), static_cast<int>(table.size(1)),
                                      data<int32_t>(&lens), data<int32_t>(&starts), static_cast<int>(B), max_queries, scale, window, sinks,
                                      data<uint16_t>(&out), data<float>(lse), workspace.data_ptr(), static_cast<size_t>(workspace.numel()), stream_of(q));
    return answer(st, {given_or(a[9], out), lse ? given_or(a[10], *lse) : nullptr});
}

// tokens, target, draft, uniforms, counts, accepted, out
PyObject* verify(PyObject* const* a) {
    Device on;
    const at::Tensor& tokens = dense(on, a[0], at::kInt, "tokens");
    const at::Tensor& target = dense(on, a[1], at::kFloat, "target");
    const at::Tensor& uniforms = dense(on, a[3], at::kFloat, "uniforms");
    if (tokens.dim() != 2 || target.dim() != 3)
        fail(PyExc_ValueError, "%s must be [batch][drafts] and target [batch][drafts + 1][vocab]", "tokens");
    const int64_t B = tokens.size(0), K = tokens.size(1), V = target.size(2);
    if (target.size(0) != B || target.size(1) != K + 1 || uniforms.numel() != B * (K + 1))
        fail(PyExc_ValueError, "%s and uniforms must have one row more than there are drafts", "target");
    const at::Tensor* draft = nullptr;
    if (a[2] != Py_None) {
        draft = &dense(on, a[2], at::kFloat, "draft");
        if (draft->dim() != 3 || draft->size(0) != B || draft->size(1) != K || draft->size(2) != V)
            fail(PyExc_ValueError, "%s must be [batch][drafts][vocab]", "draft");
    }
    if (B > INT32_MAX || K > INT32_MAX || V > INT32_MAX) fail(PyExc_ValueError, "%s is too large", "target");
    const at::Tensor* counts = optional(on, a[4], at::kInt, B, "counts", "one entry per request");
    const at::Tensor* given_accepted = optional(on, a[5], at::kInt, B, "accepted", "[batch]");
    const at::Tensor* given_out = optional(on, a[6], at::kInt, B * (K + 1), "out", "[batch][drafts + 1]");
    const c10::cuda::CUDAGuard guard(target.device());
    const at::Tensor accepted = given_accepted ? *given_accepted : fresh({B}, at::kInt);
    const at::Tensor out = given_out ? *given_out : fresh({B, K + 1}, at::kInt);
    const pn_status st = pn_verify(data<int32_t>(&tokens), data<float>(&target), V, data<float>(draft), V, data<float>(&uniforms),
                                   data<int32_t>(counts), static_cast<int>(B), static_cast<int>(K), static_cast<int>(V),
                                   data<int32_t>(&accepted), data<int32_t>(&out), stream_of(target));
    return answer(st, {given_or(a[5], accepted), given_or(a[6], out)});
}

// A shortage of device memory, as PyTorch's own calls raise it.
void raise_out_of_memory(const char* what) {
    PyObject* torch = PyImport_ImportModule("torch");
    PyObject* type = torch ? PyObject_GetAttrString(torch, "OutOfMemoryError") : nullptr;
    Py_XDECREF(torch);
    if (!type) return;                         // (that error stands)
    PyErr_SetString(type, what);
    Py_DECREF(type);
}

// No C++ exception leaves an entry.
template <PyObject* (*F)(PyObject* const*), Py_ssize_t N>
PyObject* entry(PyObject*, PyObject* const* args, Py_ssize_t n) {
    if (n != N) {
        PyErr_Format(PyExc_TypeError, "%zd arguments expected, %zd given", N, n);
        return nullptr;
    }
    try {
        return F(args);
    } catch (const PythonError&) {
    } catch (const c10::OutOfMemoryError& e) {
        if (!PyErr_Occurred()) raise_out_of_memory(e.what_without_backtrace());
    } catch (const std::exception& e) {
        if (!PyErr_Occurred()) PyErr_SetString(PyExc_RuntimeError, e.what());
    } catch (...) {
        if (!PyErr_Occurred()) PyErr_SetString(PyExc_RuntimeError, "unknown error");
    }
    return nullptr;
}

template <PyObject* (*F)(PyObject* const*), Py_ssize_t N>
PyMethodDef method(const char* name) {
    return {name, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(entry<F, N>)), METH_FASTCALL, nullptr};
}

PyMethodDef g_methods[] = {method<kv_plan, 9>("kv_plan"), method<kv_append, 13>("kv_append"), method<kv_read, 4>("kv_read"),
                           method<attention, 13>("attention"), method<verify, 7>("verify"), {nullptr, nullptr, 0, nullptr}};
PyModuleDef g_module = {PyModuleDef_HEAD_INIT, "_step", nullptr, -1, g_methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__step() { return PyModule_Create(&g_module); }
