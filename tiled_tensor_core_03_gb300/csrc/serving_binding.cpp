// serving_binding.cpp -- CPython extension between serving.py and the C ABI of libgemmrelu.so:
// checks torch tensors and passes their pointers, sizes and strides on.  It computes nothing.
//
// A decode step's kernels take 4 to 10 us; the same checks in Python took 11 to 20 us a call.
// The library's functions are handed over as addresses by bind(), so this file links against
// torch alone.  No C++ exception leaves an entry point: each becomes a Python error.
#define PY_SSIZE_T_CLEAN
#include <Python.h>

#include <ATen/ATen.h>
#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/autograd/python_variable.h>

#include <algorithm>
#include <cstdint>
#include <map>
#include <mutex>
#include <sstream>
#include <string>
#include <utility>

#include "flash_attention.h"
#include "gemm_relu.h"
#include "kv_cache.h"

namespace {

decltype(&flash_attention_window_x16) f_window;
decltype(&kv_cache_append_x16) f_append;
decltype(&kv_cache_attention_x16) f_attention;
decltype(&kv_cache_attention_x16_workspace_bytes) f_workspace_bytes;
decltype(&kv_cache_evict_e4m3) f_evict;
decltype(&gemm_relu_stream_capturing) f_capturing;
decltype(&gemm_relu_stream_id) f_stream_id;
PyObject *g_error, *g_no_memory;   // GemmReluError, torch.OutOfMemoryError

struct Refusal {
    PyObject *type;
    std::string what;
};

template <typename... Parts>
[[noreturn]] void refuse(PyObject *type, const Parts &...parts) {
    std::ostringstream s;
    (s << ... << parts);
    throw Refusal{type, s.str()};
}

// A Python error is already set.
struct Raised {};

const at::Tensor &tensor(PyObject *o, const char *name) {
    if (!THPVariable_Check(o))
        refuse(PyExc_TypeError, name, " must be a torch.Tensor, not ", Py_TYPE(o)->tp_name);
    return THPVariable_Unpack(o);
}

int64_t integer(PyObject *o, const char *name) {
    const long long v = PyLong_AsLongLong(o);
    if (v == -1 && PyErr_Occurred()) {
        PyErr_Clear();
        refuse(PyExc_TypeError, name, " must be an integer of 64 bits");
    }
    return v;
}

// The current device, which every tensor of a call must be on.
int current_device_of(const at::Tensor &t) {
    if (!t.is_cuda() || t.get_device() != c10::cuda::current_device())
        refuse(PyExc_ValueError, "tensors must be on the current CUDA device");
    return (int)t.get_device();
}

bool on(const at::Tensor &t, int d) { return t.is_cuda() && t.get_device() == d; }

void *stream_of(int d) { return (void *)c10::cuda::getCurrentCUDAStream((c10::DeviceIndex)d).stream(); }

int dtype_of(const at::Tensor &t) {
    return t.scalar_type() == at::kHalf ? GEMMRELU_F16 : t.scalar_type() == at::kBFloat16 ? GEMMRELU_BF16 : -1;
}

// The pool of a cache (k, v, k_scale, v_scale).
kv_cache_pool pool_of(PyObject *cache, int d) {
    PyObject *items[4];
    if (!PyTuple_Check(cache) || PyTuple_GET_SIZE(cache) != 4)
        refuse(PyExc_TypeError, "a cache is a tuple (k, v, k_scale, v_scale)");
    for (int i = 0; i < 4; ++i)
        items[i] = PyTuple_GET_ITEM(cache, i);
    const at::Tensor &k = tensor(items[0], "cache k"), &v = tensor(items[1], "cache v");
    const at::Tensor &ks = tensor(items[2], "cache k_scale"), &vs = tensor(items[3], "cache v_scale");
    const auto type = k.scalar_type();
    if (k.dim() != 4 || v.sizes() != k.sizes() || (type != at::kFloat8_e4m3fn && type != at::kByte) ||
        v.scalar_type() != type || !k.is_contiguous() || !v.is_contiguous())
        refuse(PyExc_ValueError, "cache k and v must be contiguous e4m3 tensors of one shape "
                                 "[num_pages, kv_heads, page, head_dim]");
    const int64_t page = k.size(2), dim = k.size(3);
    if ((dim != 64 && dim != 128) || (page != 16 && page != 32 && page != 64 && page != 128))
        refuse(PyExc_ValueError, "head_dim must be 64 or 128, page 16, 32, 64 or 128: got ", k.sizes());
    for (const at::Tensor *s : {&ks, &vs})
        if (s->dim() != 2 || s->size(0) != k.size(0) || s->size(1) != k.size(1) ||
            s->scalar_type() != at::kFloat || !s->is_contiguous())
            refuse(PyExc_ValueError, "cache scales must be contiguous float32 [num_pages, kv_heads]");
    if (!on(k, d) || !on(v, d) || !on(ks, d) || !on(vs, d))
        refuse(PyExc_ValueError, "the cache must be on cuda:", d);
    return kv_cache_pool{k.data_ptr(), v.data_ptr(), ks.data_ptr<float>(), vs.data_ptr<float>(),
                         k.size(0), k.size(1), page, dim};
}

// An int32 tensor [batch], or [batch, any] where `width` is asked for.
const int32_t *ints(const at::Tensor &t, const char *name, int64_t batch, int d, int64_t *width = nullptr) {
    if (t.scalar_type() != at::kInt || t.dim() != (width ? 2 : 1) || t.size(0) != batch ||
        !t.is_contiguous() || !on(t, d))
        refuse(PyExc_ValueError, name, " must be a contiguous int32 tensor [", batch,
               width ? ", max_pages" : "", "] on cuda:", d);
    if (width)
        *width = t.size(1);
    return t.data_ptr<int32_t>();
}

// {sequence, token, head} strides of a 16-bit tensor whose heads are contiguous and start on
// 16-byte boundaries; an axis of one element is never stepped over.
struct Strides {
    int64_t s[3];
};

Strides strides_of(const at::Tensor &t, const char *name) {
    Strides r;
    bool ok = t.stride(3) == 1 && reinterpret_cast<uintptr_t>(t.data_ptr()) % 16 == 0;
    for (int i = 0; i < 3; ++i) {
        r.s[i] = t.size(i) == 1 ? 0 : t.stride(i);
        ok = ok && r.s[i] % 8 == 0;
    }
    if (!ok)
        refuse(PyExc_ValueError, name, ": heads must be contiguous and start on 16-byte boundaries (strides ",
               t.strides(), ")");
    return r;
}

void done(int rc, const char *what) {
    if (rc == GEMMRELU_OK)
        return;
    PyObject *e = PyObject_CallFunction(g_error, "is", rc, what);
    if (e) {
        PyErr_SetObject(g_error, e);
        Py_DECREF(e);
    }
    throw Raised{};
}

// A contiguous tensor like `q`: `out` itself where one is given.
at::Tensor output(const at::Tensor &q, PyObject *out, int d) {
    if (out == Py_None)
        return at::empty(q.sizes(), q.options());
    const at::Tensor &o = tensor(out, "out");
    if (o.sizes() != q.sizes() || o.scalar_type() != q.scalar_type() || !on(o, d) || !o.is_contiguous())
        refuse(PyExc_ValueError, "out must be a contiguous tensor like q");
    return o;
}

// What an entry point returns: `out` itself where the caller gave one.
PyObject *returned(const at::Tensor &t, PyObject *out) {
    if (out != Py_None) {
        Py_INCREF(out);
        return out;
    }
    return THPVariable_Wrap(t);
}

// ---------------------------------------------------------------- entry points
// `a` holds the positional arguments that serving.py passes, whose number it fixes.

PyObject *window_impl(PyObject *const *a) {
    const at::Tensor &q = tensor(a[0], "q"), &k = tensor(a[1], "k"), &v = tensor(a[2], "v");
    const int64_t window = integer(a[3], "window"), sinks = integer(a[4], "sinks");
    const int d = current_device_of(q), type = dtype_of(q);
    if (type < 0 || k.scalar_type() != q.scalar_type() || v.scalar_type() != q.scalar_type())
        refuse(PyExc_TypeError, "q, k and v must all be float16 or all bfloat16");
    if (q.dim() != 4 || k.dim() != 4 || v.sizes() != k.sizes() || !on(k, d) || !on(v, d))
        refuse(PyExc_ValueError, "q must be [batch, q_seq, q_heads, d], k and v [batch, kv_seq, kv_heads, d], "
                                 "all on one device");
    const int64_t dim = q.size(3);
    if (k.size(0) != q.size(0) || k.size(3) != dim || (dim != 64 && dim != 128) || k.size(2) == 0 ||
        q.size(2) % k.size(2) != 0)
        refuse(PyExc_ValueError, "shapes ", q.sizes(), " and ", k.sizes(), " do not go together");
    if (window < 0 || sinks < 0)
        refuse(PyExc_ValueError, "window and sinks must not be negative");
    const at::Tensor o = output(q, a[5], d);
    if (q.numel() > 0) {
        const Strides qs = strides_of(q, "q"), ks = strides_of(k, "k"), vs = strides_of(v, "v");
        done(f_window(q.data_ptr(), k.data_ptr(), v.data_ptr(), o.data_ptr(), type, q.size(0), q.size(1),
                      k.size(1), q.size(2), k.size(2), dim, qs.s, ks.s, vs.s, window, sinks, stream_of(d)),
             "flash_attention_window_x16");
    }
    return returned(o, a[5]);
}

PyObject *append_impl(PyObject *const *a) {
    const at::Tensor &k = tensor(a[1], "k"), &v = tensor(a[2], "v");
    const int d = current_device_of(k), type = dtype_of(k);
    if (type < 0 || v.scalar_type() != k.scalar_type())
        refuse(PyExc_TypeError, "k and v must both be float16 or both bfloat16");
    if (k.dim() != 4 || v.sizes() != k.sizes() || !on(v, d))
        refuse(PyExc_ValueError, "k and v must have the same shape [batch, tokens, kv_heads, head_dim]");
    const kv_cache_pool pool = pool_of(a[0], d);
    if (k.size(2) != pool.kv_heads || k.size(3) != pool.head_dim)
        refuse(PyExc_ValueError, "k has ", k.size(2), " heads of ", k.size(3), ", the cache ", pool.kv_heads,
               " of ", pool.head_dim);
    const int64_t batch = k.size(0);
    int64_t max_pages = 0;
    const int32_t *pages = ints(tensor(a[3], "pages"), "pages", batch, d, &max_pages);
    const int32_t *lengths = ints(tensor(a[4], "lengths"), "lengths", batch, d);
    const int32_t *counts = a[5] == Py_None ? nullptr : ints(tensor(a[5], "counts"), "counts", batch, d);
    if (batch > 0 && k.size(1) > 0) {
        const Strides ks = strides_of(k, "k"), vs = strides_of(v, "v");
        done(f_append(&pool, k.data_ptr(), v.data_ptr(), type, batch, k.size(1), ks.s, vs.s, pages, max_pages,
                      lengths, counts, stream_of(d)),
             "kv_cache_append_x16");
    }
    Py_RETURN_NONE;
}

size_t workspace_bytes(const at::Tensor &q, int64_t kv_heads, int64_t width) {
    return std::max<size_t>(f_workspace_bytes(q.size(0), q.size(1), q.size(2), kv_heads, q.size(3), width),
                            GEMMRELU_KV_COUNTER_BYTES);
}

at::Tensor new_workspace(const at::Tensor &q, size_t bytes) {
    at::Tensor w = at::empty({(int64_t)bytes}, q.options().dtype(at::kByte));
    w.narrow(0, 0, GEMMRELU_KV_COUNTER_BYTES).zero_();
    return w;
}

// Workspaces of calls that bring none, one per device and stream, as large as its calls needed so
// far: calls on a stream follow one another, and one that is replaced goes back to torch's
// allocator for that stream.  A stream is known by its id, since two may share a handle.  Calls being
// captured get their own, since their graph may run anywhere, and so do those that need more
// than kKeep (scores of many weights), which torch then has back at once.  So that streams that
// are gone do not hold memory for ever, all go back once there are kMostKept.  The map is
// never destroyed: at exit torch's allocator may be gone before it.
constexpr size_t kKeep = (size_t)64 << 20;
constexpr size_t kMostKept = 64;

at::Tensor workspace_for(const at::Tensor &q, int64_t kv_heads, int64_t width, int d, void *stream) {
    const size_t bytes = workspace_bytes(q, kv_heads, width);
    uint64_t id;
    if (bytes > kKeep || f_capturing(stream) || f_stream_id(stream, &id) != GEMMRELU_OK)
        return new_workspace(q, bytes);
    static auto *kept = new std::map<std::pair<int, uint64_t>, at::Tensor>;   // (the GIL is held)
    if (kept->size() >= kMostKept && kept->count({d, id}) == 0)
        kept->clear();
    at::Tensor &w = (*kept)[{d, id}];
    if (!w.defined() || w.nbytes() < bytes)
        w = new_workspace(q, bytes);
    return w;
}

PyObject *attention_impl(PyObject *const *a) {
    const at::Tensor &q = tensor(a[1], "q");
    const int64_t window = integer(a[4], "window"), sinks = integer(a[5], "sinks");
    const int d = current_device_of(q), type = dtype_of(q);
    if (type < 0)
        refuse(PyExc_TypeError, "q must be float16 or bfloat16");
    if (q.dim() != 4)
        refuse(PyExc_ValueError, "q must be [batch, tokens, q_heads, head_dim]");
    const kv_cache_pool pool = pool_of(a[0], d);
    const int64_t batch = q.size(0), tokens = q.size(1), heads = q.size(2);
    if (q.size(3) != pool.head_dim || pool.kv_heads == 0 || heads == 0 || heads % pool.kv_heads != 0)
        refuse(PyExc_ValueError, "q has ", heads, " heads of ", q.size(3), ", the cache ", pool.kv_heads, " of ",
               pool.head_dim);
    if (window < 0 || sinks < 0)
        refuse(PyExc_ValueError, "window and sinks must not be negative");
    int64_t max_pages = 0, width = 0;
    const int32_t *pages = ints(tensor(a[2], "pages"), "pages", batch, d, &max_pages);
    const int32_t *lengths = ints(tensor(a[3], "lengths"), "lengths", batch, d);
    float *weights = nullptr;
    if (a[6] != Py_None) {
        const at::Tensor &w = tensor(a[6], "weights");
        if (w.scalar_type() != at::kFloat || w.dim() != 3 || !w.is_contiguous() || w.size(0) != batch ||
            w.size(1) != pool.kv_heads || !on(w, d) || w.size(2) < max_pages * pool.page)
            refuse(PyExc_ValueError, "weights must be contiguous float32 [batch, kv_heads, at least ",
                   max_pages * pool.page, "] on cuda:", d);
        weights = w.data_ptr<float>();
        width = w.size(2);
    }
    const at::Tensor o = output(q, a[7], d);
    if (batch > 0 && tokens > 0) {
        const Strides qs = strides_of(q, "q");
        void *stream = stream_of(d);
        at::Tensor space;
        if (a[8] == Py_None) {
            space = workspace_for(q, pool.kv_heads, width, d, stream);
        } else {
            space = tensor(a[8], "workspace");
            if (!on(space, d) || !space.is_contiguous())
                refuse(PyExc_ValueError, "workspace must be a contiguous tensor on cuda:", d);
        }
        done(f_attention(&pool, q.data_ptr(), type, batch, tokens, heads, qs.s, o.data_ptr(), pages, max_pages,
                         lengths, window, sinks, weights, width, space.data_ptr(), space.nbytes(), stream),
             "kv_cache_attention_x16");
    }
    return returned(o, a[7]);
}

PyObject *workspace_impl(PyObject *const *a) {
    const at::Tensor &q = tensor(a[0], "q");
    const int d = current_device_of(q);
    if (q.dim() != 4)
        refuse(PyExc_ValueError, "q must be [batch, tokens, q_heads, head_dim]");
    const kv_cache_pool pool = pool_of(a[1], d);
    const int64_t width = a[2] == Py_None ? 0 : tensor(a[2], "weights").size(-1);
    return THPVariable_Wrap(new_workspace(q, workspace_bytes(q, pool.kv_heads, width)));
}

PyObject *evict_impl(PyObject *const *a) {
    const at::Tensor &weights = tensor(a[1], "weights");
    const int d = current_device_of(weights);
    const kv_cache_pool pool = pool_of(a[0], d), to = pool_of(a[7], d);
    if (to.kv_heads != pool.kv_heads || to.page != pool.page || to.head_dim != pool.head_dim)
        refuse(PyExc_ValueError, "both pools must have the same kv_heads, page and head_dim");
    if (weights.dim() != 3 || weights.scalar_type() != at::kFloat || !weights.is_contiguous() ||
        weights.size(1) != pool.kv_heads)
        refuse(PyExc_ValueError, "weights must be contiguous float32 [batch, kv_heads, tokens]");
    const int64_t batch = weights.size(0), width = weights.size(2);
    const int64_t budget = integer(a[4], "budget"), sinks = integer(a[5], "sinks"), recent = integer(a[6], "recent");
    int64_t max_pages = 0, to_max = 0;
    const int32_t *pages = ints(tensor(a[2], "pages"), "pages", batch, d, &max_pages);
    const int32_t *lengths = ints(tensor(a[3], "lengths"), "lengths", batch, d);
    const int32_t *to_pages = ints(tensor(a[8], "to_pages"), "to_pages", batch, d, &to_max);
    if (width < max_pages * pool.page)
        refuse(PyExc_ValueError, "weights has room for ", width, " tokens, the page table for ", max_pages * pool.page);
    if (budget < 1 || sinks < 0 || recent < 0 || sinks > budget || recent > budget - sinks)
        refuse(PyExc_ValueError, "need budget >= 1, sinks and recent >= 0, sinks + recent <= budget");
    if (to_max * pool.page < budget)
        refuse(PyExc_ValueError, "to_pages has room for ", to_max * pool.page, " tokens, the budget is ", budget);
    const auto i32 = weights.options().dtype(at::kInt);
    const at::Tensor new_lengths = at::empty({batch}, i32);
    const at::Tensor new_weights = at::empty({batch, pool.kv_heads, to_max * pool.page}, weights.options());
    const at::Tensor kept = at::empty({batch, pool.kv_heads, budget}, i32);
    if (batch > 0)
        done(f_evict(&pool, weights.data_ptr<float>(), width, pages, max_pages, lengths, batch, budget, sinks,
                     recent, &to, to_pages, to_max, new_lengths.data_ptr<int32_t>(),
                     new_weights.data_ptr<float>(), kept.data_ptr<int32_t>(), stream_of(d)),
             "kv_cache_evict_e4m3");
    PyObject *x = THPVariable_Wrap(new_lengths), *y = THPVariable_Wrap(new_weights), *z = THPVariable_Wrap(kept);
    PyObject *r = x && y && z ? PyTuple_Pack(3, x, y, z) : nullptr;
    Py_XDECREF(x);
    Py_XDECREF(y);
    Py_XDECREF(z);
    return r;
}

template <PyObject *(*kImpl)(PyObject *const *), Py_ssize_t kArgs>
PyObject *entry(PyObject *, PyObject *const *args, Py_ssize_t n) {
    try {
        if (n != kArgs)
            refuse(PyExc_TypeError, "expected ", kArgs, " arguments, got ", n);
        if (!g_error)
            refuse(PyExc_RuntimeError, "bind() has not been called");
        return kImpl(args);
    } catch (const Raised &) {
    } catch (const Refusal &r) {
        PyErr_SetString(r.type, r.what.c_str());
    } catch (const c10::OutOfMemoryError &e) {   // what a caller who sheds load catches
        PyErr_SetString(g_no_memory, e.what_without_backtrace());
    } catch (const std::bad_alloc &) {
        PyErr_NoMemory();
    } catch (const std::exception &e) {
        PyErr_SetString(PyExc_RuntimeError, e.what());
    } catch (...) {
        PyErr_SetString(PyExc_RuntimeError, "unknown C++ exception");
    }
    return nullptr;
}

// bind(GemmReluError, torch.OutOfMemoryError, addresses of the seven library functions in the order below)
PyObject *bind(PyObject *, PyObject *args) {
    PyObject *error, *no_memory;
    unsigned long long f[7];
    if (!PyArg_ParseTuple(args, "OOKKKKKKK", &error, &no_memory, &f[0], &f[1], &f[2], &f[3], &f[4], &f[5], &f[6]))
        return nullptr;
    f_window = reinterpret_cast<decltype(f_window)>((uintptr_t)f[0]);
    f_append = reinterpret_cast<decltype(f_append)>((uintptr_t)f[1]);
    f_attention = reinterpret_cast<decltype(f_attention)>((uintptr_t)f[2]);
    f_workspace_bytes = reinterpret_cast<decltype(f_workspace_bytes)>((uintptr_t)f[3]);
    f_evict = reinterpret_cast<decltype(f_evict)>((uintptr_t)f[4]);
    f_capturing = reinterpret_cast<decltype(f_capturing)>((uintptr_t)f[5]);
    f_stream_id = reinterpret_cast<decltype(f_stream_id)>((uintptr_t)f[6]);
    Py_INCREF(error);
    Py_INCREF(no_memory);
    g_error = error;
    g_no_memory = no_memory;
    Py_RETURN_NONE;
}

#define ENTRY(name, impl, args) \
    {name, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(&entry<impl, args>)), METH_FASTCALL, nullptr}

PyMethodDef methods[] = {
    ENTRY("window", window_impl, 6),
    ENTRY("append", append_impl, 6),
    ENTRY("attention", attention_impl, 9),
    ENTRY("workspace", workspace_impl, 3),
    ENTRY("evict", evict_impl, 9),
    {"bind", bind, METH_VARARGS, nullptr},
    {nullptr, nullptr, 0, nullptr},
};

PyModuleDef module = {PyModuleDef_HEAD_INIT, "_serving", "Checks and calls of the serving operators.", -1, methods,
                      nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__serving(void) { return PyModule_Create(&module); }
