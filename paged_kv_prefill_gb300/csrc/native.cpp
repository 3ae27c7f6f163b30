// native.cpp -- the calls of include/b2pa.h that take many tensors and a few
// microseconds of GPU time, bound to Python without ctypes: a tensor becomes a
// descriptor in C++ and outputs are allocated here.  Marshalling only.  (For a
// rotation of 32 tokens ctypes and Python took 20 us, the kernel 4.)
//
// Every function takes the stream's handle first; its device is current and
// new tensors come from the memory of its current stream (the Python side sees
// to both).  They return their output, or the status of a call that failed.
#include <Python.h>

#include <ATen/core/Tensor.h>
#include <c10/cuda/CUDACachingAllocator.h>
#include <torch/csrc/autograd/python_variable.h>

#include <exception>
#include <utility>

#include "../../include/b2pa.h"

namespace {

struct Refused {  // a Python error is set
};

// The arguments of a call: descriptors of its tensors, all on one CUDA device.
class Args {
public:
    Args(PyObject* const* args, Py_ssize_t n, Py_ssize_t want) : args_(args)
    {
        if (n != want) {
            PyErr_Format(PyExc_TypeError, "%zd arguments, not %zd", want, n);
            throw Refused{};
        }
    }
    const at::Tensor& tensor(int i)
    {
        if (!THPVariable_Check(args_[i])) {
            PyErr_Format(PyExc_TypeError, "argument %d must be a tensor, not %.100s", i, Py_TYPE(args_[i])->tp_name);
            throw Refused{};
        }
        return THPVariable_Unpack(args_[i]);
    }
    bool none(int i) const { return args_[i] == Py_None; }
    // null for None where that is allowed
    const b2pa_tensor* desc(int i, bool optional = false)
    {
        return optional && none(i) ? nullptr : describe(tensor(i));
    }
    const b2pa_tensor* describe(const at::Tensor& t)
    {
        if (!t.is_cuda()) {
            PyErr_Format(PyExc_ValueError, "tensors on %s: CUDA tensors are needed", t.device().str().c_str());
            throw Refused{};
        }
        if (used_ > 0 && t.device() != device_) {
            PyErr_Format(PyExc_ValueError, "tensors on %s and %s: one device per call", device_.str().c_str(),
                         t.device().str().c_str());
            throw Refused{};
        }
        device_ = t.device();
        b2pa_tensor& d = d_[used_++];
        switch (t.scalar_type()) {
        case at::kBFloat16: d.dtype = B2PA_BF16; break;
        case at::kFloat8_e4m3fn: d.dtype = B2PA_FP8_E4M3; break;
        case at::kFloat: d.dtype = B2PA_FP32; break;
        case at::kInt: d.dtype = B2PA_INT32; break;
        default:
            PyErr_Format(PyExc_TypeError, "unsupported dtype %s", c10::toString(t.scalar_type()));
            throw Refused{};
        }
        const int64_t n = t.dim();
        if (n > 5) {
            PyErr_SetString(PyExc_ValueError, "rank > 5");
            throw Refused{};
        }
        d.data = t.data_ptr();
        d.ndim = (int32_t)n;
        for (int64_t k = 0; k < n; ++k) {
            d.shape[k] = t.size(k);
            d.stride[k] = t.stride(k);
        }
        return &d;
    }
    long long integer(int i)
    {
        const long long v = PyLong_AsLongLong(args_[i]);
        if (v == -1 && PyErr_Occurred())
            throw Refused{};
        return v;
    }
    int32_t int32(int i)
    {
        const long long v = integer(i);
        if (v < INT32_MIN || v > INT32_MAX) {
            PyErr_Format(PyExc_OverflowError, "argument %d: %lld does not fit 32 bits", i, v);
            throw Refused{};
        }
        return (int32_t)v;
    }
    float number(int i)
    {
        const double v = PyFloat_AsDouble(args_[i]);
        if (v == -1.0 && PyErr_Occurred())
            throw Refused{};
        return (float)v;
    }
    b2pa_stream_t stream()
    {
        const unsigned long long v = PyLong_AsUnsignedLongLong(args_[0]);
        if (PyErr_Occurred())
            throw Refused{};
        return reinterpret_cast<b2pa_stream_t>(v);
    }
    // the tensor given, or a new contiguous one
    template <typename T = at::BFloat16>
    at::Tensor output(int i, at::IntArrayRef shape)
    {
        if (!none(i))
            return tensor(i);
        return part<T>(memory<T>(c10::multiply_integers(shape)), 0, shape);
    }
    // Two of them.  New ones share one allocation, the second behind the first
    // (bf16: 16-byte aligned, its rows are multiples of 8 elements): an allocation and
    // its release cost about as much as the launch of a small kernel.
    template <typename T = at::BFloat16>
    std::pair<at::Tensor, at::Tensor> outputs(int i, at::IntArrayRef a, int j, at::IntArrayRef b)
    {
        if (!none(i) || !none(j))
            return {output<T>(i, a), output<T>(j, b)};
        const int64_t n = c10::multiply_integers(a);
        const c10::Storage both = memory<T>(n + c10::multiply_integers(b));
        return {part<T>(both, 0, a), part<T>(both, n, b)};
    }

private:
    // What at::empty takes too, from the same allocator, without its dispatch and
    // device guard (the device is current).
    template <typename T>
    static c10::Storage memory(int64_t elements)
    {
        c10::Allocator* const from = c10::cuda::CUDACachingAllocator::get();
        const size_t bytes = (size_t)elements * sizeof(T);
        return c10::Storage(c10::Storage::use_byte_size_t(), bytes, from->allocate(bytes), from, true);
    }
    // a contiguous tensor over memory from element `at` on
    template <typename T>
    static at::Tensor part(c10::Storage all, int64_t at, at::IntArrayRef shape)
    {
        at::Tensor t = at::detail::make_tensor<c10::TensorImpl>(
            std::move(all), c10::DispatchKeySet(c10::DispatchKey::CUDA), caffe2::TypeMeta::Make<T>());
        t.unsafeGetTensorImpl()->set_sizes_contiguous(shape);
        t.unsafeGetTensorImpl()->set_storage_offset(at);
        return t;
    }
    PyObject* const* args_;
    at::Device device_ = at::kCPU;
    int used_ = 0;
    b2pa_tensor d_[12];
};

// No C++ exception may reach Python.
template <typename F>
PyObject* guarded(F&& f)
{
    try {
        return f();
    } catch (const Refused&) {
    } catch (const c10::OutOfMemoryError& e) {
        PyObject* torch = PyImport_ImportModule("torch");
        PyObject* type = torch ? PyObject_GetAttrString(torch, "OutOfMemoryError") : nullptr;
        if (type)
            PyErr_SetString(type, e.what_without_backtrace());
        Py_XDECREF(type);
        Py_XDECREF(torch);
    } catch (const std::exception& e) {
        PyErr_SetString(PyExc_RuntimeError, e.what());
    } catch (...) {
        PyErr_SetString(PyExc_RuntimeError, "unknown error");
    }
    return nullptr;
}

PyObject* two(int status, const at::Tensor& a, const at::Tensor& b)
{
    if (status != B2PA_OK)
        return PyLong_FromLong(status);
    PyObject* x = THPVariable_Wrap(a);
    PyObject* y = x ? THPVariable_Wrap(b) : nullptr;
    PyObject* t = y ? PyTuple_Pack(2, x, y) : nullptr;
    Py_XDECREF(x);
    Py_XDECREF(y);
    return t;
}

// stream, q, k, cos_sin, positions, q_weight, k_weight, eps, axis_of (bytes), interleaved, q_out, k_out
PyObject* qk_norm_rope(PyObject*, PyObject* const* args, Py_ssize_t n)
{
    return guarded([&]() -> PyObject* {
        Args a(args, n, 12);
        const b2pa_tensor *q = a.desc(1), *k = a.desc(2), *cs = a.desc(3), *pos = a.desc(4);
        const b2pa_tensor *qw = a.desc(5, true), *kw = a.desc(6, true);
        const int32_t* axes = nullptr;
        if (!a.none(8)) {
            const char* bytes = PyBytes_AsString(args[8]);
            if (!bytes)
                throw Refused{};
            axes = reinterpret_cast<const int32_t*>(bytes);
        }
        const auto [qo, ko] = a.outputs(10, a.tensor(1).sizes(), 11, a.tensor(2).sizes());
        // (the outputs' descriptors are read only)
        return two(b2pa_qk_norm_rope(q, k, cs, pos, qw, kw, a.number(7), axes, a.int32(9),
                                     const_cast<b2pa_tensor*>(a.describe(qo)), const_cast<b2pa_tensor*>(a.describe(ko)),
                                     a.stream()),
                   qo, ko);
    });
}

// stream, k_new, v_new, k_pool, v_pool, k_scales, v_scales, cache_loc, layout
PyObject* append_kv_scaled(PyObject*, PyObject* const* args, Py_ssize_t n)
{
    return guarded([&]() -> PyObject* {
        Args a(args, n, 9);
        const b2pa_tensor* d[7];
        for (int i = 0; i < 7; ++i)
            d[i] = a.desc(1 + i);
        return PyLong_FromLong(b2pa_append_kv_scaled(d[0], d[1], d[2], d[3], d[4], d[5], d[6], a.int32(8), a.stream()));
    });
}

// stream, k_pool, v_pool, k_scales, v_scales, cache_loc, layout, k_out, v_out
PyObject* read_kv_scaled(PyObject*, PyObject* const* args, Py_ssize_t n)
{
    return guarded([&]() -> PyObject* {
        Args a(args, n, 9);
        const b2pa_tensor* d[5];
        for (int i = 0; i < 5; ++i)
            d[i] = a.desc(1 + i);
        const int32_t layout = a.int32(6);
        // (shapes that cannot be are refused by the call)
        const bool ok = d[0]->ndim == 4 && d[4]->ndim == 1;
        const int64_t shape[3] = {ok ? d[4]->shape[0] : 0, ok ? d[0]->shape[layout == B2PA_HND ? 1 : 2] : 0,
                                  ok ? d[0]->shape[3] : 0};
        const auto [ko, vo] = a.outputs(7, shape, 8, shape);
        return two(b2pa_read_kv_scaled(d[0], d[1], d[2], d[3], d[4], layout, const_cast<b2pa_tensor*>(a.describe(ko)),
                                       const_cast<b2pa_tensor*>(a.describe(vo)), a.stream()),
                   ko, vo);
    });
}

// A call that says how much workspace it needs.  That comes from torch's allocator
// for this call, so that every captured graph keeps its own.
template <typename F>
int with_workspace(F&& call)
{
    uint64_t need = 0;
    const int st = call(nullptr, 0, &need);
    if (st != B2PA_ERR_WORKSPACE)
        return st;
    const c10::DataPtr workspace = c10::cuda::CUDACachingAllocator::get()->allocate(need);
    return call(workspace.get(), need, &need);
}

// stream, q, k_pool, v_pool, block_tables, seq_lens, cum_q, tree_mask, positions, max_q_len, max_kv_len, bmm1_scale,
// bmm2_scale, window_left, sinks, layout, out
PyObject* tree_attention(PyObject*, PyObject* const* args, Py_ssize_t n)
{
    return guarded([&]() -> PyObject* {
        Args a(args, n, 17);
        const b2pa_tensor *q = a.desc(1), *k = a.desc(2), *v = a.desc(3), *bt = a.desc(4), *seq = a.desc(5);
        const b2pa_tensor *cum = a.desc(6), *mask = a.desc(7), *pos = a.desc(8, true), *sinks = a.desc(14, true);
        const at::Tensor out = a.output(16, a.tensor(1).sizes());
        b2pa_tensor* o = const_cast<b2pa_tensor*>(a.describe(out));
        const int st = with_workspace([&](void* workspace, uint64_t bytes, uint64_t* need) {
            return b2pa_tree_attention(q, k, v, bt, seq, cum, mask, pos, a.int32(9), a.int32(10), a.number(11),
                                       a.number(12), a.int32(13), sinks, a.int32(15), o, workspace, bytes, need,
                                       a.stream());
        });
        return st == B2PA_OK ? THPVariable_Wrap(out) : PyLong_FromLong(st);
    });
}

// stream, q, k_pool, v_pool, prefix_tables, prefix_lens, cum_groups, block_tables, seq_lens, cum_q, max_q_len,
// max_group_q_len, max_prefix_len, max_kv_len, bmm1_scale, bmm2_scale, sinks, layout, out
PyObject* prefix_attention(PyObject*, PyObject* const* args, Py_ssize_t n)
{
    return guarded([&]() -> PyObject* {
        Args a(args, n, 19);
        const b2pa_tensor *q = a.desc(1), *k = a.desc(2), *v = a.desc(3), *pt = a.desc(4), *pl = a.desc(5);
        const b2pa_tensor *cg = a.desc(6), *bt = a.desc(7), *seq = a.desc(8), *cum = a.desc(9), *sinks = a.desc(16, true);
        const at::Tensor out = a.output(18, a.tensor(1).sizes());
        b2pa_tensor* o = const_cast<b2pa_tensor*>(a.describe(out));
        const int st = with_workspace([&](void* workspace, uint64_t bytes, uint64_t* need) {
            return b2pa_prefix_attention(q, k, v, pt, pl, cg, bt, seq, cum, a.int32(10), a.int32(11), a.int32(12),
                                         a.int32(13), a.number(14), a.number(15), sinks, a.int32(17), o, workspace,
                                         bytes, need, a.stream());
        });
        return st == B2PA_OK ? THPVariable_Wrap(out) : PyLong_FromLong(st);
    });
}

// stream, target_probs, draft_probs, tokens, parents, uniforms, last_uniforms, cum_q, max_q_len, accepted, counts,
// next_tokens
PyObject* verify_trees(PyObject*, PyObject* const* args, Py_ssize_t n)
{
    return guarded([&]() -> PyObject* {
        Args a(args, n, 12);
        const b2pa_tensor *p = a.desc(1), *q = a.desc(2, true), *tok = a.desc(3), *par = a.desc(4), *u = a.desc(5);
        const b2pa_tensor *last = a.desc(6), *cum = a.desc(7);
        const int32_t width = a.int32(8);
        // (shapes that cannot be are refused by the call)
        const int64_t B = last->ndim == 1 ? last->shape[0] : 0;
        const at::Tensor acc = a.output<int32_t>(9, {B, width > 0 ? width : 0});
        const auto [cnt, next] = a.outputs<int32_t>(10, {B}, 11, {B});
        const int st = b2pa_verify_trees(p, q, tok, par, u, last, cum, width, const_cast<b2pa_tensor*>(a.describe(acc)),
                                         const_cast<b2pa_tensor*>(a.describe(cnt)),
                                         const_cast<b2pa_tensor*>(a.describe(next)), a.stream());
        if (st != B2PA_OK)
            return PyLong_FromLong(st);
        PyObject* o[3] = {THPVariable_Wrap(acc), THPVariable_Wrap(cnt), THPVariable_Wrap(next)};
        PyObject* t = o[0] && o[1] && o[2] ? PyTuple_Pack(3, o[0], o[1], o[2]) : nullptr;
        for (PyObject* x : o)
            Py_XDECREF(x);
        return t;
    });
}

// stream, k_pool, v_pool, k_scales, v_scales, src, dst, layout
PyObject* copy_pages(PyObject*, PyObject* const* args, Py_ssize_t n)
{
    return guarded([&]() -> PyObject* {
        Args a(args, n, 8);
        const b2pa_tensor *k = a.desc(1), *v = a.desc(2), *ks = a.desc(3, true), *vs = a.desc(4, true);
        const b2pa_tensor *src = a.desc(5), *dst = a.desc(6);
        return PyLong_FromLong(b2pa_copy_pages(k, v, ks, vs, src, dst, a.int32(7), a.stream()));
    });
}

// stream, k_pool, v_pool, k_scales, v_scales, block_tables, seq_lens, cum_q, accepted, counts, new_lens, layout
PyObject* compact_kv(PyObject*, PyObject* const* args, Py_ssize_t n)
{
    return guarded([&]() -> PyObject* {
        Args a(args, n, 12);
        const b2pa_tensor *k = a.desc(1), *v = a.desc(2), *ks = a.desc(3, true), *vs = a.desc(4, true);
        const b2pa_tensor *bt = a.desc(5), *seq = a.desc(6), *cum = a.desc(7), *acc = a.desc(8), *cnt = a.desc(9);
        const at::Tensor lens = a.output<int32_t>(10, a.tensor(6).sizes());
        const int st = b2pa_compact_kv(k, v, ks, vs, bt, seq, cum, acc, cnt, const_cast<b2pa_tensor*>(a.describe(lens)),
                                       a.int32(11), a.stream());
        return st == B2PA_OK ? THPVariable_Wrap(lens) : PyLong_FromLong(st);
    });
}

// stream, block_tables, seq_lens, page_refs, rows, page_size
PyObject* free_pages(PyObject*, PyObject* const* args, Py_ssize_t n)
{
    return guarded([&]() -> PyObject* {
        Args a(args, n, 6);
        const b2pa_tensor *bt = a.desc(1), *seq = a.desc(2), *refs = a.desc(3), *rows = a.desc(4);
        return PyLong_FromLong(b2pa_free_pages(bt, seq, refs, rows, a.int32(5), a.stream()));
    });
}

// stream, block_tables, seq_lens, page_refs, parents, children, page_size, src, dst
PyObject* fork_pages(PyObject*, PyObject* const* args, Py_ssize_t n)
{
    return guarded([&]() -> PyObject* {
        Args a(args, n, 9);
        const b2pa_tensor *bt = a.desc(1), *seq = a.desc(2), *refs = a.desc(3), *from = a.desc(4), *to = a.desc(5);
        const auto [src, dst] = a.outputs<int32_t>(7, a.tensor(5).sizes(), 8, a.tensor(5).sizes());
        return two(b2pa_fork_pages(bt, seq, refs, from, to, a.int32(6), const_cast<b2pa_tensor*>(a.describe(src)),
                                   const_cast<b2pa_tensor*>(a.describe(dst)), a.stream()),
                   src, dst);
    });
}

// stream, block_tables, seq_lens, page_refs, rows, new_lens, page_size
PyObject* grow_pages(PyObject*, PyObject* const* args, Py_ssize_t n)
{
    return guarded([&]() -> PyObject* {
        Args a(args, n, 7);
        const b2pa_tensor *bt = a.desc(1), *seq = a.desc(2), *refs = a.desc(3), *rows = a.desc(4), *to = a.desc(5);
        return PyLong_FromLong(b2pa_grow_pages(bt, seq, refs, rows, to, a.int32(6), a.stream()));
    });
}

PyMethodDef methods[] = {
    {"qk_norm_rope", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(qk_norm_rope)), METH_FASTCALL, nullptr},
    {"append_kv_scaled", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(append_kv_scaled)), METH_FASTCALL,
     nullptr},
    {"read_kv_scaled", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(read_kv_scaled)), METH_FASTCALL,
     nullptr},
    {"tree_attention", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(tree_attention)), METH_FASTCALL,
     nullptr},
    {"prefix_attention", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(prefix_attention)), METH_FASTCALL,
     nullptr},
    {"verify_trees", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(verify_trees)), METH_FASTCALL, nullptr},
    {"copy_pages", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(copy_pages)), METH_FASTCALL, nullptr},
    {"compact_kv", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(compact_kv)), METH_FASTCALL, nullptr},
    {"free_pages", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(free_pages)), METH_FASTCALL, nullptr},
    {"fork_pages", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(fork_pages)), METH_FASTCALL, nullptr},
    {"grow_pages", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(grow_pages)), METH_FASTCALL, nullptr},
    {nullptr, nullptr, 0, nullptr},
};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_native", "Direct bindings of a few calls of libb2pa.so.", -1, methods,
                      nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__native(void) { return PyModule_Create(&module); }
