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
    // the tensor given, or a new contiguous bf16 one
    at::Tensor output(int i, at::IntArrayRef shape)
    {
        if (!none(i))
            return tensor(i);
        return part(memory(c10::multiply_integers(shape)), 0, shape);
    }
    // Two of them.  New ones share one allocation, the second behind the first
    // (16-byte aligned: its rows are multiples of 8 elements): an allocation and
    // its release cost about as much as the launch of a small kernel.
    std::pair<at::Tensor, at::Tensor> outputs(int i, at::IntArrayRef a, int j, at::IntArrayRef b)
    {
        if (!none(i) || !none(j))
            return {output(i, a), output(j, b)};
        const int64_t n = c10::multiply_integers(a);
        const c10::Storage both = memory(n + c10::multiply_integers(b));
        return {part(both, 0, a), part(both, n, b)};
    }

private:
    // What at::empty takes too, from the same allocator, without its dispatch and
    // device guard (the device is current).
    static c10::Storage memory(int64_t elements)
    {
        c10::Allocator* const from = c10::cuda::CUDACachingAllocator::get();
        const size_t bytes = (size_t)elements * sizeof(at::BFloat16);
        return c10::Storage(c10::Storage::use_byte_size_t(), bytes, from->allocate(bytes), from, true);
    }
    // a contiguous bf16 tensor over memory from element `at` on
    static at::Tensor part(c10::Storage all, int64_t at, at::IntArrayRef shape)
    {
        at::Tensor t = at::detail::make_tensor<c10::TensorImpl>(
            std::move(all), c10::DispatchKeySet(c10::DispatchKey::CUDA), caffe2::TypeMeta::Make<at::BFloat16>());
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
        uint64_t need = 0;
        auto call = [&](void* workspace, uint64_t bytes) {
            return b2pa_tree_attention(q, k, v, bt, seq, cum, mask, pos, a.int32(9), a.int32(10), a.number(11),
                                       a.number(12), a.int32(13), sinks, a.int32(15), o, workspace, bytes, &need,
                                       a.stream());
        };
        int st = call(nullptr, 0);
        if (st == B2PA_ERR_WORKSPACE) {
            // from torch's allocator for this call, so that every captured graph keeps its own
            const c10::DataPtr workspace = c10::cuda::CUDACachingAllocator::get()->allocate(need);
            st = call(workspace.get(), need);
        }
        return st == B2PA_OK ? THPVariable_Wrap(out) : PyLong_FromLong(st);
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
    {nullptr, nullptr, 0, nullptr},
};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_native", "Direct bindings of a few calls of libb2pa.so.", -1, methods,
                      nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__native(void) { return PyModule_Create(&module); }
