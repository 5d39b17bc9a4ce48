// torch_args.h -- what the modules behind the caches' Python classes share:
// checks of torch tensors and numbers, and the calls of a plan and a release.
// H is a cache's handle: `desc` with head_dim and max_pages, `device`.
#pragma once
#include <torch/csrc/autograd/python_variable.h>

#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAStream.h>

#include <exception>

#include "../../include/lookahead.h"

namespace {

// Thrown by the checks below; turned into ValueError.
struct Refused {
    const char* what;
};

const at::Tensor& tensor_of(PyObject* o, const char* what)
{
    if (!THPVariable_Check(o)) throw Refused{what};
    return THPVariable_Unpack(o);
}

long int_of(PyObject* o)
{
    const long v = PyLong_AsLong(o);
    if (v == -1 && PyErr_Occurred()) {
        PyErr_Clear();
        throw Refused{"expected a whole number"};
    }
    if (v < INT32_MIN || v > INT32_MAX) throw Refused{"a number does not fit 32 bits"};
    return v;
}

template <typename H>
bool here(const H& h, const at::Tensor& t) { return t.is_cuda() && t.get_device() == h.device; }

template <typename H>
const at::Tensor& ints(const H& h, PyObject* o)
{
    constexpr const char* kWhat = "expected contiguous int32 tensors on the cache's device";
    const at::Tensor& t = tensor_of(o, kWhat);
    if (t.scalar_type() != at::kInt || !here(h, t) || !t.is_contiguous()) throw Refused{kWhat};
    return t;
}

const int32_t* data(const at::Tensor& t) { return static_cast<const int32_t*>(t.data_ptr()); }
int32_t* out(const at::Tensor& t) { return static_cast<int32_t*>(t.data_ptr()); }

// whether two contiguous tensors share memory
bool share(const at::Tensor& a, const at::Tensor& b)
{
    const char *p = static_cast<const char*>(a.data_ptr()), *q = static_cast<const char*>(b.data_ptr());
    return p < q + b.nbytes() && q < p + a.nbytes();
}

// Row stride (elements) of [rows, heads * D] or [rows, heads, D] with dense rows.
template <typename H>
long row_stride(const H& h, const at::Tensor& t, long heads, const char* what)
{
    const long D = h.desc.head_dim;
    if (!here(h, t)) throw Refused{what};
    bool ok = false;
    if (t.dim() == 2) ok = t.size(1) == heads * D && t.stride(1) == 1;
    else if (t.dim() == 3) ok = t.size(1) == heads && t.size(2) == D && t.stride(2) == 1 && (heads == 1 || t.stride(1) == D);
    if (!ok) throw Refused{what};
    // the stride of a single row says nothing, and may differ between tensors of one layout
    const long ld = t.size(0) < 2 ? heads * D : t.stride(0);
    if (ld > INT32_MAX || t.size(0) > INT32_MAX) throw Refused{what};
    return ld;
}

int dtype_of(const at::Tensor& t)
{
    if (t.scalar_type() == at::kBFloat16) return LA_BF16;
    if (t.scalar_type() == at::kFloat) return LA_FP32;
    throw Refused{"k and v: bf16 or fp32"};
}

template <typename H>
void* stream_of(const H& h)
{
    if (c10::cuda::current_device() != h.device) throw Refused{"the cache's device is not the current one"};
    return c10::cuda::getCurrentCUDAStream(h.device).stream();
}

long count(const at::Tensor& t)
{
    if (t.numel() > INT32_MAX) throw Refused{"too many entries"};
    return t.numel();
}

template <typename H>
void rows_of_table(const H& h, const at::Tensor& table, long batch)
{
    if (table.dim() != 2 || table.size(0) != batch || table.size(1) != h.desc.max_pages)
        throw Refused{"table is [batch, max_pages]"};
}

// la_kv4_plan and la_kv4_release, which any cache of 4-bit pages' shapes can call: d describes it.
template <typename H>
int plan_of(const H& h, const la_kv4_desc& d, PyObject* const* a)
{
    const auto &lens = ints(h, a[1]), &n_new = ints(h, a[2]), &free_pages = ints(h, a[3]), &n_free = ints(h, a[4]),
               &table = ints(h, a[5]), &slots = ints(h, a[6]), &new_lens = ints(h, a[7]), &left = ints(h, a[8]);
    const long B = count(lens);
    if (n_new.numel() != B || new_lens.numel() != B) throw Refused{"plan: lens, n_new and new_lens of one length"};
    if (n_free.numel() < 1 || left.numel() < 1) throw Refused{"plan: n_free and pages_left hold one number"};
    rows_of_table(h, table, B);
    // (the C call does not know how far free_pages goes)
    for (const at::Tensor* t : {&table, &slots, &new_lens, &left})
        if (share(free_pages, *t)) throw Refused{"plan: free_pages shares memory with an output"};
    return la_kv4_plan(&d, data(lens), data(n_new), (int)B, data(free_pages), data(n_free), out(table), out(slots),
                       (int)count(slots), (int)int_of(a[9]), out(new_lens), out(left), stream_of(h));
}

template <typename H>
int release_of(const H& h, const la_kv4_desc& d, PyObject* const* a)
{
    const auto &done = ints(h, a[1]), &lens = ints(h, a[2]), &table = ints(h, a[3]), &free_pages = ints(h, a[4]),
               &n_free = ints(h, a[5]);
    const long B = count(lens);
    if (done.numel() != B) throw Refused{"release: done and lens of one length"};
    rows_of_table(h, table, B);
    if (free_pages.numel() < d.n_pages) throw Refused{"release: free_pages needs room for every page"};
    if (n_free.numel() < 1) throw Refused{"release: n_free holds one number"};
    return la_kv4_release(&d, data(done), (int)B, out(lens), data(table), out(free_pages), out(n_free), stream_of(h));
}

template <int (*F)(PyObject* const*), int NARGS>
PyObject* entry(PyObject*, PyObject* const* args, Py_ssize_t n)
{
    if (n != NARGS) {
        PyErr_SetString(PyExc_TypeError, "wrong number of arguments");
        return nullptr;
    }
    try {
        return PyLong_FromLong(F(args));
    } catch (const Refused& r) {
        PyErr_SetString(PyExc_ValueError, r.what);
    } catch (const std::exception& e) {
        PyErr_SetString(PyExc_RuntimeError, e.what());
    }
    return nullptr;
}

#define FAST(f) reinterpret_cast<PyCFunction>(reinterpret_cast<void*>(static_cast<PyObject* (*)(PyObject*, PyObject* const*, Py_ssize_t)>(f)))

}  // namespace
