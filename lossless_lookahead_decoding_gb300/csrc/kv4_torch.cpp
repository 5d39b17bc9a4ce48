// kv4_torch.cpp -- KV4Cache's calls from Python: checks torch tensors and
// calls the la_kv4_* C entry points on torch's current stream.
//
// A step of a served batch makes three of these calls per layer, each a launch
// of a few microseconds, so the checks run here and not in Python: a call
// costs about as much as the launch itself.  The functions return the C status
// code; a tensor that does not fit raises ValueError.  A handle (a capsule)
// holds one cache's description and keeps its tensors alive.
#include <torch/csrc/autograd/python_variable.h>

#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAStream.h>

#include <exception>

#include "../../include/lookahead.h"

namespace {

constexpr char kName[] = "la_kv4";

struct Handle {
    la_kv4_desc desc;
    at::Tensor pages, status;
    int device;
};

// Thrown by the checks below; turned into ValueError.
struct Refused {
    const char* what;
};

Handle* handle_of(PyObject* o)
{
    auto* h = static_cast<Handle*>(PyCapsule_GetPointer(o, kName));
    if (!h) {
        PyErr_Clear();
        throw Refused{"not a cache handle"};
    }
    return h;
}

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

bool here(const Handle& h, const at::Tensor& t) { return t.is_cuda() && t.get_device() == h.device; }

const at::Tensor& ints(const Handle& h, PyObject* o)
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
long row_stride(const Handle& h, const at::Tensor& t, long heads, const char* what)
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

void* stream_of(const Handle& h)
{
    if (c10::cuda::current_device() != h.device) throw Refused{"the cache's device is not the current one"};
    return c10::cuda::getCurrentCUDAStream(h.device).stream();
}

long count(const at::Tensor& t)
{
    if (t.numel() > INT32_MAX) throw Refused{"too many entries"};
    return t.numel();
}

void rows_of_table(const Handle& h, const at::Tensor& table, long batch)
{
    if (table.dim() != 2 || table.size(0) != batch || table.size(1) != h.desc.max_pages)
        throw Refused{"table is [batch, max_pages]"};
}

int call_plan(PyObject* const* a)
{
    Handle& h = *handle_of(a[0]);
    const auto &lens = ints(h, a[1]), &n_new = ints(h, a[2]), &free_pages = ints(h, a[3]), &n_free = ints(h, a[4]),
               &table = ints(h, a[5]), &slots = ints(h, a[6]), &new_lens = ints(h, a[7]), &left = ints(h, a[8]);
    const long B = count(lens);
    if (n_new.numel() != B || new_lens.numel() != B) throw Refused{"plan: lens, n_new and new_lens of one length"};
    if (n_free.numel() < 1 || left.numel() < 1) throw Refused{"plan: n_free and pages_left hold one number"};
    rows_of_table(h, table, B);
    // (the C call does not know how far free_pages goes)
    for (const at::Tensor* t : {&table, &slots, &new_lens, &left})
        if (share(free_pages, *t)) throw Refused{"plan: free_pages shares memory with an output"};
    return la_kv4_plan(&h.desc, data(lens), data(n_new), (int)B, data(free_pages), data(n_free), out(table), out(slots),
                       (int)count(slots), (int)int_of(a[9]), out(new_lens), out(left), stream_of(h));
}

int call_release(PyObject* const* a)
{
    Handle& h = *handle_of(a[0]);
    const auto &done = ints(h, a[1]), &lens = ints(h, a[2]), &table = ints(h, a[3]), &free_pages = ints(h, a[4]),
               &n_free = ints(h, a[5]);
    const long B = count(lens);
    if (done.numel() != B) throw Refused{"release: done and lens of one length"};
    rows_of_table(h, table, B);
    if (free_pages.numel() < h.desc.n_pages) throw Refused{"release: free_pages needs room for every page"};
    if (n_free.numel() < 1) throw Refused{"release: n_free holds one number"};
    return la_kv4_release(&h.desc, data(done), (int)B, out(lens), data(table), out(free_pages), out(n_free), stream_of(h));
}

int call_append(PyObject* const* a)
{
    Handle& h = *handle_of(a[0]);
    constexpr const char* kRows = "k, v: rows of heads x head_dim with unit stride inside a row, on the cache's device";
    const auto &k = tensor_of(a[1], kRows), &v = tensor_of(a[2], kRows), &slots = ints(h, a[3]);
    const long ld = row_stride(h, k, h.desc.n_kv_heads, kRows), n = count(slots);
    if (row_stride(h, v, h.desc.n_kv_heads, kRows) != ld || v.scalar_type() != k.scalar_type() || v.size(0) != k.size(0))
        throw Refused{"k and v of one type and layout"};
    const int32_t* rows = nullptr;
    if (a[4] != Py_None) {
        const auto& r = ints(h, a[4]);
        if (r.numel() != n) throw Refused{"append: one row for each slot"};
        rows = data(r);
    }
    return la_kv4_append(&h.desc, k.data_ptr(), v.data_ptr(), dtype_of(k), (int)ld, (int)k.size(0), rows, data(slots),
                         (int)n, stream_of(h));
}

int call_read(PyObject* const* a)
{
    Handle& h = *handle_of(a[0]);
    constexpr const char* kRows = "k, v: rows of heads x head_dim with unit stride inside a row, on the cache's device";
    const auto &slots = ints(h, a[1]), &k = tensor_of(a[2], kRows), &v = tensor_of(a[3], kRows);
    const long ld = row_stride(h, k, h.desc.n_kv_heads, kRows), n = count(slots);
    if (row_stride(h, v, h.desc.n_kv_heads, kRows) != ld || v.scalar_type() != k.scalar_type())
        throw Refused{"k and v of one type and layout"};
    if (k.size(0) < n || v.size(0) < n) throw Refused{"read: fewer rows than slots"};
    return la_kv4_read(&h.desc, data(slots), (int)n, k.data_ptr(), v.data_ptr(), dtype_of(k), (int)ld, stream_of(h));
}

int call_attention(PyObject* const* a)
{
    Handle& h = *handle_of(a[0]);
    const auto &q = tensor_of(a[1], "q: a tensor"), &k = tensor_of(a[2], "k_step: a tensor"),
               &v = tensor_of(a[3], "v_step: a tensor"), &lens = ints(h, a[4]), &table = ints(h, a[5]),
               &o = tensor_of(a[9], "out: a tensor");
    const long D = h.desc.head_dim, B = count(lens), W = int_of(a[6]), N = int_of(a[7]), G = int_of(a[8]);
    if (W < 0 || G < 0 || W > 127 || G > 127 || N < 2 || N > 128) throw Refused{"attention: W, N or G out of range"};
    const long rows = B * (1 + (W + G) * (N - 1));
    if (o.dim() != 2 || !o.is_contiguous() || !here(h, o) || o.size(0) != rows || o.size(1) % D)
        throw Refused{"attention: out is contiguous [batch * T, n_heads * head_dim] on the cache's device"};
    const long H = o.size(1) / D;
    if (q.scalar_type() != at::kBFloat16 || k.scalar_type() != at::kBFloat16 || v.scalar_type() != at::kBFloat16 ||
        o.scalar_type() != at::kBFloat16)
        throw Refused{"attention: bf16 only"};
    if (q.dim() < 1 || k.dim() < 1 || v.dim() < 1 || q.size(0) != rows || k.size(0) != rows || v.size(0) != rows)
        throw Refused{"attention: q, k_step and v_step have out's rows"};
    rows_of_table(h, table, B);
    la_kv4_attn c;
    c.q = q.data_ptr(), c.k_step = k.data_ptr(), c.v_step = v.data_ptr(), c.out = o.data_ptr();
    c.lens = data(lens), c.table = data(table);
    c.batch = (int)B, c.n_heads = (int)H, c.W = (int)W, c.N = (int)N, c.G = (int)G;
    c.q_ld = (int)row_stride(h, q, H, "q: rows of n_heads x head_dim with unit stride inside a row, on the cache's device");
    constexpr const char* kRows = "k_step, v_step: rows of KV heads x head_dim, of one layout, on the cache's device";
    c.kv_ld = (int)row_stride(h, k, h.desc.n_kv_heads, kRows);
    if (row_stride(h, v, h.desc.n_kv_heads, kRows) != c.kv_ld) throw Refused{kRows};
    c.workspace = nullptr, c.ws_bytes = 0;
    if (a[10] != Py_None) {
        const auto& ws = tensor_of(a[10], "workspace: a tensor");
        if (!here(h, ws) || !ws.is_contiguous()) throw Refused{"workspace: contiguous, on the cache's device"};
        c.workspace = ws.data_ptr();
        c.ws_bytes = ws.nbytes();
    }
    c.max_len = (int)int_of(a[11]);
    return la_kv4_attention(&h.desc, &c, stream_of(h));
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

void drop(PyObject* o) { delete static_cast<Handle*>(PyCapsule_GetPointer(o, kName)); }

// handle(pages, status, address of an la_kv4_desc): the description is copied
PyObject* make_handle(PyObject*, PyObject* const* a, Py_ssize_t n)
{
    if (n != 3 || !THPVariable_Check(a[0]) || !THPVariable_Check(a[1]) || !PyLong_Check(a[2])) {
        PyErr_SetString(PyExc_TypeError, "handle(pages, status, address)");
        return nullptr;
    }
    try {
        const auto* d = static_cast<const la_kv4_desc*>(PyLong_AsVoidPtr(a[2]));
        auto* h = new Handle{*d, THPVariable_Unpack(a[0]), THPVariable_Unpack(a[1]), 0};
        h->device = h->pages.get_device();
        return PyCapsule_New(h, kName, drop);
    } catch (const std::exception& e) {
        PyErr_SetString(PyExc_RuntimeError, e.what());
    }
    return nullptr;
}

#define FAST(f) reinterpret_cast<PyCFunction>(reinterpret_cast<void*>(static_cast<PyObject* (*)(PyObject*, PyObject* const*, Py_ssize_t)>(f)))
PyMethodDef kMethods[] = {{"handle", FAST(make_handle), METH_FASTCALL, nullptr},
                          {"plan", FAST((entry<call_plan, 10>)), METH_FASTCALL, nullptr},
                          {"release", FAST((entry<call_release, 6>)), METH_FASTCALL, nullptr},
                          {"append", FAST((entry<call_append, 5>)), METH_FASTCALL, nullptr},
                          {"read", FAST((entry<call_read, 4>)), METH_FASTCALL, nullptr},
                          {"attention", FAST((entry<call_attention, 12>)), METH_FASTCALL, nullptr},
                          {nullptr, nullptr, 0, nullptr}};
PyModuleDef kModule = {PyModuleDef_HEAD_INIT, "_kv4", nullptr, -1, kMethods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

extern "C" __attribute__((visibility("default"))) PyObject* PyInit__kv4() { return PyModule_Create(&kModule); }
