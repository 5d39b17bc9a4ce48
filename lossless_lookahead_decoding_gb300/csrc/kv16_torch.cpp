// kv16_torch.cpp -- KV16Cache's calls from Python, as kv4_torch.cpp: checks
// torch tensors and calls the la_kv16_* C entry points (and la_kv4_plan and
// la_kv4_release) on torch's current stream.
#include "torch_args.h"

namespace {

constexpr char kName[] = "la_kv16";

struct Handle {
    la_kv16_desc desc;
    at::Tensor k_pages, v_pages, status;
    int device;
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

// the book-keeping calls do not look at the pages
la_kv4_desc book(const Handle& h)
{
    const la_kv16_desc& d = h.desc;
    return la_kv4_desc{d.n_kv_heads, d.head_dim, d.page, d.n_pages, d.max_pages, nullptr, d.status};
}

int call_plan(PyObject* const* a)
{
    Handle& h = *handle_of(a[0]);
    return plan_of(h, book(h), a);
}

int call_release(PyObject* const* a)
{
    Handle& h = *handle_of(a[0]);
    return release_of(h, book(h), a);
}

// an output of turned rows: bf16 [n, heads * D] or [n, heads, D]; its row stride
int out_rows(const Handle& h, const at::Tensor& t, long heads, long n, const char* what)
{
    const long ld = row_stride(h, t, heads, what);
    if (t.scalar_type() != at::kBFloat16 || t.size(0) != n) throw Refused{what};
    return (int)ld;
}

// 0 handle, 1 k, 2 v, 3 slots, 4 rows, 5 positions, 6 address of an la_rope, 7 k_out, 8 q, 9 q_out
int call_append(PyObject* const* a)
{
    Handle& h = *handle_of(a[0]);
    constexpr const char* kRows = "k, v, q: rows of heads x head_dim with unit stride inside a row, on the cache's device";
    la_kv16_rows r = {};
    const long D = h.desc.head_dim;
    const auto& k = tensor_of(a[1], kRows);
    r.k_ld = (int)row_stride(h, k, h.desc.n_kv_heads, kRows);
    r.k = k.data_ptr(), r.dtype = dtype_of(k), r.n_rows = (int)k.size(0);
    if (a[2] != Py_None) {
        const auto& v = tensor_of(a[2], kRows);
        r.v_ld = (int)row_stride(h, v, h.desc.n_kv_heads, kRows);
        if (v.scalar_type() != k.scalar_type() || v.size(0) != k.size(0)) throw Refused{"k and v of one type, with the same rows"};
        r.v = v.data_ptr();
    }
    long n = -1;  // the call's rows: all index tensors agree
    auto index = [&](PyObject* o) -> const int32_t* {
        if (o == Py_None) return nullptr;
        const auto& t = ints(h, o);
        if (n >= 0 && t.numel() != n) throw Refused{"append: slots, rows and positions of one length"};
        n = count(t);
        // (an empty tensor has no address, and a call without slots is another call)
        static const int32_t none = 0;
        return n ? data(t) : &none;
    };
    r.slots = index(a[3]), r.rows = index(a[4]), r.positions = index(a[5]);
    if (n < 0) n = k.size(0);
    r.n = (int)n;
    if (r.slots && !r.v) throw Refused{"append: slots need v"};
    if (a[6] != Py_None) {
        r.rope = static_cast<const la_rope*>(PyLong_AsVoidPtr(a[6]));
        if (!r.rope || PyErr_Occurred()) {
            PyErr_Clear();
            throw Refused{"append: not a rope"};
        }
        if (!r.positions) throw Refused{"append: a rope needs positions"};
    }
    if (a[7] != Py_None) {
        constexpr const char* kOut = "k_out: bf16 rows of KV heads x head_dim, one for each row of the call, on the cache's device";
        const auto& o = tensor_of(a[7], kOut);
        r.k_out_ld = out_rows(h, o, h.desc.n_kv_heads, n, kOut);
        r.k_out = o.data_ptr();
    }
    if ((a[8] == Py_None) != (a[9] == Py_None)) throw Refused{"append: q and q_out go together"};
    if (a[8] != Py_None) {
        constexpr const char* kOut = "q_out: bf16 rows as wide as q's, one for each row of the call, on the cache's device";
        const auto &q = tensor_of(a[8], kRows), &o = tensor_of(a[9], kOut);
        if (q.dim() < 2 || q.size(0) != k.size(0) || q.scalar_type() != k.scalar_type()) throw Refused{"append: q has k's type and rows"};
        const long H = q.dim() == 2 ? q.size(1) / D : q.size(1);
        if (H < 1) throw Refused{kRows};
        r.q_ld = (int)row_stride(h, q, H, kRows);
        r.q_out_ld = out_rows(h, o, H, n, kOut);
        r.q = q.data_ptr(), r.q_out = o.data_ptr(), r.n_heads = (int)H;
    }
    return la_kv16_append(&h.desc, &r, stream_of(h));
}

// 0 handle, 1 q, 2 k_step, 3 v_step, 4 lens, 5 table, 6 W, 7 N, 8 G, 9 out, 10 workspace, 11 max_len, 12 prefix_lens,
// 13 prefix_table, 14 prefix_first, 15 max_prefix_len
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
    la_kv16_attn c = {};
    c.q = q.data_ptr(), c.k_step = k.data_ptr(), c.v_step = v.data_ptr(), c.out = o.data_ptr();
    c.lens = data(lens), c.table = data(table);
    c.batch = (int)B, c.n_heads = (int)H, c.W = (int)W, c.N = (int)N, c.G = (int)G;
    c.q_ld = (int)row_stride(h, q, H, "q: rows of n_heads x head_dim with unit stride inside a row, on the cache's device");
    constexpr const char* kRows = "k_step, v_step: rows of KV heads x head_dim with unit stride inside a row, on the cache's device";
    c.k_ld = (int)row_stride(h, k, h.desc.n_kv_heads, kRows);
    c.v_ld = (int)row_stride(h, v, h.desc.n_kv_heads, kRows);
    if (a[10] != Py_None) {
        const auto& ws = tensor_of(a[10], "workspace: a tensor");
        if (!here(h, ws) || !ws.is_contiguous()) throw Refused{"workspace: contiguous, on the cache's device"};
        c.workspace = ws.data_ptr();
        c.ws_bytes = ws.nbytes();
    }
    c.max_len = (int)int_of(a[11]);
    if ((a[12] == Py_None) != (a[13] == Py_None) || (a[12] == Py_None) != (a[14] == Py_None))
        throw Refused{"attention: prefix_lens, prefix_table and prefix_first go together"};
    if (a[12] != Py_None) {
        const auto &pl = ints(h, a[12]), &pt = ints(h, a[13]), &pf = ints(h, a[14]);
        const long nP = count(pl);
        if (nP > 8192) throw Refused{"attention: at most 8192 prefixes"};
        if (nP && (pt.dim() != 2 || pt.size(0) != nP || pt.size(1) < 1 || pt.size(1) > INT32_MAX || pf.numel() != nP + 1))
            throw Refused{"attention: prefix_table is [prefixes, pages], prefix_first holds one number more than prefix_lens"};
        c.n_prefix = (int)nP;
        if (nP) c.prefix_pages = (int)pt.size(1), c.prefix_lens = data(pl), c.prefix_table = data(pt), c.prefix_first = data(pf);
    }
    c.max_prefix_len = (int)int_of(a[15]);
    return la_kv16_attention(&h.desc, &c, stream_of(h));
}

void drop(PyObject* o) { delete static_cast<Handle*>(PyCapsule_GetPointer(o, kName)); }

// handle(k_pages, v_pages, status, address of an la_kv16_desc): the description is copied
PyObject* make_handle(PyObject*, PyObject* const* a, Py_ssize_t n)
{
    if (n != 4 || !THPVariable_Check(a[0]) || !THPVariable_Check(a[1]) || !THPVariable_Check(a[2]) || !PyLong_Check(a[3])) {
        PyErr_SetString(PyExc_TypeError, "handle(k_pages, v_pages, status, address)");
        return nullptr;
    }
    try {
        const auto* d = static_cast<const la_kv16_desc*>(PyLong_AsVoidPtr(a[3]));
        auto* h = new Handle{*d, THPVariable_Unpack(a[0]), THPVariable_Unpack(a[1]), THPVariable_Unpack(a[2]), 0};
        h->device = h->k_pages.get_device();
        return PyCapsule_New(h, kName, drop);
    } catch (const std::exception& e) {
        PyErr_SetString(PyExc_RuntimeError, e.what());
    }
    return nullptr;
}

PyMethodDef kMethods[] = {{"handle", FAST(make_handle), METH_FASTCALL, nullptr},
                          {"plan", FAST((entry<call_plan, 10>)), METH_FASTCALL, nullptr},
                          {"release", FAST((entry<call_release, 6>)), METH_FASTCALL, nullptr},
                          {"append", FAST((entry<call_append, 10>)), METH_FASTCALL, nullptr},
                          {"attention", FAST((entry<call_attention, 16>)), METH_FASTCALL, nullptr},
                          {nullptr, nullptr, 0, nullptr}};
PyModuleDef kModule = {PyModuleDef_HEAD_INIT, "_kv16", nullptr, -1, kMethods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

extern "C" __attribute__((visibility("default"))) PyObject* PyInit__kv16() { return PyModule_Create(&kModule); }
