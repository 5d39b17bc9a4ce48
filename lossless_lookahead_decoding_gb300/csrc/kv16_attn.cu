// kv16_attn.cu -- the step's masked attention over the paged bf16 cache, for
// sequences that share prefixes.
//
// A row's keys are its prefix's tokens, its sequence's own and the step's rows
// that it sees: o = sum p_j v_j / sum p_j, p_j = exp2(s_j f - m) with f =
// log2(e) / sqrt(D) and m the running largest of s_j f.
#include "kv16.cuh"

namespace la {
namespace {

constexpr float kNoRef = -3e38f;  // below every score

// One warp per row and query head; a lane holds D / 32 channels.
template <int D>
__global__ void __launch_bounds__(256) k_kv16_simple(const __grid_constant__ Kv16Attn a)
{
    constexpr int C = D / 32;
    pdl_wait();
    pdl_trigger();
    const int lane = threadIdx.x & 31;
    const long long item = (long long)blockIdx.x * 8 + (threadIdx.x >> 5);
    if (item >= (long long)a.B * a.T * a.H) return;
    const int h = (int)(item % a.H), row = (int)(item / a.H), b = row / a.T, i = row - b * a.T, g = h / (a.H / a.Hkv);
    bool skip = false;
    int pre = -1, plen = 0;
    for (int p = lane; p < a.nP; p += 32) {
        const int lo = a.pfirst[p], hi = a.pfirst[p + 1];
        if (lo < 0 || hi > a.B || lo > hi) skip = true;
        if (lo <= b && b < hi) pre = p;
    }
    skip = __any_sync(0xffffffffu, skip);
    pre = __reduce_max_sync(0xffffffffu, pre);
    if (pre >= 0) plen = a.plens[pre];
    const int len = a.lens[b];
    if (plen > a.max_plen || len > a.max_len) skip = true;
    if (skip && lane == 0) kv4_raise(a.status, LA_ERR_ARG);
    if (skip || len < 0) return;
    float q[C], o[C] = {}, m = kNoRef, l = 0.f;
    for (int c = 0; c < C; c++) q[c] = __bfloat162float(a.q[(size_t)row * a.q_ld + (size_t)h * D + c * 32 + lane]) * a.sl2;
    auto key = [&](const __nv_bfloat16* k, const __nv_bfloat16* v) {
        float s = 0.f;
        for (int c = 0; c < C; c++) s += q[c] * __bfloat162float(k[c * 32 + lane]);
        s = warp_sum(s);
        const float top = fmaxf(m, s), f = exp2f(m - top), p = exp2f(s - top);
        m = top;
        l = l * f + p;
        for (int c = 0; c < C; c++) o[c] = o[c] * f + p * __bfloat162float(v[c * 32 + lane]);
    };
    auto cached = [&](const int* table, int n) {
        for (int t = 0; t < n; t++) {
            const int page = table[t >> a.page_log2];
            if ((unsigned)page >= (unsigned)a.n_pages) {
                if (lane == 0) kv4_raise(a.status, LA_ERR_ARG);
                continue;
            }
            const size_t at = ((((size_t)page * a.Hkv + g) << a.page_log2) + (t & ((1 << a.page_log2) - 1))) * D;
            key(a.kp + at, a.vp + at);
        }
    };
    if (plen > 0) cached(a.ptable + (size_t)pre * a.pp, plen);
    cached(a.table + (size_t)b * a.max_pages, len);
    for (int j = 0; j < a.T; j++)
        if (kv4_sees(i, j, a.W, a.n1)) {
            const size_t r = (size_t)b * a.T + j, at = (size_t)g * D;
            key(a.ks + r * a.k_ld + at, a.vs + r * a.v_ld + at);
        }
    for (int c = 0; c < C; c++) a.out[((size_t)row * a.H + h) * D + c * 32 + lane] = __float2bfloat16_rn(o[c] / l);
}

}  // namespace

size_t kv16_attn_bytes(const la_kv16_desc&, const la_kv16_attn&) { return 0; }

int launch_kv16_attn(cudaStream_t s, const la_kv16_desc& c, const la_kv16_attn& a)
{
    Kv16Attn k;
    k.q = (const __nv_bfloat16*)a.q, k.ks = (const __nv_bfloat16*)a.k_step, k.vs = (const __nv_bfloat16*)a.v_step;
    k.out = (__nv_bfloat16*)a.out;
    k.lens = a.lens, k.table = a.table, k.status = c.status;
    k.plens = a.prefix_lens, k.ptable = a.prefix_table, k.pfirst = a.prefix_first;
    k.kp = (const __nv_bfloat16*)c.k_pages, k.vp = (const __nv_bfloat16*)c.v_pages;
    k.B = a.batch, k.H = a.n_heads, k.Hkv = c.n_kv_heads;
    k.W = a.W, k.n1 = a.N - 1, k.T = 1 + (a.W + a.G) * k.n1;
    k.q_ld = a.q_ld, k.k_ld = a.k_ld, k.v_ld = a.v_ld;
    k.n_pages = c.n_pages, k.max_pages = c.max_pages, k.page_log2 = log2_of(c.page);
    auto bound = [](int given, int room) { return given > 0 && given < room ? given : room; };
    k.max_len = bound(a.max_len, c.max_pages * c.page);
    k.nP = a.n_prefix, k.pp = a.prefix_pages;
    k.max_plen = a.n_prefix ? bound(a.max_prefix_len, a.prefix_pages * c.page) : 0;
    k.sl2 = 1.4426950408889634f / sqrtf((float)c.head_dim);
    const long long items = (long long)k.B * k.T * k.H;
    const dim3 grid((unsigned)((items + 7) / 8));
    const cudaError_t e = c.head_dim == 128 ? launch_pdl(k_kv16_simple<128>, grid, dim3(256), 0, s, k)
                                            : launch_pdl(k_kv16_simple<64>, grid, dim3(256), 0, s, k);
    return e == cudaSuccess ? LA_OK : LA_ERR_CUDA;
}

}  // namespace la
