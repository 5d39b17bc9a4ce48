// kv16_cache.cu -- the paged bf16 KV cache: rows turned to their positions on
// the way into their slots (and to the step's attention), and the entry points
// of the cache.
//
// Rotation.  Pair i at position t turns by the angle t f_i.  f_i is held as a
// 64-bit fraction of a circle, u_i = f_i / (2 pi) 2^64: t u_i modulo 2^64 is
// the exact angle of u_i modulo a circle, one 64-bit product whatever t is,
// where t f_i in fp32 would be off by 2^-24 t radians (0.06 at a million).
// Its upper 32 bits, in half circles, go to sincospi in fp32: an angle within
// 2^-24 pi of t times u_i's frequency, which is f_i to a double's precision.  y = x cos - x' sin and x' cos + x sin in fp32,
// one rounding to bf16.
#include <math.h>

#include <algorithm>

#include "kv16.cuh"

namespace la {
namespace {

constexpr int kThreads = 256;
constexpr int kMaxTokens = 8;  // tokens of a CTA

struct Turns {
    uint64_t u[64];
};

struct AppendArgs {
    const uint8_t *q, *k, *v;
    __nv_bfloat16 *q_out, *k_out, *kp, *vp;
    const int *rows, *slots, *pos;
    int* status;
    long long q_ld, k_ld, v_ld, qo_ld, ko_ld;  // bytes of a row
    int n, n_rows, H, Hkv, page_log2, n_slots;
    int heads;             // queries', keys' and values' heads that the call moves
    int share;             // heads of a CTA
    int tokens;            // tokens of a CTA
    uint32_t inv_share;    // ceil(2^32 / share) modulo 2^32: 0 for a single head
    int rot, neighbours;   // rot 0: nothing turns
    Turns t;
};

__device__ __forceinline__ uint32_t pack2(float lo, float hi)
{
    __nv_bfloat162 v = __floats2bfloat162_rn(lo, hi);
    return *reinterpret_cast<uint32_t*>(&v);
}

// Eight channels as fp32.
template <bool F32>
struct Piece {
    uint4 w[F32 ? 2 : 1];
    __device__ __forceinline__ void load(const uint8_t* p)
    {
#pragma unroll
        for (int i = 0; i < (F32 ? 2 : 1); i++) w[i] = ((const uint4*)p)[i];  // (in place: no read-only load)
    }
    __device__ __forceinline__ void get(float (&x)[8]) const
    {
        const uint32_t* u = (const uint32_t*)w;
#pragma unroll
        for (int i = 0; i < 8; i++)
            x[i] = F32 ? __uint_as_float(u[i & (F32 ? 7 : 3)]) : __uint_as_float((i & 1) ? u[i >> 1 & 3] & 0xffff0000u : u[i >> 1 & 3] << 16);
    }
};

__device__ __forceinline__ uint4 pack8(const float (&x)[8])
{
    return make_uint4(pack2(x[0], x[1]), pack2(x[2], x[3]), pack2(x[4], x[5]), pack2(x[6], x[7]));
}

// A CTA: a.tokens tokens x a.share heads.  The tokens' sines and cosines go to
// shared memory once; then a thread takes 2 x 8 channels of a head at a time,
// those that turn together.  HBM bound for many tokens: 18 441 of 64 + 8 + 8 heads
// (793 MB) 127 us, 6.25 TB/s; for few, the launch: 228 rows of 32 heads 3.9 us.
// Measured for the former: 2, 4, 8 and 16 tokens a CTA 134.6, 128.6, 127.3, 127.8 us.
template <int D, bool F32>
__global__ void __launch_bounds__(kThreads) k_kv16_append(const __grid_constant__ AppendArgs a)
{
    constexpr int E = F32 ? 4 : 2, kUnits = D / 16;
    __shared__ float2 cs[kMaxTokens][D / 2];
    __shared__ int s_row[kMaxTokens], s_slot[kMaxTokens];
    pdl_wait();
    pdl_trigger();
    const int i0 = blockIdx.x * a.tokens, h0 = blockIdx.y * a.share;
    const int tokens = min(a.tokens, a.n - i0), half = a.rot / 2;
    if ((int)threadIdx.x < tokens) {
        const int i = i0 + threadIdx.x;
        int row = a.rows ? a.rows[i] : i, slot = a.slots ? a.slots[i] : -1;
        if ((unsigned)row >= (unsigned)a.n_rows || slot >= a.n_slots) {
            kv4_raise(a.status, LA_ERR_ARG);
            row = -1;
        }
        s_row[threadIdx.x] = row, s_slot[threadIdx.x] = slot;
    }
    for (int j = threadIdx.x; j < tokens * (D / 2); j += kThreads) {
        const int t = j / (D / 2), i = j % (D / 2);
        if (i >= half) continue;
        const uint64_t at = (uint64_t)(int64_t)a.pos[i0 + t] * a.t.u[i];
        float s, c;
        sincospif((float)(int32_t)(at >> 32) * 0x1p-31f, &s, &c);
        cs[t][i] = make_float2(c, s);
    }
    __syncthreads();
    const int share = min(a.share, a.heads - h0), nq = a.q_out ? a.H : 0, all = tokens * a.share * kUnits;
    // A unit's two pieces: partners half a rotation apart, or next to each other.
    struct Unit {
        int t, h, what, p0, p1, slot;  // token, head, 0 query, 1 key, 2 value; pieces; slot
        bool live, turns, apart;
        Piece<F32> x0, x1;
    };
    auto fetch = [&](int j, Unit& n) {
        const int item = j / kUnits, u = j % kUnits, t = a.inv_share ? __umulhi((uint32_t)item, a.inv_share) : item, hh = item - t * a.share;
        n.live = false;
        if (j >= all || hh >= share) return;
        const int row = s_row[t], h = h0 + hh;
        n.t = t, n.slot = s_slot[t];
        n.what = h < nq ? 0 : h < nq + a.Hkv ? 1 : 2;
        n.h = h - (n.what == 0 ? 0 : n.what == 1 ? nq : nq + a.Hkv);
        n.live = row >= 0 && !(n.slot < 0 && (n.what == 2 || (n.what == 1 && !a.k_out)));
        if (!n.live) return;
        n.turns = n.what < 2 && 16 * u < a.rot, n.apart = 16 * u < a.rot && !a.neighbours;
        n.p0 = n.apart ? u : 2 * u, n.p1 = n.apart ? u + a.rot / 16 : 2 * u + 1;
        const uint8_t* src = n.what == 0 ? a.q + row * a.q_ld : n.what == 1 ? a.k + row * a.k_ld : a.v + row * a.v_ld;
        src += (size_t)n.h * D * E;
        n.x0.load(src + n.p0 * 8 * E);
        n.x1.load(src + n.p1 * 8 * E);
    };
    auto put = [&](int j, const Unit& n) {
        if (!n.live) return;
        const int u = j % kUnits;
        uint4 y0, y1;
        if (n.turns || F32) {
            float a0[8], a1[8];
            n.x0.get(a0), n.x1.get(a1);
            if (n.turns) {
                const float2* w = cs[n.t] + 8 * u;
                if (n.apart) {
#pragma unroll
                    for (int i = 0; i < 8; i++) {
                        const float2 r = w[i];
                        const float lo = a0[i] * r.x - a1[i] * r.y;
                        a1[i] = a1[i] * r.x + a0[i] * r.y;
                        a0[i] = lo;
                    }
                } else {
#pragma unroll
                    for (int i = 0; i < 8; i += 2) {
                        const float2 r = w[i / 2], s = w[4 + i / 2];
                        float lo = a0[i] * r.x - a0[i + 1] * r.y;
                        a0[i + 1] = a0[i + 1] * r.x + a0[i] * r.y;
                        a0[i] = lo;
                        lo = a1[i] * s.x - a1[i + 1] * s.y;
                        a1[i + 1] = a1[i + 1] * s.x + a1[i] * s.y;
                        a1[i] = lo;
                    }
                }
            }
            y0 = pack8(a0), y1 = pack8(a1);
        } else {
            y0 = n.x0.w[0], y1 = n.x1.w[0];
        }
        const int i = i0 + n.t;
        if (n.what == 0) {
            uint4* o = (uint4*)((uint8_t*)a.q_out + (long long)i * a.qo_ld) + (size_t)n.h * (D / 8);
            o[n.p0] = y0, o[n.p1] = y1;
            return;
        }
        if (n.what == 1 && a.k_out) {
            uint4* o = (uint4*)((uint8_t*)a.k_out + (long long)i * a.ko_ld) + (size_t)n.h * (D / 8);
            o[n.p0] = y0, o[n.p1] = y1;
        }
        if (n.slot >= 0) {
            const size_t at = ((((size_t)(n.slot >> a.page_log2) * a.Hkv + n.h) << a.page_log2) + (n.slot & ((1 << a.page_log2) - 1))) * D;
            uint4* o = (uint4*)((n.what == 1 ? a.kp : a.vp) + at);
            o[n.p0] = y0, o[n.p1] = y1;
        }
    };
    // kAhead units of a thread on their way at once (1, 2, 4: 138.6, 126.8, 147 us; fp32's are twice as long).  (In
    // place: a unit writes only what it has read itself.)
    constexpr int kAhead = F32 ? 1 : 2;
#pragma unroll 1
    for (int j = threadIdx.x; j < all; j += kAhead * kThreads) {
        Unit n[kAhead];
#pragma unroll
        for (int k = 0; k < kAhead; k++) fetch(j + k * kThreads, n[k]);
#pragma unroll
        for (int k = 0; k < kAhead; k++) put(j + k * kThreads, n[k]);
    }
}

// Do two sets of rows share memory?  Rows of equal stride (views of one matrix)
// may lie between each other's.
struct Rows {
    uintptr_t at;
    size_t ld, width, n;  // bytes; rows
    size_t span() const { return n ? (n - 1) * ld + width : 0; }
};

bool share_memory(const Rows& a, const Rows& b)
{
    if (!a.at || !b.at || !a.n || !b.n || a.at >= b.at + b.span() || b.at >= a.at + a.span()) return false;
    if (a.ld != b.ld || a.n < 2 || b.n < 2) return true;
    const size_t off = b.at >= a.at ? (b.at - a.at) % a.ld : (a.ld - (a.at - b.at) % a.ld) % a.ld;
    return off < a.width || off + b.width > a.ld;
}

int launch_append(cudaStream_t s, const la_kv16_desc& c, const la_kv16_rows& r)
{
    const bool f32 = r.dtype == LA_FP32;
    const int E = f32 ? 4 : 2;
    AppendArgs a = {};
    a.q = (const uint8_t*)r.q, a.k = (const uint8_t*)r.k, a.v = (const uint8_t*)r.v;
    a.q_out = (__nv_bfloat16*)r.q_out, a.k_out = (__nv_bfloat16*)r.k_out;
    a.kp = (__nv_bfloat16*)c.k_pages, a.vp = (__nv_bfloat16*)c.v_pages;
    a.rows = r.rows, a.slots = r.slots, a.pos = r.positions, a.status = c.status;
    a.q_ld = (long long)r.q_ld * E, a.k_ld = (long long)r.k_ld * E, a.v_ld = (long long)r.v_ld * E;
    a.qo_ld = (long long)r.q_out_ld * 2, a.ko_ld = (long long)r.k_out_ld * 2;
    a.n = r.n, a.n_rows = r.n_rows, a.H = r.n_heads, a.Hkv = c.n_kv_heads;
    a.page_log2 = log2_of(c.page), a.n_slots = c.n_pages * c.page;
    a.heads = (r.q_out ? r.n_heads : 0) + (r.slots ? 2 : r.k_out ? 1 : 0) * c.n_kv_heads;
    if (r.rope) {
        a.rot = r.rope->rot_dim, a.neighbours = r.rope->neighbours;
        for (int i = 0; i < a.rot / 2; i++) a.t.u[i] = r.rope->turn[i];
    }
    // Few tokens: many small CTAs, at least a thread for each unit; many: fewer sines for each head.
    const int units = c.head_dim / 16, least = kThreads / units;  // heads for a unit a thread
    a.tokens = 1, a.share = std::min(a.heads, least);
    const long long ctas = (long long)r.n * ((a.heads + a.share - 1) / a.share);
    if (ctas > 8 * 152) {
        a.tokens = kMaxTokens;
        a.share = a.heads;
    }
    while (a.share > 1024) a.share = (a.share + 1) / 2;
    a.inv_share = (uint32_t)(((1ull << 32) + a.share - 1) / a.share);
    auto kern = c.head_dim == 128 ? (f32 ? k_kv16_append<128, true> : k_kv16_append<128, false>)
                                  : (f32 ? k_kv16_append<64, true> : k_kv16_append<64, false>);
    const dim3 grid((unsigned)((r.n + a.tokens - 1) / a.tokens), (unsigned)((a.heads + a.share - 1) / a.share));
    return launch_pdl(kern, grid, dim3(kThreads), 0, s, a) == cudaSuccess ? LA_OK : LA_ERR_CUDA;
}

}  // namespace

bool kv16_desc_ok(const la_kv16_desc* c)
{
    if (!c || (c->head_dim != 64 && c->head_dim != 128) || c->n_kv_heads < 1 || c->n_kv_heads > 1024) return false;
    if (c->page != 16 && c->page != 32 && c->page != 64 && c->page != 128) return false;
    if (c->n_pages < 1 || (long long)c->n_pages * c->page >= (1LL << 31)) return false;
    return c->max_pages >= 1 && (long long)c->max_pages * c->page <= (1LL << 30);
}

bool kv16_pool_ok(const la_kv16_desc* c)
{
    return kv16_desc_ok(c) && c->k_pages && c->v_pages && aligned(c->k_pages, 16) && aligned(c->v_pages, 16) && aligned(c->status, 4);
}

}  // namespace la

// -------------------------------------------------------------- C entries ---

using namespace la;

extern "C" size_t la_kv16_page_bytes(const la_kv16_desc* c)
{
    return kv16_desc_ok(c) ? (size_t)c->n_kv_heads * c->page * c->head_dim * 2 : 0;
}

extern "C" int la_rope_init(la_rope* r, int rot_dim, int neighbours, double theta, const double* freq)
{
    if (!r || rot_dim < 16 || rot_dim > 128 || rot_dim % 16 || (neighbours != 0 && neighbours != 1)) return LA_ERR_ARG;
    if (!freq && !(theta > 0 && std::isfinite(theta))) return LA_ERR_ARG;
    la_rope t = {};
    t.rot_dim = rot_dim, t.neighbours = neighbours;
    for (int i = 0; i < rot_dim / 2; i++) {
        const double f = freq ? freq[i] : pow(theta, -2.0 * i / rot_dim);
        if (!(fabs(f) <= 0x1p20)) return LA_ERR_ARG;
        // of a circle: the fraction, in units of 2^-64 (a double has 53 bits of it)
        const double part = f / (2 * M_PI), frac = part - floor(part);
        t.turn[i] = frac >= 1.0 ? 0 : (uint64_t)ldexp(frac, 64);
    }
    *r = t;
    return LA_OK;
}

extern "C" int la_kv16_append(const la_kv16_desc* c, const la_kv16_rows* r, void* stream)
{
    if (!kv16_pool_ok(c) || !r || r->n < 0 || r->n_rows < 0 || (r->dtype != LA_FP32 && r->dtype != LA_BF16)) return LA_ERR_ARG;
    const bool keys = r->slots || r->k_out;
    if (r->q_out && (!r->q || r->n_heads < 1 || r->n_heads > 16384)) return LA_ERR_ARG;
    if (r->rope) {
        const int rot = r->rope->rot_dim;
        if (rot < 16 || rot > c->head_dim || rot % 16 || (r->rope->neighbours != 0 && r->rope->neighbours != 1)) return LA_ERR_ARG;
    }
    if (r->n == 0 || (!keys && !r->q_out)) return LA_OK;
    if ((keys && !r->k) || (r->slots && !r->v) || (r->rope && !r->positions)) return LA_ERR_ARG;
    if (!ints_aligned(r->rows, r->slots, r->positions)) return LA_ERR_ARG;
    if (!r->rows && r->n > r->n_rows) return LA_ERR_ARG;
    const int kv_width = c->n_kv_heads * c->head_dim, q_width = r->q_out ? r->n_heads * c->head_dim : 0;
    const size_t E = r->dtype == LA_FP32 ? 4 : 2;
    if (keys && (!aligned(r->k, 16) || r->k_ld < kv_width || r->k_ld * E % 16)) return LA_ERR_ARG;
    if (r->slots && (!aligned(r->v, 16) || r->v_ld < kv_width || r->v_ld * E % 16)) return LA_ERR_ARG;
    if (r->k_out && (!aligned(r->k_out, 16) || r->k_out_ld < kv_width || r->k_out_ld % 8)) return LA_ERR_ARG;
    if (r->q_out && (!aligned(r->q, 16) || !aligned(r->q_out, 16) || r->q_ld < q_width || r->q_out_ld < q_width || r->q_ld * E % 16 ||
                     r->q_out_ld % 8))
        return LA_ERR_ARG;
    // what is written may share memory with nothing but its own input, in place
    const size_t n = r->n, n_rows = r->n_rows, pool = c->n_pages * la_kv16_page_bytes(c);
    auto rows_of = [](const void* p, size_t ld, size_t width, size_t rows) { return Rows{(uintptr_t)p, ld, width, rows}; };
    const Rows q = rows_of(r->q_out ? r->q : nullptr, r->q_ld * E, q_width * E, n_rows), k = rows_of(keys ? r->k : nullptr, r->k_ld * E, kv_width * E, n_rows),
               v = rows_of(r->slots ? r->v : nullptr, r->v_ld * E, kv_width * E, n_rows);
    const Rows qo = rows_of(r->q_out, r->q_out_ld * 2ull, q_width * 2ull, n), ko = rows_of(r->k_out, r->k_out_ld * 2ull, kv_width * 2ull, n);
    const Rows kp = rows_of(r->slots ? c->k_pages : nullptr, pool, pool, 1), vp = rows_of(r->slots ? c->v_pages : nullptr, pool, pool, 1);
    const Rows idx[4] = {rows_of(r->rows, 4 * n, 4 * n, 1), rows_of(r->slots, 4 * n, 4 * n, 1),
                         rows_of(r->rope ? r->positions : nullptr, 4 * n, 4 * n, 1), rows_of(c->status, 4, 4, 1)};
    auto in_place = [&](const Rows& in, const Rows& o) {
        return E == 2 && !r->rows && in.at == o.at && (in.ld == o.ld || (n == 1 && n_rows == 1));
    };
    if ((share_memory(q, qo) && !in_place(q, qo)) || (share_memory(k, ko) && !in_place(k, ko))) return LA_ERR_ARG;
    if (share_memory(qo, k) || share_memory(qo, v) || share_memory(ko, q) || share_memory(ko, v) || share_memory(qo, ko)) return LA_ERR_ARG;
    for (const Rows* p : {&kp, &vp})
        for (const Rows* x : {&q, &k, &v, &qo, &ko})
            if (share_memory(*p, *x)) return LA_ERR_ARG;
    if (share_memory(kp, vp)) return LA_ERR_ARG;
    for (const Rows& i : idx)
        for (const Rows* x : {&qo, &ko, &kp, &vp})
            if (share_memory(i, *x)) return LA_ERR_ARG;
    return launch_append((cudaStream_t)stream, *c, *r);
}

namespace {

// Shapes of an attention call (no pointers).
bool attn_shape_ok(const la_kv16_desc* c, const la_kv16_attn* a)
{
    if (!kv16_desc_ok(c) || !a || a->batch < 0 || a->batch > 8192) return false;
    if (a->n_heads < 1 || a->n_heads % c->n_kv_heads || a->n_heads > 16384 || a->n_heads / c->n_kv_heads > 128) return false;
    if (a->W < 0 || a->G < 0 || a->N < 2 || a->N > 128 || a->W > 127 || a->G > 127) return false;
    if (1 + (a->W + a->G) * (a->N - 1) > kRows || a->max_len < 0) return false;
    if (a->n_prefix < 0 || a->n_prefix > 8192 || a->max_prefix_len < 0) return false;
    return a->n_prefix == 0 || (a->prefix_pages >= 1 && (long long)a->prefix_pages * c->page <= (1LL << 30));
}

}  // namespace

extern "C" size_t la_kv16_attention_bytes(const la_kv16_desc* c, const la_kv16_attn* a)
{
    return attn_shape_ok(c, a) && a->batch ? kv16_attn_bytes(*c, *a) : 0;
}

extern "C" int la_kv16_attention(const la_kv16_desc* c, const la_kv16_attn* a, void* stream)
{
    if (!kv16_pool_ok(c) || !attn_shape_ok(c, a)) return LA_ERR_ARG;
    if (a->batch == 0) return LA_OK;
    if (!a->q || !a->k_step || !a->v_step || !a->out || !a->lens || !a->table) return LA_ERR_ARG;
    if (a->n_prefix && (!a->prefix_lens || !a->prefix_table || !a->prefix_first)) return LA_ERR_ARG;
    if (!ints_aligned(a->lens, a->table)) return LA_ERR_ARG;
    if (a->n_prefix && !ints_aligned(a->prefix_lens, a->prefix_table, a->prefix_first)) return LA_ERR_ARG;
    if (!aligned(a->q, 16) || !aligned(a->k_step, 16) || !aligned(a->v_step, 16) || !aligned(a->out, 16)) return LA_ERR_ARG;
    const int kv_width = c->n_kv_heads * c->head_dim;
    if (a->q_ld < a->n_heads * c->head_dim || a->q_ld % 8 || a->k_ld < kv_width || a->k_ld % 8 || a->v_ld < kv_width || a->v_ld % 8)
        return LA_ERR_ARG;
    const size_t need = kv16_attn_bytes(*c, *a);
    if (need && (!a->workspace || !aligned(a->workspace, 16) || a->ws_bytes < need)) return LA_ERR_ARG;
    return launch_kv16_attn((cudaStream_t)stream, *c, *a);
}
