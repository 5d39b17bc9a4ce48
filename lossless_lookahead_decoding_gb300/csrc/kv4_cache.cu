// kv4_cache.cu -- the paged 4-bit KV cache's book-keeping and its tokens: page
// planning and release from the sequences' lengths, quantising tokens into
// pages, reading them back, and the C entry points of all of la_kv4_*.
#include <algorithm>
#include <climits>
#include <mutex>

#include "kv4.cuh"

namespace la {

namespace {

using namespace ptx;

// ------------------------------------------------------------------ plan ---
//
// Sequence b holds lens[b] tokens in ceil(lens / page) pages and gets n_new[b]
// more.  With f[b] new pages, F = exclusive sum of f and S = exclusive sum of
// n_new, its j-th new page is free_pages[n_free - 1 - F[b] - j] and its i-th
// new token, at position p = lens[b] + i, goes to slot
// page_of(p / page) * page + p % page.
//
// Latency bound: a few kilobytes in, the slots out.  So every CTA scans all
// sequences by itself (the lengths come out of L2) and keeps both sums in
// shared memory; no CTA waits for another.  Work is then split over slots,
// four neighbouring ones a thread (one search, one 16-byte store), and over
// new pages.  One CTA serves up to 16 K slots; beyond that one more for every 8 K.
// The new lengths are written by CTA 0 of the same launch when they go to
// buffers of their own; updated in place they are written by a second,
// one-CTA launch (kCommit) because other CTAs may still be reading them.

constexpr int kPlanThreads = 1024;
constexpr int kPlanMaxBatch = 8192;
enum PlanMode { kPlanAll, kPlanMap, kPlanCommit };

struct PlanArgs {
    const int *lens, *n_new, *free_pages, *n_free;
    int *table, *slots, *new_lens, *left, *status;
    int B, page_log2, max_pages, n_slots, stride, mode;
};

struct Scan2 {
    long long a, b;
};

__device__ __forceinline__ Scan2 block_scan2(Scan2 v, Scan2* total)
{
    // exclusive sums of both over the block, and their totals
    __shared__ Scan2 wsum[kPlanThreads / 32];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    Scan2 x = v;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const long long ya = __shfl_up_sync(0xffffffffu, x.a, o), yb = __shfl_up_sync(0xffffffffu, x.b, o);
        if (lane >= o) x.a += ya, x.b += yb;
    }
    if (lane == 31) wsum[warp] = x;
    __syncthreads();
    if (warp == 0) {
        Scan2 w = wsum[lane];
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const long long ya = __shfl_up_sync(0xffffffffu, w.a, o), yb = __shfl_up_sync(0xffffffffu, w.b, o);
            if (lane >= o) w.a += ya, w.b += yb;
        }
        wsum[lane] = w;
    }
    __syncthreads();
    *total = wsum[kPlanThreads / 32 - 1];
    const Scan2 before = warp ? wsum[warp - 1] : Scan2{0, 0};
    return Scan2{before.a + x.a - v.a, before.b + x.b - v.b};
}

// the last index whose entry of the ascending array is <= x
__device__ __forceinline__ int last_not_above(const int* a, int n, int x)
{
    int lo = 0, hi = n;  // a[lo] <= x < a[hi]
    while (hi - lo > 1) {
        const int m = (lo + hi) >> 1;
        if (a[m] <= x) lo = m;
        else hi = m;
    }
    return lo;
}

__global__ void __launch_bounds__(kPlanThreads) k_kv4_plan(PlanArgs a)
{
    extern __shared__ int plan_smem[];
    int *first_tok = plan_smem, *first_page = plan_smem + a.B;  // exclusive sums
    pdl_wait();
    pdl_trigger();
    const int n_free = *a.n_free, per = ceil_div(a.B, kPlanThreads), b0 = threadIdx.x * per;
    const int page = 1 << a.page_log2;
    const long long room = (long long)a.max_pages << a.page_log2;
    Scan2 mine{0, 0};
    int bad = n_free < 0 ? LA_ERR_ARG : 0;
    for (int b = b0; b < min(b0 + per, a.B); b++) {
        const int len = a.lens[b], n = len < 0 ? 0 : a.n_new[b];
        if (n < 0) bad = LA_ERR_ARG;
        else if (a.stride && n > a.stride) bad = LA_ERR_CAPACITY;
        else if ((long long)len + n > room) bad = LA_ERR_CAPACITY;
        else if (n > 0) {
            mine.a += n;
            mine.b += ((len + n + page - 1) >> a.page_log2) - ((len + page - 1) >> a.page_log2);
        }
    }
    Scan2 total;
    Scan2 at = block_scan2(mine, &total);
    if (!bad && ((!a.stride && total.a > a.n_slots) || total.b > n_free)) bad = LA_ERR_CAPACITY;
    const bool any_arg = __syncthreads_or(bad == LA_ERR_ARG), ok = !__syncthreads_or(bad != 0);
    if (!ok && blockIdx.x == 0 && threadIdx.x == 0 && a.mode != kPlanCommit)
        kv4_raise(a.status, any_arg ? LA_ERR_ARG : LA_ERR_CAPACITY);
    if (ok && a.mode != kPlanCommit) {
        for (int b = b0; b < min(b0 + per, a.B); b++) {
            first_tok[b] = (int)at.a;
            first_page[b] = (int)at.b;
            const int len = a.lens[b], n = len < 0 ? 0 : a.n_new[b];
            if (n > 0) {
                at.a += n;
                at.b += ((len + n + page - 1) >> a.page_log2) - ((len + page - 1) >> a.page_log2);
            }
        }
    }
    __syncthreads();
    const int tid = blockIdx.x * kPlanThreads + threadIdx.x, nthr = gridDim.x * kPlanThreads;
    if (a.mode != kPlanCommit) {
        // slots, four at a time
        const int live = ok ? (a.stride ? a.B * a.stride : (int)total.a) : 0;
        const bool wide = ((uintptr_t)a.slots & 15) == 0;
        for (int t0 = tid * 4; t0 < a.n_slots; t0 += nthr * 4) {
            int s[4] = {-1, -1, -1, -1};
            if (t0 < live) {
                int b = a.stride ? t0 / a.stride : last_not_above(first_tok, a.B, t0), seen = -1;
                int len = 0, n = 0, base = 0;
#pragma unroll
                for (int i = 0; i < 4; i++) {
                    const int t = t0 + i;
                    if (t >= live) break;
                    if (a.stride) b = t / a.stride;
                    else
                        while (b + 1 < a.B && first_tok[b + 1] <= t) b++;
                    if (b != seen) {
                        seen = b;
                        len = a.lens[b];
                        n = len < 0 ? 0 : a.n_new[b];
                        base = a.stride ? b * a.stride : first_tok[b];
                    }
                    if (t - base >= n) continue;
                    const int pos = len + (t - base), had = (len + page - 1) >> a.page_log2, j = pos >> a.page_log2;
                    const int pg = j < had ? a.table[(size_t)b * a.max_pages + j]
                                           : a.free_pages[n_free - 1 - first_page[b] - (j - had)];
                    s[i] = pg < 0 ? -1 : (pg << a.page_log2) + (pos & (page - 1));
                }
            }
            if (wide && t0 + 4 <= a.n_slots) {
                *(int4*)(a.slots + t0) = make_int4(s[0], s[1], s[2], s[3]);
            } else {
                for (int i = 0; i < 4 && t0 + i < a.n_slots; i++) a.slots[t0 + i] = s[i];
            }
        }
        // new pages into the block table
        if (ok)
            for (int f = tid; f < (int)total.b; f += nthr) {
                const int b = last_not_above(first_page, a.B, f);
                const int had = (a.lens[b] + page - 1) >> a.page_log2;
                a.table[(size_t)b * a.max_pages + had + (f - first_page[b])] = a.free_pages[n_free - 1 - f];
            }
    }
    if (a.mode == kPlanMap || blockIdx.x) return;
    if (a.mode == kPlanAll && gridDim.x == 1) __syncthreads();  // in place: every read above is done
    for (int b = threadIdx.x; b < a.B; b += kPlanThreads) {
        const int len = a.lens[b];
        a.new_lens[b] = ok && len >= 0 ? len + a.n_new[b] : len;
    }
    if (threadIdx.x == 0) *a.left = ok ? n_free - (int)total.b : n_free;
}

// --------------------------------------------------------------- release ---
//
// The pages of the sequences with done[b] != 0 go back onto the stack, b
// ascending and each sequence's pages in order; those sequences' lengths
// become 0.  One CTA: a scan, then one thread a page.

struct ReleaseArgs {
    const int *done, *table;
    int *lens, *free_pages, *n_free, *status;
    int B, page_log2, max_pages, n_pages;
};

__global__ void __launch_bounds__(kPlanThreads) k_kv4_release(ReleaseArgs a)
{
    extern __shared__ int plan_smem[];
    int* first_page = plan_smem;
    pdl_wait();
    pdl_trigger();
    const int n_free = *a.n_free, per = ceil_div(a.B, kPlanThreads), b0 = threadIdx.x * per;
    const int page = 1 << a.page_log2;
    Scan2 mine{0, 0};
    int bad = n_free < 0 ? 1 : 0;
    for (int b = b0; b < min(b0 + per, a.B); b++) {
        const int len = a.done[b] ? a.lens[b] : 0;
        const long long k = len > 0 ? ((long long)len + page - 1) >> a.page_log2 : 0;
        if (k > a.max_pages) bad = 1;
        mine.b += k;
    }
    Scan2 total;
    Scan2 at = block_scan2(mine, &total);
    if (total.b + n_free > a.n_pages) bad = 1;  // more pages than there are: one was given back twice
    if (__syncthreads_or(bad)) {
        if (threadIdx.x == 0) kv4_raise(a.status, LA_ERR_ARG);
        return;
    }
    for (int b = b0; b < min(b0 + per, a.B); b++) {
        first_page[b] = (int)at.b;
        const int len = a.done[b] ? a.lens[b] : 0;
        if (len > 0) at.b += ((long long)len + page - 1) >> a.page_log2;
    }
    __syncthreads();
    for (int f = threadIdx.x; f < (int)total.b; f += kPlanThreads) {
        const int b = last_not_above(first_page, a.B, f);
        a.free_pages[n_free + f] = a.table[(size_t)b * a.max_pages + (f - first_page[b])];
    }
    for (int b = threadIdx.x; b < a.B; b += kPlanThreads)
        if (a.done[b] && a.lens[b] > 0) a.lens[b] = 0;
    if (threadIdx.x == 0) *a.n_free = n_free + (int)total.b;
}

// ---------------------------------------------------------------- append ---
//
// One vector is quantised by D / 16 neighbouring lanes, 16 channels a lane,
// with four tokens (D = 128) or eight (D = 64) of the same head in a warp: a
// warp reads whole vectors, and writes the neighbouring 32-byte panel rows of
// consecutive slots.  K and V of a token are in flight together.
// HBM bound by design: one pass, extremes by packed max/min, no division per
// element.  The decisions are exact (the codes are those of exact
// arithmetic, whatever the inputs):
//  * s: 15 s against hi - lo with the rounding error of the subtraction;
//  * bf16 inputs: x / s is either a tie or at least 2^-10 away from one (both
//    have 8 significant bits and |x| >= s / 2 where a tie is near), so x * (1
//    / s), off by less than 2^-18, rounded to multiples of 2^-11 is a tie
//    exactly when x / s is;
//  * fp32 inputs: the residual x - k s is exact in one fused multiply-add
//    (12 bits in k s), and is compared with s / 2.

constexpr float kRound11 = 6144.f;       // 1.5 x 2^12: adding it rounds to multiples of 2^-11
constexpr float kRound0 = 12582912.f;    // 1.5 x 2^23: adding it rounds to whole numbers, ties to even

struct Quant {
    float s, inv;   // scale as the elements are compared with it, its reciprocal
    int z;
    uint32_t param;
    bool some;      // codes differ from z (s is neither 0 nor NaN)
    bool tiny;      // the elements are to be multiplied by 2^64
};

template <bool F32>
__device__ __forceinline__ int nearest(float x, float s, float inv)
{
    if (!F32) {
        const float t = (__fmul_rn(x, inv) + kRound11) - kRound11;
        return __float_as_int(t + kRound0) - 0x4B400000;
    }
    int k = __float_as_int(__fmul_rn(x, inv) + kRound0) - 0x4B400000;
    const float r = 2.f * __fmaf_rn(-(float)k, s, x);
    if (fabsf(r) > s || (fabsf(r) == s && (k & 1))) k += r > 0.f ? 1 : -1;
    return k;
}

// Scale, zero point and parameter word from the extremes (hi or lo NaN or
// infinite when the vector holds such a value).
template <bool F32>
__device__ __forceinline__ Quant quant_params(float hi, float lo)
{
    Quant q;
    hi = fmaxf(hi, 0.f) + (hi - hi);  // NaN and infinity stay
    lo = fminf(lo, 0.f) + (lo - lo);
    q.tiny = false;
    if (!(hi < INFINITY) || !(lo > -INFINITY)) {
        q.s = q.inv = 0.f;
        q.z = 0;
        q.param = 0x7fc00000u | 0x4300u;
        q.some = false;
        return q;
    }
    // the span of values near the type's end does not fit: take 2^-8 of both
    const bool huge = hi > 1e38f || lo < -1e38f;
    float h = hi, l = lo;
    if (huge) {
        h = fmaxf(h * 0x1p-8f, h > 0.f ? 0x1p-149f : 0.f);
        l = fminf(l * 0x1p-8f, l < 0.f ? -0x1p-149f : 0.f);
    }
    const float sp = h - l, bb = sp - h, err = (h - (sp - bb)) + (-l - bb);  // sp + err = h - l
    uint32_t c = __float_as_uint(__fdiv_rn(sp, 15.f)) & 0xffff0000u;
#pragma unroll
    for (int i = 0; i < 2; i++) {
        const float d = 15.f * __uint_as_float(c) - sp;  // exact: 12 bits, and near sp
        if (d < 0.f || (d == 0.f && err > 0.f)) c += 0x10000u;
    }
    float s = __uint_as_float(c);
    if (huge) s *= 256.f;
    q.some = s > 0.f;
    q.tiny = s < 0x1p-100f;
    const float s0 = s;
    if (q.tiny) s *= 0x1p64f, lo *= 0x1p64f;
    q.s = s;
    q.inv = q.some ? __frcp_rn(s) : 0.f;
    q.z = q.some ? nearest<F32>(-lo, s, q.inv) : 0;
    q.param = __float_as_uint(s0) | 0x4300u | (uint32_t)q.z;
    return q;
}

template <bool F32>
struct Elems {
    // 16 channels of one lane
    uint4 w[F32 ? 4 : 2];
    __device__ __forceinline__ void load(const void* p)
    {
        const uint4* s = (const uint4*)p;
#pragma unroll
        for (int i = 0; i < (F32 ? 4 : 2); i++) w[i] = __ldg(s + i);
    }
    __device__ __forceinline__ float at(int i) const
    {
        const uint32_t* u = (const uint32_t*)w;
        if (F32) return __uint_as_float(u[i]);
        return __uint_as_float(i & 1 ? u[i >> 1] & 0xffff0000u : u[i >> 1] << 16);
    }
    __device__ __forceinline__ void extremes(float& hi, float& lo) const
    {
        const uint32_t* u = (const uint32_t*)w;
        if (F32) {
            hi = lo = __uint_as_float(u[0]);
            bool bad = !(fabsf(hi) < INFINITY);
#pragma unroll
            for (int i = 1; i < 16; i++) {
                const float x = __uint_as_float(u[i]);
                hi = fmaxf(hi, x);
                lo = fminf(lo, x);
                bad |= !(fabsf(x) < INFINITY);
            }
            if (bad) hi = lo = __uint_as_float(0x7fc00000u);
        } else {
            __nv_bfloat162 h = *(const __nv_bfloat162*)&u[0], l = h;
#pragma unroll
            for (int i = 1; i < 8; i++) {
                const __nv_bfloat162 x = *(const __nv_bfloat162*)&u[i];
                h = __hmax2_nan(h, x);
                l = __hmin2_nan(l, x);
            }
            const float2 hf = __bfloat1622float2(h), lf = __bfloat1622float2(l);
            hi = fmaxf(hf.x, hf.y) + (hf.x - hf.x) + (hf.y - hf.y);
            lo = fminf(lf.x, lf.y) + (lf.x - lf.x) + (lf.y - lf.y);
        }
    }
};

template <bool F32>
__device__ __forceinline__ void quantise(const Elems<F32>& e, const Quant& q, uint32_t* word)
{
#pragma unroll
    for (int wd = 0; wd < 2; wd++) {
        uint32_t u = 0;
#pragma unroll
        for (int i = 0; i < 8; i++) {
            float x = e.at(wd * 8 + i);
            if (q.tiny) x *= 0x1p64f;
            const int c = __vimin_s32_relu(nearest<F32>(x, q.s, q.inv) + q.z, 15);
            u |= (uint32_t)c << (4 * (i >> 1) + 16 * (i & 1));
        }
        word[wd] = q.some ? u : 0u;  // s = 0 or NaN: every code 0
    }
}

struct AppendArgs {
    uint8_t* pages;
    const uint8_t *k, *v;
    const int *rows, *slots;
    int* status;
    long long row_bytes;
    int n, n_rows, Hkv, page_log2, blk_log2, n_slots;
};

template <int D, bool F32>
__global__ void __launch_bounds__(256) k_kv4_append(AppendArgs a)
{
    constexpr int L = D / 16, TOK = 32 / L;  // lanes of a vector, tokens of a warp
    constexpr int E = F32 ? 4 : 2;
    pdl_wait();
    pdl_trigger();
    const int lane = threadIdx.x & 31, sub = lane % L, grp = lane / L;
    const long long tasks = (long long)((a.n + TOK - 1) / TOK) * a.Hkv;
    for (long long task = (long long)blockIdx.x * 8 + (threadIdx.x >> 5); task < tasks; task += (long long)gridDim.x * 8) {
        const int h = (int)(task % a.Hkv), i = (int)(task / a.Hkv) * TOK + grp;
        int slot = -1, row = i;
        if (i < a.n) {
            slot = a.slots[i];
            if (a.rows) row = a.rows[i];
            if (slot >= a.n_slots || (slot >= 0 && (row < 0 || row >= a.n_rows))) {
                kv4_raise(a.status, LA_ERR_ARG);
                slot = -1;
            }
        }
        const bool live = slot >= 0;
        Elems<F32> e[2];
        if (live) {
            const size_t at = (size_t)row * a.row_bytes + ((size_t)h * D + sub * 16) * E;
            e[0].load(a.k + at);
            e[1].load(a.v + at);
        } else {
#pragma unroll
            for (int p = 0; p < 2; p++)
#pragma unroll
                for (int j = 0; j < (F32 ? 4 : 2); j++) e[p].w[j] = make_uint4(0, 0, 0, 0);
        }
        const int in_page = slot & ((1 << a.page_log2) - 1), tok = slot & 15;
        uint8_t* blk = a.pages + kv4_block_at(slot >> a.page_log2, h, in_page >> 4, a.Hkv, a.blk_log2, D);
#pragma unroll
        for (int p = 0; p < 2; p++) {
            float hi, lo;
            e[p].extremes(hi, lo);
#pragma unroll
            for (int o = 1; o < L; o <<= 1) {
                const float h2 = __shfl_xor_sync(0xffffffffu, hi, o), l2 = __shfl_xor_sync(0xffffffffu, lo, o);
                hi = fmaxf(hi, h2) + ((hi - hi) + (h2 - h2));
                lo = fminf(lo, l2) + ((lo - lo) + (l2 - l2));
            }
            const Quant q = quant_params<F32>(hi, lo);
            uint32_t w[2];
            quantise<F32>(e[p], q, w);
            if (live) {
                *(uint2*)(blk + p * 8 * D + (sub >> 2) * 512 + tok * 32 + (sub & 3) * 8) = make_uint2(w[0], w[1]);
                if (sub == 0) *(uint32_t*)(blk + 16 * D + p * 64 + tok * 4) = q.param;
            }
        }
    }
}

// ------------------------------------------------------------------ read ---
//
// The values (c - z) s of tokens, in fp32 (exact: 4 + 8 bits) or rounded to
// bf16.  The mirror image of append; HBM bound.

struct ReadArgs {
    const uint8_t* pages;
    uint8_t *k, *v;
    const int* slots;
    int* status;
    long long row_bytes;
    int n, Hkv, page_log2, blk_log2, n_slots;
};

template <int D, bool F32>
__global__ void __launch_bounds__(256) k_kv4_read(ReadArgs a)
{
    constexpr int L = D / 16, TOK = 32 / L, E = F32 ? 4 : 2;
    pdl_wait();
    pdl_trigger();
    const int lane = threadIdx.x & 31, sub = lane % L, grp = lane / L;
    const long long tasks = (long long)((a.n + TOK - 1) / TOK) * a.Hkv;
    for (long long task = (long long)blockIdx.x * 8 + (threadIdx.x >> 5); task < tasks; task += (long long)gridDim.x * 8) {
        const int h = (int)(task % a.Hkv), i = (int)(task / a.Hkv) * TOK + grp;
        if (i >= a.n) continue;
        const int slot = a.slots[i];
        if (slot < 0) continue;
        if (slot >= a.n_slots) {
            kv4_raise(a.status, LA_ERR_ARG);
            continue;
        }
        const int in_page = slot & ((1 << a.page_log2) - 1), tok = slot & 15;
        const uint8_t* blk = a.pages + kv4_block_at(slot >> a.page_log2, h, in_page >> 4, a.Hkv, a.blk_log2, D);
        uint2 w[2];
        uint32_t prm[2];
#pragma unroll
        for (int p = 0; p < 2; p++) {
            w[p] = *(const uint2*)(blk + p * 8 * D + (sub >> 2) * 512 + tok * 32 + (sub & 3) * 8);
            prm[p] = *(const uint32_t*)(blk + 16 * D + p * 64 + tok * 4);
        }
        const size_t at = (size_t)i * a.row_bytes + ((size_t)h * D + sub * 16) * E;
#pragma unroll
        for (int p = 0; p < 2; p++) {
            const float s = __uint_as_float(prm[p] & 0xffff0000u);
            const float z = __uint_as_float(prm[p] << 16);  // 128 + z
            float x[16];
#pragma unroll
            for (int c = 0; c < 16; c++) {
                const uint32_t u = c < 8 ? w[p].x : w[p].y;
                const uint32_t code = (u >> (4 * ((c & 7) >> 1) + 16 * (c & 1))) & 15u;
                // code into the mantissa of 128 (fp32: 2^16 per unit)
                x[c] = (__uint_as_float(0x43000000u | code << 16) - z) * s;
            }
            uint8_t* dst = (p ? a.v : a.k) + at;
            if (F32) {
#pragma unroll
                for (int j = 0; j < 4; j++)
                    *(float4*)(dst + 16 * j) = make_float4(x[4 * j], x[4 * j + 1], x[4 * j + 2], x[4 * j + 3]);
            } else {
                uint32_t y[8];
#pragma unroll
                for (int j = 0; j < 8; j++) {
                    __nv_bfloat162 b = __floats2bfloat162_rn(x[2 * j], x[2 * j + 1]);
                    y[j] = *(uint32_t*)&b;
                }
                *(uint4*)dst = make_uint4(y[0], y[1], y[2], y[3]);
                *(uint4*)(dst + 16) = make_uint4(y[4], y[5], y[6], y[7]);
            }
        }
    }
}

int log2_of(int x)
{
    int l = 0;
    while ((1 << l) < x) l++;
    return l;
}

// More shared memory than 48 KB for the large-batch plan, once per device.
std::mutex g_plan_mu;
bool g_plan_ready[256];

int plan_ready()
{
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 256) return LA_ERR_CUDA;
    std::lock_guard<std::mutex> lock(g_plan_mu);
    if (!g_plan_ready[dev]) {
        if (cudaFuncSetAttribute(k_kv4_plan, cudaFuncAttributeMaxDynamicSharedMemorySize, 2 * kPlanMaxBatch * 4) !=
            cudaSuccess)
            return LA_ERR_CUDA;
        g_plan_ready[dev] = true;
    }
    return LA_OK;
}

int done(cudaError_t e) { return e == cudaSuccess ? LA_OK : LA_ERR_CUDA; }

}  // namespace

int launch_kv4_plan(cudaStream_t s, const la_kv4_desc& c, const int* lens, const int* n_new, int B, const int* free_pages,
                    const int* n_free, int* table, int* slots, int n_slots, int stride, int* new_lens, int* left)
{
    if (int rc = plan_ready()) return rc;
    PlanArgs a{lens, n_new, free_pages, n_free, table, slots, new_lens, left, c.status, B, log2_of(c.page), c.max_pages,
               n_slots, stride, kPlanAll};
    const size_t smem = (size_t)B * 8;
    const int grid = n_slots <= 16384 ? 1 : (int)std::min(152LL, (n_slots + 8191LL) / 8192);
    const bool in_place = new_lens == lens || left == n_free;
    if (grid > 1 && in_place) a.mode = kPlanMap;
    cudaError_t e = launch_pdl(k_kv4_plan, dim3(grid), dim3(kPlanThreads), smem, s, a);
    if (e == cudaSuccess && a.mode == kPlanMap) {
        a.mode = kPlanCommit;
        e = launch_pdl(k_kv4_plan, dim3(1), dim3(kPlanThreads), smem, s, a);
    }
    return done(e);
}

int launch_kv4_release(cudaStream_t s, const la_kv4_desc& c, const int* done_, int B, int* lens, const int* table,
                       int* free_pages, int* n_free)
{
    ReleaseArgs a{done_, table, lens, free_pages, n_free, c.status, B, log2_of(c.page), c.max_pages, c.n_pages};
    return done(launch_pdl(k_kv4_release, dim3(1), dim3(kPlanThreads), (size_t)B * 4, s, a));
}

int launch_kv4_append(cudaStream_t s, const la_kv4_desc& c, const void* k, const void* v, int dtype, int ld, int n_rows,
                      const int* rows, const int* slots, int n)
{
    const bool f32 = dtype == LA_FP32;
    AppendArgs a{(uint8_t*)c.pages, (const uint8_t*)k, (const uint8_t*)v, rows, slots, c.status,
                 (long long)ld * (f32 ? 4 : 2), n, n_rows, c.n_kv_heads, log2_of(c.page), log2_of(c.page / 16),
                 c.n_pages * c.page};
    const int tok = 512 / c.head_dim;
    const long long tasks = (n + (long long)tok - 1) / tok * c.n_kv_heads;
    const dim3 grid((unsigned)std::min((tasks + 7) / 8, 152LL * 8));
    auto kern = c.head_dim == 128 ? (f32 ? k_kv4_append<128, true> : k_kv4_append<128, false>)
                                  : (f32 ? k_kv4_append<64, true> : k_kv4_append<64, false>);
    return done(launch_pdl(kern, grid, dim3(256), 0, s, a));
}

int launch_kv4_read(cudaStream_t s, const la_kv4_desc& c, const int* slots, int n, void* k, void* v, int dtype, int ld)
{
    const bool f32 = dtype == LA_FP32;
    ReadArgs a{(const uint8_t*)c.pages, (uint8_t*)k, (uint8_t*)v, slots, c.status, (long long)ld * (f32 ? 4 : 2), n,
               c.n_kv_heads, log2_of(c.page), log2_of(c.page / 16), c.n_pages * c.page};
    const int tok = 512 / c.head_dim;
    const long long tasks = (n + (long long)tok - 1) / tok * c.n_kv_heads;
    const dim3 grid((unsigned)std::min((tasks + 7) / 8, 152LL * 8));
    auto kern = c.head_dim == 128 ? (f32 ? k_kv4_read<128, true> : k_kv4_read<128, false>)
                                  : (f32 ? k_kv4_read<64, true> : k_kv4_read<64, false>);
    return done(launch_pdl(kern, grid, dim3(256), 0, s, a));
}

}  // namespace la

// -------------------------------------------------------------- C entries ---

using namespace la;

namespace {

bool desc_ok(const la_kv4_desc* c)
{
    if (!c || (c->head_dim != 64 && c->head_dim != 128) || c->n_kv_heads < 1 || c->n_kv_heads > 1024) return false;
    if (c->page != 16 && c->page != 32 && c->page != 64 && c->page != 128) return false;
    if (c->n_pages < 1 || (long long)c->n_pages * c->page >= (1LL << 31)) return false;
    return c->max_pages >= 1 && (long long)c->max_pages * c->page < (1LL << 31);
}

bool aligned(const void* p, int to) { return ((uintptr_t)p & (uintptr_t)(to - 1)) == 0; }

bool pool_ok(const la_kv4_desc* c) { return desc_ok(c) && c->pages && aligned(c->pages, 16) && aligned(c->status, 4); }

// do [a, a + n) and [b, b + n) of ints share memory
bool overlap(const int* a, const int* b, size_t n, size_t m) { return a < b + m && b < a + n; }

}  // namespace

extern "C" size_t la_kv4_page_bytes(const la_kv4_desc* c)
{
    if (!desc_ok(c)) return 0;
    return (size_t)c->n_kv_heads * (c->page / 16) * kv4_block_bytes(c->head_dim);
}

extern "C" int la_kv4_plan(const la_kv4_desc* c, const int32_t* lens, const int32_t* n_new, int batch,
                           const int32_t* free_pages, const int32_t* n_free, int32_t* table, int32_t* slots, int n_slots,
                           int slot_stride, int32_t* new_lens, int32_t* pages_left, void* stream)
{
    if (!desc_ok(c) || batch < 0 || batch > kPlanMaxBatch || n_slots < 0 || slot_stride < 0) return LA_ERR_ARG;
    if (!n_free || !pages_left || (batch && (!lens || !n_new || !free_pages || !table || !new_lens))) return LA_ERR_ARG;
    if (n_slots && !slots) return LA_ERR_ARG;
    if (slot_stride && (long long)batch * slot_stride != n_slots) return LA_ERR_ARG;
    // the lengths and the page count may be updated in place; anything else
    // written over something read is refused
    const size_t tab = (size_t)batch * c->max_pages;
    if ((new_lens != lens && overlap(new_lens, lens, batch, batch)) || overlap(new_lens, n_new, batch, batch)) return LA_ERR_ARG;
    if (overlap(slots, lens, n_slots, batch) || overlap(slots, n_new, n_slots, batch) || overlap(slots, table, n_slots, tab) ||
        overlap(slots, new_lens, n_slots, batch) || overlap(table, lens, tab, batch) || overlap(table, n_new, tab, batch) ||
        overlap(table, new_lens, tab, batch) || overlap(pages_left, lens, 1, batch) || overlap(pages_left, n_new, 1, batch) ||
        overlap(pages_left, new_lens, 1, batch) || overlap(pages_left, slots, 1, n_slots) || overlap(pages_left, table, 1, tab))
        return LA_ERR_ARG;
    return launch_kv4_plan((cudaStream_t)stream, *c, lens, n_new, batch, free_pages, n_free, table, slots, n_slots,
                           slot_stride, new_lens, pages_left);
}

extern "C" int la_kv4_release(const la_kv4_desc* c, const int32_t* done, int batch, int32_t* lens, const int32_t* table,
                              int32_t* free_pages, int32_t* n_free, void* stream)
{
    if (!desc_ok(c) || batch < 0 || batch > kPlanMaxBatch) return LA_ERR_ARG;
    if (batch == 0) return LA_OK;
    if (!done || !lens || !table || !free_pages || !n_free) return LA_ERR_ARG;
    return launch_kv4_release((cudaStream_t)stream, *c, done, batch, lens, table, free_pages, n_free);
}

extern "C" int la_kv4_append(const la_kv4_desc* c, const void* k, const void* v, int dtype, int ld, int n_rows,
                             const int32_t* rows, const int32_t* slots, int n, void* stream)
{
    if (!pool_ok(c) || n < 0 || n_rows < 0 || (dtype != LA_FP32 && dtype != LA_BF16)) return LA_ERR_ARG;
    if (n == 0) return LA_OK;
    if (!k || !v || !slots || !aligned(k, 16) || !aligned(v, 16)) return LA_ERR_ARG;
    if (ld < c->n_kv_heads * c->head_dim || (ld * (dtype == LA_FP32 ? 4LL : 2LL)) % 16) return LA_ERR_ARG;
    if (!rows && n > n_rows) return LA_ERR_ARG;
    return launch_kv4_append((cudaStream_t)stream, *c, k, v, dtype, ld, n_rows, rows, slots, n);
}

extern "C" int la_kv4_read(const la_kv4_desc* c, const int32_t* slots, int n, void* k, void* v, int dtype, int ld,
                           void* stream)
{
    if (!pool_ok(c) || n < 0 || (dtype != LA_FP32 && dtype != LA_BF16)) return LA_ERR_ARG;
    if (n == 0) return LA_OK;
    if (!k || !v || !slots || !aligned(k, 16) || !aligned(v, 16)) return LA_ERR_ARG;
    if (ld < c->n_kv_heads * c->head_dim || (ld * (dtype == LA_FP32 ? 4LL : 2LL)) % 16) return LA_ERR_ARG;
    return launch_kv4_read((cudaStream_t)stream, *c, slots, n, k, v, dtype, ld);
}

namespace {

// Shapes of an attention call (no pointers).
bool attn_shape_ok(const la_kv4_desc* c, const la_kv4_attn* a)
{
    if (!desc_ok(c) || !a || a->batch < 0 || a->batch > 65535) return false;
    if (a->n_heads < 1 || a->n_heads % c->n_kv_heads || a->n_heads > 16384) return false;
    if (a->W < 0 || a->G < 0 || a->N < 2 || a->N > 128 || a->W > 127 || a->G > 127) return false;
    return 1 + (a->W + a->G) * (a->N - 1) <= kRows && a->max_len >= 0;
}

}  // namespace

extern "C" size_t la_kv4_attention_bytes(const la_kv4_desc* c, const la_kv4_attn* a)
{
    return attn_shape_ok(c, a) ? kv4_attn_bytes(*c, *a) : 0;
}

extern "C" int la_kv4_attention(const la_kv4_desc* c, const la_kv4_attn* a, void* stream)
{
    if (!pool_ok(c) || !attn_shape_ok(c, a)) return LA_ERR_ARG;
    if (a->batch == 0) return LA_OK;
    if (!a->q || !a->k_step || !a->v_step || !a->out || !a->lens || !a->table) return LA_ERR_ARG;
    if (!aligned(a->q, 16) || !aligned(a->k_step, 16) || !aligned(a->v_step, 16) || !aligned(a->out, 16)) return LA_ERR_ARG;
    if (a->q_ld < a->n_heads * c->head_dim || a->q_ld % 8 || a->kv_ld < c->n_kv_heads * c->head_dim || a->kv_ld % 8)
        return LA_ERR_ARG;
    const size_t need = kv4_attn_bytes(*c, *a);
    if (need && (!a->workspace || !aligned(a->workspace, 16) || a->ws_bytes < need)) return LA_ERR_ARG;
    return launch_kv4_attn((cudaStream_t)stream, *c, *a);
}
