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
// eight neighbouring ones a thread, and over new pages.  One CTA serves up to
// 16 K slots; beyond that one more for every 8 K.
// The new lengths are written by CTA 0 of the same launch when they go to
// buffers of their own; updated in place they are written by a second,
// one-CTA launch (kCommit) because other CTAs may still be reading them.
// 1024 sequences of up to 5 tokens (8192 slots): 5.5 us in a graph; 512 prompts of
// 1 M tokens (126 CTAs): 6.6 us in a graph on the same inputs, 9 us on new ones, and
// 9 us in place.  The launch and two trips to memory take 3.5 us of either.

constexpr int kPlanThreads = 1024;
constexpr int kPlanMaxBatch = 8192;
constexpr int kPlanPer = 8;  // slots a thread: one search, whole 16-byte stores
enum PlanMode { kPlanAll, kPlanMap, kPlanCommit };

struct PlanArgs {
    const int *lens, *n_new, *free_pages, *n_free;
    int *table, *slots, *new_lens, *left, *status;
    int B, page_log2, max_pages, n_pages, n_slots, stride, mode;
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
    const bool any_arg = __syncthreads_or(bad == LA_ERR_ARG), any = __syncthreads_or(bad != 0);
    const bool ok = !any && n_free <= a.n_pages;  // (a higher stack than there are pages is not read)
    if (!ok && blockIdx.x == 0 && threadIdx.x == 0 && a.mode != kPlanCommit)
        kv4_raise(a.status, any_arg || !any ? LA_ERR_ARG : LA_ERR_CAPACITY);
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
        // slots, eight at a time, in runs of neighbours: tokens of one sequence and page,
        // or places that no token takes
        const int live = ok ? (a.stride ? a.B * a.stride : (int)total.a) : 0;
        const bool wide = ((uintptr_t)a.slots & 15) == 0;
        for (long long at0 = (long long)tid * kPlanPer; at0 < a.n_slots; at0 += (long long)nthr * kPlanPer) {
            const int t0 = (int)at0, t1 = min(a.n_slots - t0, kPlanPer);
            int s[kPlanPer];
#pragma unroll
            for (int i = 0; i < kPlanPer; i++) s[i] = -1;
            int b = t0 >= live ? 0 : a.stride ? t0 / a.stride : last_not_above(first_tok, a.B, t0);
#pragma unroll 1
            for (int i0 = 0; i0 < t1 && t0 + i0 < live;) {
                const int len = a.lens[b], n = len < 0 ? 0 : a.n_new[b];
                const int off = t0 + i0 - (a.stride ? b * a.stride : first_tok[b]);
                int run = a.stride - off, slot = -1;  // to the sequence's end
                if (off < n) {
                    const int pos = len + off, had = (len + page - 1) >> a.page_log2, j = pos >> a.page_log2;
                    const int pg = j < had ? a.table[(size_t)b * a.max_pages + j]
                                           : a.free_pages[n_free - 1 - first_page[b] - (j - had)];
                    if ((unsigned)pg < (unsigned)a.n_pages) slot = (pg << a.page_log2) + (pos & (page - 1));
                    else kv4_raise(a.status, LA_ERR_ARG);
                    run = min(page - (pos & (page - 1)), n - off);
                }
                const int i1 = i0 + min(run, kPlanPer - i0);
#pragma unroll
                for (int i = 0; i < kPlanPer; i++)
                    if (i >= i0 && i < i1 && slot >= 0) s[i] = slot + (i - i0);
                i0 = i1;
                if (a.stride) b += off + run == a.stride;
                else
                    while (b + 1 < a.B && first_tok[b + 1] <= t0 + i0) b++;
            }
            if (wide && t1 == kPlanPer) {
#pragma unroll
                for (int i = 0; i < kPlanPer; i += 4) *(int4*)(a.slots + t0 + i) = make_int4(s[i], s[i + 1], s[i + 2], s[i + 3]);
            } else {
#pragma unroll
                for (int i = 0; i < kPlanPer; i++)
                    if (i < t1) a.slots[t0 + i] = s[i];
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
// become 0.  One CTA: a scan, then one thread a page: 8 sequences of 20 pages 2.6 us,
// 1024 of 64 (65 536 pages, a search for each) 48 us.

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
// consecutive slots.  K and V of a token are in flight together, and even
// lanes work out K's parameters while odd ones work out V's.
// HBM bound by design: one pass, extremes by packed max/min, and 3.5
// instructions an element for the codes: they stay in pairs, the way the
// format keeps them (channel 2i in bits 4i, 2i + 1 in bits 16 + 4i).
// 18 K tokens of 8 heads, D = 128: bf16 14.7 us (96 MB: 14.1 us at a plain copy's
// rate; integer pipe 70 % busy), fp32 29.9 us (171 MB: 25.2).
// The decisions are exact (the codes are those of exact
// arithmetic, whatever the inputs):
//  * s: 15 s against hi - lo with the rounding error of the subtraction;
//  * bf16 inputs: x / s is either a tie or at least 2^-10 away from one (both
//    have 8 significant bits and |x| >= s / 2 where a tie is near), so x * (1
//    / s), off by less than 2^-17, rounded to multiples of 2^-11 is a tie
//    exactly when x / s is;
//  * fp32 inputs: x (1 / s) decides where it is further than 2^-17 from a tie;
//    for a lane that holds another, the residual x - k s, exact in one fused
//    multiply-add (12 bits in k s), is compared with s / 2.

constexpr float kRound11 = 6144.f;       // 1.5 x 2^12: adding it rounds to multiples of 2^-11
constexpr float kRound0 = 12582912.f;    // 1.5 x 2^23: adding it rounds to whole numbers, ties to even; its bits' lower half is 0
constexpr uint32_t kKvNan = 0x7fc04300u; // the parameter word of a vector with a NaN or an infinity

template <bool F32>
__device__ __forceinline__ int nearest(float x, float s, float inv)
{
    if (!F32) return __float_as_int(__fadd_rn(__fmaf_rn(x, inv, kRound11), kRound0 - kRound11)) - 0x4B400000;
    int k = __float_as_int(__fmul_rn(x, inv) + kRound0) - 0x4B400000;
    const float r = 2.f * __fmaf_rn(-(float)k, s, x);
    if (fabsf(r) > s || (fabsf(r) == s && (k & 1))) k += r > 0.f ? 1 : -1;
    return k;
}

__device__ __forceinline__ float scale_of(uint32_t param) { return __uint_as_float(param & 0xffff0000u); }
// scales below this are compared with elements times 2^64 (their reciprocals would not fit)
__device__ __forceinline__ bool tiny_scale(float s) { return s < 0x1p-100f; }

// Parameter word and reciprocal of the scale from the extremes hi = max x and
// nlo = -min x (NaN or infinite when the vector holds such a value).
template <bool F32>
__device__ __forceinline__ uint32_t quant_params(float hi, float nlo, float* inv)
{
    *inv = 0.f;
    if (!(hi < INFINITY) || !(nlo < INFINITY)) return kKvNan;
    hi = fmaxf(hi, 0.f);
    nlo = fmaxf(nlo, 0.f);
    // the span of values near the type's end does not fit: take 2^-8 of both
    const bool huge = fmaxf(hi, nlo) > 1e38f;
    float h = hi, l = nlo;
    if (huge) {
        h = fmaxf(h * 0x1p-8f, h > 0.f ? 0x1p-149f : 0.f);
        l = fmaxf(l * 0x1p-8f, l > 0.f ? 0x1p-149f : 0.f);
    }
    const float sp = h + l, bb = sp - h, err = (h - (sp - bb)) + (l - bb);  // sp + err = h + l
    // sp / 15 to within an ulp; cut to bf16 it is at most two steps low and never high
    uint32_t c = __float_as_uint(sp * (1.f / 15.f)) & 0xffff0000u;
#pragma unroll
    for (int i = 0; i < 2; i++) {
        const float d = 15.f * __uint_as_float(c) - sp;  // exact: 12 bits, and near sp
        if (d < 0.f || (d == 0.f && err > 0.f)) c += 0x10000u;
    }
    float s = __uint_as_float(c);
    if (huge) s *= 256.f;
    c = __float_as_uint(s);
    if (c == 0) return 0x4300u;
    if (tiny_scale(s)) s *= 0x1p64f, nlo *= 0x1p64f;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(*inv) : "f"(s));  // s and 1 / s are normal numbers
    return c | 0x4300u | (uint32_t)nearest<F32>(nlo, s, *inv);
}

__device__ __forceinline__ float max_nan(float a, float b)
{
    float r;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
    return r;
}
__device__ __forceinline__ uint32_t max_nan2(uint32_t a, uint32_t b)
{
    const __nv_bfloat162 r = __hmax2_nan(*(const __nv_bfloat162*)&a, *(const __nv_bfloat162*)&b);
    return *(const uint32_t*)&r;
}
__device__ __forceinline__ uint32_t min_nan2(uint32_t a, uint32_t b)
{
    const __nv_bfloat162 r = __hmin2_nan(*(const __nv_bfloat162*)&a, *(const __nv_bfloat162*)&b);
    return *(const uint32_t*)&r;
}

// max x and -min x of some channels: one word of two bf16 numbers, or two of fp32
template <bool F32>
struct Ends {
    uint32_t w[F32 ? 2 : 1];
    __device__ __forceinline__ void join(const Ends& o)
    {
#pragma unroll
        for (int i = 0; i < (F32 ? 2 : 1); i++)
            w[i] = F32 ? __float_as_uint(max_nan(__uint_as_float(w[i]), __uint_as_float(o.w[i]))) : max_nan2(w[i], o.w[i]);
    }
    __device__ __forceinline__ Ends from(int lane_xor) const
    {
        Ends r;
#pragma unroll
        for (int i = 0; i < (F32 ? 2 : 1); i++) r.w[i] = __shfl_xor_sync(0xffffffffu, w[i], lane_xor);
        return r;
    }
    __device__ __forceinline__ float hi() const { return __uint_as_float(F32 ? w[0] : w[0] << 16); }
    __device__ __forceinline__ float nlo() const { return __uint_as_float(F32 ? w[F32 ? 1 : 0] : w[0] & 0xffff0000u); }
};

template <bool F32>
struct Elems {
    // 16 channels of one lane
    uint32_t w[F32 ? 16 : 8];
    __device__ __forceinline__ void load(const void* p)
    {
#pragma unroll
        for (int i = 0; i < (F32 ? 4 : 2); i++) {
            const uint4 x = __ldg((const uint4*)p + i);
            w[4 * i] = x.x, w[4 * i + 1] = x.y, w[4 * i + 2] = x.z, w[4 * i + 3] = x.w;
        }
    }
    __device__ __forceinline__ void zero()
    {
#pragma unroll
        for (int i = 0; i < (F32 ? 16 : 8); i++) w[i] = 0;
    }
    __device__ __forceinline__ Ends<F32> ends() const
    {
        Ends<F32> r;
        if (F32) {
            float hi = __uint_as_float(w[0]), nlo = -hi;
#pragma unroll
            for (int i = 1; i < 16; i++) {
                hi = max_nan(hi, __uint_as_float(w[F32 ? i : 0]));
                nlo = max_nan(nlo, -__uint_as_float(w[F32 ? i : 0]));
            }
            r.w[0] = __float_as_uint(hi);
            r.w[F32 ? 1 : 0] = __float_as_uint(nlo);
        } else {
            uint32_t h = w[0], l = w[0];
#pragma unroll
            for (int i = 1; i < 8; i++) h = max_nan2(h, w[i]), l = min_nan2(l, w[i]);
            l ^= 0x80008000u;
            r.w[0] = max_nan2(__byte_perm(h, l, 0x5410), __byte_perm(h, l, 0x7632));
        }
        return r;
    }
    __device__ __forceinline__ void times_2_64()
    {
#pragma unroll
        for (int i = 0; i < (F32 ? 16 : 8); i++) {
            if (F32) {
                w[i] = __float_as_uint(__uint_as_float(w[i]) * 0x1p64f);
            } else {  // exact: these vectors' elements are below 2^-96
                const float a = __uint_as_float(w[i] << 16) * 0x1p64f, b = __uint_as_float(w[i] & 0xffff0000u) * 0x1p64f;
                w[i] = __byte_perm(__float_as_uint(a), __float_as_uint(b), 0x7632);
            }
        }
    }
    // The codes, 8 a word, of a vector with a scale.
    __device__ __forceinline__ void codes(uint32_t param, float inv, uint32_t* word) const
    {
        const uint32_t z2 = (param & 15) * 0x10001u;
        const uint64_t inv2 = pair(inv, inv);
        // two codes less z, 16 bits each, to their places
        auto put = [&](int i, uint32_t k2) {
            const uint32_t c = __viaddmin_s16x2_relu(k2, z2, 0x000f000fu) << (4 * (i & 3));
            word[i >> 2] = i & 3 ? word[i >> 2] + c : c;
        };
        if (F32) {
            uint32_t k2[8];
            // x (1 / s) is off by less than 2^-18, so only next to a tie the nearest number is in doubt
            const uint64_t up = pair(kRound0, kRound0), down = pair(-kRound0, -kRound0), minus = pair(-1.f, -1.f);
            float far = 0.f;  // the largest distance from the number taken
#pragma unroll
            for (int i = 0; i < 8; i++) {
                const uint64_t x = pair(__uint_as_float(w[F32 ? 2 * i : 0]), __uint_as_float(w[F32 ? 2 * i + 1 : 0]));
                const uint64_t k = fma2(x, inv2, up);
                float k0, k1, d0, d1;
                unpair(k, k0, k1);
                unpair(fma2(x, inv2, fma2(add2(k, down), minus, 0)), d0, d1);
                far = fmaxf(far, fmaxf(fabsf(d0), fabsf(d1)));
                k2[i] = __byte_perm(__float_as_uint(k0), __float_as_uint(k1), 0x5410);
            }
            if (far > 0.5f - 0x1p-17f) {
                float s = scale_of(param);
                if (tiny_scale(s)) s *= 0x1p64f;
#pragma unroll
                for (int i = 0; i < 8; i++)
                    k2[i] = __byte_perm((uint32_t)nearest<F32>(__uint_as_float(w[F32 ? 2 * i : 0]), s, inv),
                                        (uint32_t)nearest<F32>(__uint_as_float(w[F32 ? 2 * i + 1 : 0]), s, inv), 0x5410);
            }
#pragma unroll
            for (int i = 0; i < 8; i++) put(i, k2[i]);
        } else {
            const uint64_t r11 = pair(kRound11, kRound11), r0 = pair(kRound0 - kRound11, kRound0 - kRound11);
#pragma unroll
            for (int i = 0; i < 8; i++) {
                float t0, t1;
                unpair(add2(fma2(pair(__uint_as_float(w[i] << 16), __uint_as_float(w[i] & 0xffff0000u)), inv2, r11), r0), t0, t1);
                put(i, __byte_perm(__float_as_uint(t0), __float_as_uint(t1), 0x5410));
            }
        }
    }
};

struct AppendArgs {
    uint8_t* pages;
    const uint8_t *k, *v;
    const int *rows, *slots;
    int* status;
    long long row_bytes;
    int n, n_rows, Hkv, page_log2, blk_log2, n_slots, heads_log2;
};

// A CTA's 8 warps: 2^heads_log2 heads by 8 / 2^heads_log2 groups of tokens.
template <int D, bool F32>
__global__ void __launch_bounds__(256) k_kv4_append(AppendArgs a)
{
    constexpr int L = D / 16, TOK = 32 / L;  // lanes of a vector, tokens of a warp
    constexpr int E = F32 ? 4 : 2;
    pdl_wait();
    pdl_trigger();
    const int lane = threadIdx.x & 31, sub = lane % L, warp = threadIdx.x >> 5;
    const int h = (blockIdx.y << a.heads_log2) + (warp & ((1 << a.heads_log2) - 1));
    const long long group = ((long long)blockIdx.x << (3 - a.heads_log2)) + (warp >> a.heads_log2), i = group * TOK + lane / L;
    if (h >= a.Hkv || group * TOK >= a.n) return;
    int slot = -1;
    long long row = i;
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
        e[0].zero();
        e[1].zero();
    }
    // K's extremes to the even lanes, V's to the odd ones
    const bool odd = lane & 1;
    const Ends<F32> ek = e[0].ends(), ev = e[1].ends();
    Ends<F32> m = odd ? ev : ek;
    m.join((odd ? ek : ev).from(1));
#pragma unroll
    for (int o = 2; o < L; o <<= 1) m.join(m.from(o));
    float inv[2];
    uint32_t param[2];
    {
        float mine;
        const uint32_t p = quant_params<F32>(m.hi(), m.nlo(), &mine);
        const uint32_t p2 = __shfl_xor_sync(0xffffffffu, p, 1);
        const float other = __shfl_xor_sync(0xffffffffu, mine, 1);
        param[0] = odd ? p2 : p, param[1] = odd ? p : p2;
        inv[0] = odd ? other : mine, inv[1] = odd ? mine : other;
    }
    if (!live) return;
    const int in_page = slot & ((1 << a.page_log2) - 1), tok = slot & 15;
    uint8_t* blk = a.pages + kv4_block_at(slot >> a.page_log2, h, in_page >> 4, a.Hkv, a.blk_log2, D);
#pragma unroll
    for (int p = 0; p < 2; p++) {
        uint32_t w[2];
        if (tiny_scale(scale_of(param[p]))) e[p].times_2_64();
        e[p].codes(param[p], inv[p], w);
        if (!(scale_of(param[p]) > 0.f)) w[0] = w[1] = 0;  // scale 0 or NaN: every code 0
        *(uint2*)(blk + p * 8 * D + (sub >> 2) * 512 + tok * 32 + (sub & 3) * 8) = make_uint2(w[0], w[1]);
        if (sub == p) *(uint32_t*)(blk + 16 * D + p * 64 + tok * 4) = param[p];
    }
}

// ------------------------------------------------------------------ read ---
//
// The values (c - z) s of tokens, in fp32 (exact: 4 + 8 bits) or rounded to
// bf16 (once: c - z is exact in bf16, too, so the packed product there rounds
// the exact value).  One word of codes is 8 channels and 16 bytes of bf16: a
// lane takes the same word of two tokens, K and V (or, for fp32, halves of two
// words of them), so that a warp's loads and stores cover whole lines.  HBM bound: 18 K tokens of 8 heads, D = 128, into bf16
// 13.6 us (96 MB: 14.1 us at a plain copy's rate), into fp32 27.1 us (171 MB: 25.2).

struct ReadArgs {
    const uint8_t* pages;
    uint8_t *k, *v;
    const int* slots;
    int* status;
    long long row_bytes;
    int n, Hkv, page_log2, blk_log2, n_slots, heads_log2;
};

template <int D, bool F32>
__global__ void __launch_bounds__(256) k_kv4_read(ReadArgs a)
{
    constexpr int L = D / 8, TOK = 32 / L, E = F32 ? 4 : 2;  // a warp: TOK tokens at a time, two times
    pdl_wait();
    pdl_trigger();
    const int lane = threadIdx.x & 31, sub = lane % L, warp = threadIdx.x >> 5;
    const int h = (blockIdx.y << a.heads_log2) + (warp & ((1 << a.heads_log2) - 1));
    const long long group = ((long long)blockIdx.x << (3 - a.heads_log2)) + (warp >> a.heads_log2);
    const long long i0 = group * 2 * TOK + lane / L;
    if (h >= a.Hkv) return;
    constexpr int NW = F32 ? 2 : 1;
    uint32_t w[2][2][NW], prm[2][2];
    bool live[2];
#pragma unroll
    for (int t = 0; t < 2; t++) {
        const long long i = i0 + t * TOK;
        int slot = i < a.n ? a.slots[i] : -1;
        if (slot >= a.n_slots) {
            kv4_raise(a.status, LA_ERR_ARG);
            slot = -1;
        }
        live[t] = slot >= 0;
        if (!live[t]) continue;
        const int in_page = slot & ((1 << a.page_log2) - 1), tok = slot & 15;
        const uint8_t* blk = a.pages + kv4_block_at(slot >> a.page_log2, h, in_page >> 4, a.Hkv, a.blk_log2, D);
#pragma unroll
        for (int p = 0; p < 2; p++) {
#pragma unroll
            for (int j = 0; j < NW; j++) {
                const int wd = F32 ? (j * L + sub) >> 1 : sub;
                w[t][p][j] = *(const uint32_t*)(blk + p * 8 * D + (wd >> 3) * 512 + tok * 32 + (wd & 7) * 4);
            }
            prm[t][p] = *(const uint32_t*)(blk + 16 * D + p * 64 + tok * 4);
        }
    }
#pragma unroll
    for (int t = 0; t < 2; t++) {
        if (!live[t]) continue;
        const size_t at = (size_t)(i0 + t * TOK) * a.row_bytes + (size_t)h * D * E + sub * 16;
#pragma unroll
        for (int p = 0; p < 2; p++) {
            const uint32_t q = prm[t][p];
            uint8_t* dst = (p ? a.v : a.k) + at;
            // a code in the mantissa of 128 (bf16: 1 a unit; fp32: 2^16 a unit), less 128 + z
            if (F32) {
                const float s = scale_of(q), z = __uint_as_float(q << 16);
#pragma unroll
                for (int j = 0; j < NW; j++) {
                    const uint32_t u = w[t][p][j] >> (8 * (sub & 1));
                    float x[4];
#pragma unroll
                    for (int c = 0; c < 4; c++)
                        x[c] = (__uint_as_float(0x43000000u | ((u >> (4 * (c >> 1) + 16 * (c & 1))) & 15u) << 16) - z) * s;
                    *(float4*)(dst + j * L * 16) = make_float4(x[0], x[1], x[2], x[3]);
                }
            } else {
                const uint32_t s2 = __byte_perm(q, q, 0x3232), z2 = __byte_perm(q, q, 0x1010);
                uint32_t y[4];
#pragma unroll
                for (int c = 0; c < 4; c++) {
                    const uint32_t x = (w[t][p][0] >> (4 * c) & 0x000f000fu) | 0x43004300u;
                    const __nv_bfloat162 r = __hmul2_rn(__hsub2_rn(*(const __nv_bfloat162*)&x, *(const __nv_bfloat162*)&z2),
                                                        *(const __nv_bfloat162*)&s2);
                    y[c] = *(const uint32_t*)&r;
                }
                *(uint4*)dst = make_uint4(y[0], y[1], y[2], y[3]);
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

// The CTAs of append and read: 8 warps each, a warp 512 / D tokens of a head,
// the heads of a token next to each other (their rows are).
dim3 token_grid(const la_kv4_desc& c, int n, int* heads_log2)
{
    *heads_log2 = std::min(3, log2_of(c.n_kv_heads));
    const long long tokens = (512LL / c.head_dim) << (3 - *heads_log2), heads = 1 << *heads_log2;
    return dim3((unsigned)((n + tokens - 1) / tokens), (unsigned)((c.n_kv_heads + heads - 1) / heads));
}

int done(cudaError_t e) { return e == cudaSuccess ? LA_OK : LA_ERR_CUDA; }

}  // namespace

int launch_kv4_plan(cudaStream_t s, const la_kv4_desc& c, const int* lens, const int* n_new, int B, const int* free_pages,
                    const int* n_free, int* table, int* slots, int n_slots, int stride, int* new_lens, int* left)
{
    if (int rc = plan_ready()) return rc;
    PlanArgs a{lens, n_new, free_pages, n_free, table, slots, new_lens, left, c.status, B, log2_of(c.page), c.max_pages,
               c.n_pages, n_slots, stride, kPlanAll};
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
                 c.n_pages * c.page, 0};
    const dim3 grid = token_grid(c, n, &a.heads_log2);
    auto kern = c.head_dim == 128 ? (f32 ? k_kv4_append<128, true> : k_kv4_append<128, false>)
                                  : (f32 ? k_kv4_append<64, true> : k_kv4_append<64, false>);
    return done(launch_pdl(kern, grid, dim3(256), 0, s, a));
}

int launch_kv4_read(cudaStream_t s, const la_kv4_desc& c, const int* slots, int n, void* k, void* v, int dtype, int ld)
{
    const bool f32 = dtype == LA_FP32;
    ReadArgs a{(const uint8_t*)c.pages, (uint8_t*)k, (uint8_t*)v, slots, c.status, (long long)ld * (f32 ? 4 : 2), n,
               c.n_kv_heads, log2_of(c.page), log2_of(c.page / 16), c.n_pages * c.page, 0};
    const dim3 grid = token_grid(c, n, &a.heads_log2);
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
    return c->max_pages >= 1 && (long long)c->max_pages * c->page <= (1LL << 30);  // (lengths in tiles stay within an int)
}

bool aligned(const void* p, int to) { return ((uintptr_t)p & (uintptr_t)(to - 1)) == 0; }

// every address one of an int (a misaligned access would end the context)
template <typename... P>
bool ints_aligned(const P*... p)
{
    return (aligned(p, 4) && ...);
}

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
    if (!ints_aligned(lens, n_new, free_pages, n_free, table, slots, new_lens, pages_left, c->status)) return LA_ERR_ARG;
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
    // (of free_pages only its first entry is known to be there)
    for (const int* in : {n_free, free_pages})
        if (overlap(in, slots, 1, n_slots) || overlap(in, table, 1, tab) || overlap(in, new_lens, 1, batch)) return LA_ERR_ARG;
    if (overlap(pages_left, free_pages, 1, 1)) return LA_ERR_ARG;
    return launch_kv4_plan((cudaStream_t)stream, *c, lens, n_new, batch, free_pages, n_free, table, slots, n_slots,
                           slot_stride, new_lens, pages_left);
}

extern "C" int la_kv4_release(const la_kv4_desc* c, const int32_t* done, int batch, int32_t* lens, const int32_t* table,
                              int32_t* free_pages, int32_t* n_free, void* stream)
{
    if (!desc_ok(c) || batch < 0 || batch > kPlanMaxBatch) return LA_ERR_ARG;
    if (batch == 0) return LA_OK;
    if (!done || !lens || !table || !free_pages || !n_free) return LA_ERR_ARG;
    if (!ints_aligned(done, lens, table, free_pages, n_free, c->status)) return LA_ERR_ARG;
    const size_t tab = (size_t)batch * c->max_pages, room = c->n_pages;
    if (overlap(free_pages, lens, room, batch) || overlap(free_pages, done, room, batch) || overlap(free_pages, table, room, tab) ||
        overlap(free_pages, n_free, room, 1) || overlap(lens, table, batch, tab) || (lens != done && overlap(lens, done, batch, batch)) ||
        overlap(n_free, lens, 1, batch) || overlap(n_free, done, 1, batch) || overlap(n_free, table, 1, tab))
        return LA_ERR_ARG;
    return launch_kv4_release((cudaStream_t)stream, *c, done, batch, lens, table, free_pages, n_free);
}

extern "C" int la_kv4_append(const la_kv4_desc* c, const void* k, const void* v, int dtype, int ld, int n_rows,
                             const int32_t* rows, const int32_t* slots, int n, void* stream)
{
    if (!pool_ok(c) || n < 0 || n_rows < 0 || (dtype != LA_FP32 && dtype != LA_BF16)) return LA_ERR_ARG;
    if (n == 0) return LA_OK;
    if (!k || !v || !slots || !aligned(k, 16) || !aligned(v, 16) || !ints_aligned(rows, slots)) return LA_ERR_ARG;
    if (ld < c->n_kv_heads * c->head_dim || (ld * (dtype == LA_FP32 ? 4LL : 2LL)) % 16) return LA_ERR_ARG;
    if (!rows && n > n_rows) return LA_ERR_ARG;
    return launch_kv4_append((cudaStream_t)stream, *c, k, v, dtype, ld, n_rows, rows, slots, n);
}

extern "C" int la_kv4_read(const la_kv4_desc* c, const int32_t* slots, int n, void* k, void* v, int dtype, int ld,
                           void* stream)
{
    if (!pool_ok(c) || n < 0 || (dtype != LA_FP32 && dtype != LA_BF16)) return LA_ERR_ARG;
    if (n == 0) return LA_OK;
    if (!k || !v || !slots || !aligned(k, 16) || !aligned(v, 16) || !ints_aligned(slots)) return LA_ERR_ARG;
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
    if (!ints_aligned(a->lens, a->table)) return LA_ERR_ARG;
    if (!aligned(a->q, 16) || !aligned(a->k_step, 16) || !aligned(a->v_step, 16) || !aligned(a->out, 16)) return LA_ERR_ARG;
    if (a->q_ld < a->n_heads * c->head_dim || a->q_ld % 8 || a->kv_ld < c->n_kv_heads * c->head_dim || a->kv_ld % 8)
        return LA_ERR_ARG;
    const size_t need = kv4_attn_bytes(*c, *a);
    if (need && (!a->workspace || !aligned(a->workspace, 16) || a->ws_bytes < need)) return LA_ERR_ARG;
    return launch_kv4_attn((cudaStream_t)stream, *c, *a);
}
