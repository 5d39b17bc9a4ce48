// kv16_sched.cuh -- how the attention kernels over the paged bf16 cache share
// their work.
//
// Entries are prefixes (the rows of all their sequences) or sequences.  An
// entry's keys are blocks of 16: the prefix's, the sequence's own, the step's
// rows; only the last block of each of the three has fewer keys.  For each KV
// head its rows are cut into items of row_tile rows.  All items lie end to end
// in units (a tile of keys, with `extra` units for an item's queries and its
// result) and are cut into equal runs, one per team, whatever the lengths; or,
// where there is an item or none for each team and their sizes are close, a
// team takes a whole item, which then leaves no parts.
#pragma once
#include "kv16.cuh"

namespace la {
namespace {

using namespace ptx;

constexpr int kSMs = 152;
constexpr float kNoRef = -3e38f;  // below every score: exp2(-inf - kNoRef) = 0

__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi)
{
    __nv_bfloat162 v = __floats2bfloat162_rn(lo, hi);
    return *reinterpret_cast<uint32_t*>(&v);
}

__device__ __forceinline__ int blocks_of(int n) { return (n + 15) >> 4; }

// The prefix of sequence b, or -1.
__device__ __forceinline__ int prefix_of(const Kv16Attn& a, int b)
{
    int lo = -1, hi = a.nP;  // pfirst[lo] <= b < pfirst[hi], taking the ends as -inf and inf
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (a.pfirst[mid] <= b) lo = mid;
        else hi = mid;
    }
    return lo >= 0 && b < a.pfirst[lo + 1] ? lo : -1;
}

struct Entry {
    int rows, row0;    // rows of a KV head (0: nothing to do), the first of them among all sequences'
    int b, p;          // sequence (-1: a prefix's entry); prefix whose tokens come first (-1: none)
    int plen, len;     // tokens
    int nb_pre, nb;    // blocks: the prefix's, all
    int wide, tiles, mt, nu;  // does a tile count twice; tiles; row tiles; an item's units
    __device__ __forceinline__ int nb_cached() const { return nb_pre + blocks_of(len); }
};

__device__ __forceinline__ Entry entry_of(const Kv16Attn& a, const Kv16Sched& s, int e)
{
    Entry x;
    x.plen = x.len = x.rows = x.row0 = x.nb = 0;
    if (e < s.n_pre) {
        const int lo = a.pfirst[e], n = a.plens[e];
        x.b = -1, x.p = e;
        if (n > 0 && n <= a.max_plen) x.plen = n, x.rows = (a.pfirst[e + 1] - lo) * a.R, x.row0 = lo * a.R;
    } else {
        const int b = e - s.n_pre, n = a.lens[b], p = a.nP ? prefix_of(a, b) : -1, pn = p >= 0 ? a.plens[p] : 0;
        x.b = b, x.p = p, x.row0 = b * a.R;
        if (n >= 0 && n <= a.max_len && pn <= a.max_plen) {
            x.len = n, x.rows = a.R, x.nb = blocks_of(a.T);
            if (a.concat && pn > 0) x.plen = pn;
        }
    }
    x.nb_pre = blocks_of(x.plen);
    x.nb += x.nb_pre + blocks_of(x.len);
    x.wide = x.rows > s.wide;
    x.tiles = (x.nb + (1 << s.blk_log2) - 1) >> s.blk_log2;
    x.mt = (x.rows + s.row_tile - 1) / s.row_tile;
    x.nu = x.rows ? s.extra + (x.tiles << x.wide) : 0;
    return x;
}

// The first tile at or behind unit u of an item.
__device__ __forceinline__ int tile_at(const Kv16Sched& s, const Entry& x, int u) { return max(u - s.extra + x.wide, 0) >> x.wide; }

__device__ __forceinline__ long long units_at(const Kv16Shares& h, int t) { return h.q * t + min(t, h.r); }

__device__ __noinline__ long long div_long(long long a, long long b) { return a / b; }

__device__ __forceinline__ long long div_units(long long a, long long b)
{
    // (a 64-bit division takes half a microsecond)
    return (a | b) < (1LL << 32) ? (long long)((uint32_t)a / (uint32_t)b) : div_long(a, b);
}

// The team that holds a unit.
__device__ __forceinline__ int team_of(const Kv16Shares& h, long long u)
{
    const long long wide = (h.q + 1) * h.r;
    return (int)(u < wide ? div_units(u, h.q + 1) : h.r + div_units(u - wide, h.q));
}

struct Start {
    int e, pad;
    long long off, count;  // offset in the units of entry e's items; units of the team
};

struct Scan {
    long long units[33], items[33];
    int top[32];
    Kv16Shares shares;
};

// Where each of the CTA's teams t0 .. t0 + n - 1 begins.  CTA 0 leaves the
// schedule for the merge and raises what is wrong with the sequences.
__device__ void find_starts(const Kv16Attn& a, const Kv16Sched& s, int t0, int n, Start* starts, Scan* sc)
{
    const int entries = s.n_pre + s.n_seq, per = ceil_div(entries, (int)blockDim.x), e0 = threadIdx.x * per, e1 = min(e0 + per, entries);
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, nw = blockDim.x >> 5;
    bool bad = false;
    for (int p = threadIdx.x; p < a.nP; p += blockDim.x) {
        const int lo = a.pfirst[p], hi = a.pfirst[p + 1];
        bad |= lo < 0 || hi > a.B || lo > hi;
    }
    bad = __syncthreads_or(bad);
    if (blockIdx.x == 0 && s.first) {
        bool wrong = bad;
        for (int b = threadIdx.x; b < a.B; b += blockDim.x) wrong |= a.lens[b] > a.max_len;
        for (int p = threadIdx.x; p < a.nP; p += blockDim.x) wrong |= a.plens[p] > a.max_plen;
        if (wrong) kv4_raise(a.status, LA_ERR_ARG);
    }
    long long units = 0, items = 0;
    int top = 0;
    if (!bad)
        for (int e = e0; e < e1; e++) {
            const Entry x = entry_of(a, s, e);
            const int k = a.Hkv * x.mt;
            units += (long long)k * x.nu, items += k, top = max(top, x.nu);
        }
    if ((int)threadIdx.x < n) starts[threadIdx.x].count = 0;
    long long xu = units, xi = items;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const long long yu = __shfl_up_sync(0xffffffffu, xu, o), yi = __shfl_up_sync(0xffffffffu, xi, o);
        if (lane >= o) xu += yu, xi += yi;
    }
    top = __reduce_max_sync(0xffffffffu, top);
    if (lane == 31) sc->units[warp] = xu, sc->items[warp] = xi, sc->top[warp] = top;
    __syncthreads();
    long long bu = xu - units, bi = xi - items, all_u = 0, all_i = 0;
    for (int w = 0; w < nw; w++) {
        const long long u = sc->units[w], i = sc->items[w];
        if (w < warp) bu += u, bi += i;
        all_u += u, all_i += i, top = max(top, sc->top[w]);
    }
    Kv16Shares h;
    h.whole = all_i <= s.nteams && top - s.slack <= div_units(all_u, s.nteams), h.pad = 0;
    const long long all = h.whole ? all_i : all_u;
    h.nteams = h.whole ? (int)all_i : (int)min((long long)s.nteams, max(1LL, div_units(all, s.min_run)));
    if (all == 0) h.nteams = 0;
    h.q = h.nteams ? div_units(all, h.nteams) : 0;
    h.r = (int)(all - h.q * h.nteams);
    const bool notes = blockIdx.x == 0;
    if (threadIdx.x == 0) {
        sc->shares = h;
        if (notes && s.shares) *s.shares = h;
    }
    if (h.nteams && (notes || units)) {
        long long at = h.whole ? bi : bu;
        const long long end = at + (h.whole ? items : units);
        int i = 0;
        // the teams that begin within this thread's entries
        while (i < n && (t0 + i >= h.nteams || units_at(h, t0 + i) < at)) i++;
        if (notes ? s.base != nullptr || i < n : i < n && units_at(h, t0 + i) < end)
            for (int e = e0; e < e1; e++) {
                const Entry x = entry_of(a, s, e);
                const long long c = (long long)a.Hkv * x.mt * (h.whole ? 1 : x.nu);
                if (notes && s.base) s.base[e] = at;
                for (; i < n && t0 + i < h.nteams; i++) {
                    const long long u0 = units_at(h, t0 + i);
                    if (u0 >= at + c) break;
                    starts[i] = Start{e, 0, u0 - at, units_at(h, t0 + i + 1) - u0};
                }
                at += c;
            }
    }
    __syncthreads();
}

// The run of one item's units that a team works on: tiles t0 .. t1 - 1 of KV
// head g's rows from r0 of entry e.
struct Run {
    Entry x;
    int e, item, whole, u0, u1, nu, t0, t1;
    long long left;
    __device__ __forceinline__ void cut(const Kv16Sched& s, int from)
    {
        nu = whole ? 1 : x.nu;
        u0 = from;
        u1 = (int)min((long long)nu, u0 + left);
        left -= u1 - u0;
        t0 = whole ? 0 : tile_at(s, x, u0);
        t1 = whole ? x.tiles : tile_at(s, x, u1);
    }
    __device__ __forceinline__ void begin(const Kv16Attn& a, const Kv16Sched& s, const Start& st, const Kv16Shares& h)
    {
        left = st.count, whole = h.whole, e = st.e;
        x = entry_of(a, s, e);
        const int n = whole ? 1 : x.nu;
        item = (int)div_units(st.off, n);
        cut(s, (int)(st.off - (long long)item * n));
    }
    __device__ __forceinline__ bool next(const Kv16Attn& a, const Kv16Sched& s)
    {
        if (left <= 0) return false;
        if (++item == a.Hkv * x.mt) {
            item = 0;
            do {
                if (++e >= s.n_pre + s.n_seq) return false;  // only if the lengths change under the call
                x = entry_of(a, s, e);
            } while (x.nu == 0);
        }
        cut(s, 0);
        return true;
    }
    // all of the item's units: no other team has a part of it
    __device__ __forceinline__ bool all() const { return u0 == 0 && u1 == nu; }
    // which of the team's two parts it is: 1 begins an item, 0 goes on with one
    __device__ __forceinline__ int slot() const { return u0 == 0; }
};

// Floats of a part and of the results of whole items.  A thread per row writes
// columns ([D + 2][rows]: outputs, M, sum), so that a warp's stores are lines;
// fragments of 8 rows x 4 lanes write rows ([rows][D], then [rows][M, sum]).
constexpr int kWideRows = 256;   // rows of an item of k_kv16_wide, in two tiles
__host__ __device__ constexpr size_t wide_part(int D) { return (size_t)2 * 128 * (D + 2); }
__host__ __device__ constexpr size_t rows_part(int D, int R) { return ((size_t)R * (D + 2) + 3) / 4 * 4; }  // (16-byte aligned)

}  // namespace

// Joins the parts of every row (kv16_attn.cu).
struct Kv16Merge {
    Kv16Sched pre, seq;       // n_pre of `pre` 0: no prefixes of their own
    int seq_rows;             // sequences' parts are rows (k_kv16_rows), else columns
    int rows_all;             // rows of a KV head of all sequences
};

}  // namespace la
