// kv16_sched.cuh -- how the attention kernels over the paged bf16 cache share
// their work.
//
// Entries are prefixes (the rows of all their sequences) or sequences.  An
// entry's keys are blocks of 16: the prefix's, the sequence's own, the step's
// rows; only the last block of each of the three has fewer keys.  For each KV
// head its rows are cut into items of row_tile rows.  All items lie end to end
// in units (a tile of keys, with `extra` units for an item's queries and its
// result) and are cut into equal runs, one per team, whatever the lengths; or,
// where there are few items and their sizes are close, a team takes whole items,
// which then leave no parts (240 items of 10 or 11 tiles on 152 teams, one or two
// each: 42.2 us, cut into equal runs 44.3).
#pragma once
#include <cfloat>

#include "kv16.cuh"

namespace la {
namespace {

using namespace ptx;

constexpr int kSMs = 152;
constexpr float kNoRef = -FLT_MAX;  // below every score: exp2((-inf - kNoRef) f) = 0

__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi)
{
    __nv_bfloat162 v = __floats2bfloat162_rn(lo, hi);
    return *reinterpret_cast<uint32_t*>(&v);
}

__device__ __forceinline__ int blocks_of(int n) { return (n + 15) >> 4; }

// The prefixes' bounds and lengths, copied to shared memory where they fit.
struct Prefixes {
    const int *first, *lens;
};

// The prefix of sequence b, or -1.
__device__ __forceinline__ int prefix_of(const Kv16Attn& a, const Prefixes& pre, int b)
{
    int lo = -1, hi = a.nP;  // first[lo] <= b < first[hi], taking the ends as -inf and inf
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (pre.first[mid] <= b) lo = mid;
        else hi = mid;
    }
    return lo >= 0 && b < pre.first[lo + 1] ? lo : -1;
}

struct Entry {
    int rows, row0;    // rows of a KV head (0: nothing to do), the first of them among all sequences'
    int b, p;          // sequence (-1: a prefix's entry); prefix (-1: none)
    int plen, len;     // tokens
    int nb_pre, nb;    // blocks: the prefix's, all
    int wide, tiles, mt, nu;  // does a tile count twice; tiles; row tiles; an item's units
    __device__ __forceinline__ int nb_cached() const { return nb_pre + blocks_of(len); }
};

template <class K>
__device__ __forceinline__ int tiles_of(int blocks) { return (blocks + (1 << K::blk_log2) - 1) >> K::blk_log2; }

// An entry; n: the sequence's own tokens (not looked at for a prefix's entry).
template <class K>
__device__ __forceinline__ Entry entry_with(const Kv16Attn& a, const Kv16Sched& s, const Prefixes& pre, int e, int n)
{
    Entry x;
    x.plen = x.len = x.rows = x.row0 = x.nb = 0;
    if (e < s.n_pre) {
        const int lo = pre.first[e], m = pre.lens[e];
        x.b = -1, x.p = e;
        if (m > 0 && m <= a.max_plen) x.plen = m, x.rows = (pre.first[e + 1] - lo) * a.R, x.row0 = lo * a.R;
    } else {
        const int b = e - s.n_pre, p = a.nP ? prefix_of(a, pre, b) : -1, pn = p >= 0 ? pre.lens[p] : 0;
        x.b = b, x.p = pn > 0 ? p : -1, x.row0 = b * a.R;
        if (n >= 0 && n <= a.max_len && pn <= a.max_plen) {
            x.len = n, x.rows = a.R, x.nb = blocks_of(a.T);
            if (a.concat && pn > 0) x.plen = pn;
        }
    }
    x.nb_pre = blocks_of(x.plen);
    x.nb += x.nb_pre + blocks_of(x.len);
    x.wide = K::twice && x.rows > K::twice;
    x.tiles = tiles_of<K>(x.nb);
    x.mt = K::twice ? (x.rows + K::row_tile - 1) / K::row_tile : x.rows > 0;
    x.nu = x.rows ? K::extra + (x.tiles << x.wide) : 0;
    return x;
}

template <class K>
__device__ __forceinline__ Entry entry_of(const Kv16Attn& a, const Kv16Sched& s, const Prefixes& pre, int e)
{
    return entry_with<K>(a, s, pre, e, e < s.n_pre ? 0 : a.lens[e - s.n_pre]);
}

// The first tile at or behind unit u of an item.
template <class K>
__device__ __forceinline__ int tile_at(const Entry& x, int u) { return max(u - K::extra + x.wide, 0) >> x.wide; }

// The teams' runs: team t begins at unit q t + min(t, r).  (All units fit 31 bits,
// or nothing is done: 64-bit sums and divisions took most of a small call's time.)
struct Shares {
    int q, r, nteams, whole;  // whole: a unit is a whole item
    __device__ __forceinline__ int at(int t) const { return q * t + min(t, r); }
    __device__ __forceinline__ int team_of(int u) const  // that holds unit u
    {
        const int wide = (q + 1) * r;
        return u < wide ? (int)((unsigned)u / (unsigned)(q + 1)) : r + (int)((unsigned)(u - wide) / (unsigned)q);
    }
};

struct Start {
    int e, off, count, team;  // entry, offset in the units of its items; units of the team
};

struct PreShared {
    static constexpr int kMost = 32;
    int first[kMost + 1], lens[kMost];
};

struct Scan {
    int units[32], big[32], items[32], top[32];
    Shares shares;
};

// Where some CTAs take prefixes and the others sequences, how many take prefixes: with
// uw units (a tile for a stream: 32 KB of a pair's tile, 0.95 us) and ur blocks (8 KB at
// D = 128, 0.126 us at what one SM can read) both end together.  Where HBM and not the
// SMs sets the pace, a wide unit waits for its tiles and takes 1.73 us.  (128 single
// tokens behind 1000 and 48 behind prefixes of up to 4000, us in all, at 1.0, 1.4, 1.73
// and 2.4 us a unit: 74.8, 64.0, 65.5, 67.5 and 64.4, 57.1, 54.5, 55.8; at 0.09, 0.126
// and 0.18 us a block: 67.6, 65.5, 64.1 and 55.6, 54.5, 75.4.  At D = 64 the former is
// 42.5 with 0.45 or 0.6 of these times, 51.9 with 0.8 or all.)  One kind after the other
// took 89 us for the former.
__device__ __forceinline__ int wide_sms(float uw, float ur, int D)
{
    const float half = D == 128 ? 1.f : 0.6f, tw = 0.95f * half, tr = 0.126f * half;
    const float hbm = (uw * 32.f + ur * 8.f) * (D / 128.f) / 6600.f;
    const bool waits = hbm > (uw * tw + ur * tr) / kSMs;
    const float w = uw * (waits ? 1.73f * half : tw), r = ur * tr;
    return min(max((int)(w * kSMs / fmaxf(w + r, 1e-3f)) + 1, 4), kSMs - 8);
}

// What a thread's entries come to.
struct Sums {
    int e0, e1, units, items, before;  // before: units of the warp's threads up to this one
    Entry x0;
};

// The sequences and prefixes as they are, the same for all schedules: word of what is
// wrong with them (by CTA 0), prefixes to shared memory where they fit.  True: nothing
// is to be done.
__device__ __forceinline__ bool look_over(const Kv16Attn& a, PreShared* ps, Prefixes& pre)
{
    const bool fits = a.nP <= PreShared::kMost;
    bool bad = false, wrong = false;
    for (int p = threadIdx.x; p < a.nP; p += blockDim.x) {
        const int lo = a.pfirst[p], hi = a.pfirst[p + 1], m = a.plens[p];
        bad |= lo < 0 || hi > a.B || lo > hi;
        wrong |= m > a.max_plen;
        if (fits) {
            ps->first[p] = lo, ps->lens[p] = m;
            if (p == a.nP - 1) ps->first[p + 1] = hi;
        }
    }
    if (blockIdx.x == 0) {
        for (int b = threadIdx.x; b < a.B; b += blockDim.x) wrong |= a.lens[b] > a.max_len;
        if (wrong || bad) kv4_raise(a.status, LA_ERR_ARG);
    }
    pre = fits ? Prefixes{ps->first, ps->lens} : Prefixes{a.pfirst, a.plens};
    return __syncthreads_or(bad);
}

__device__ __forceinline__ void first_entry(const Kv16Sched& s, int& e0, int& e1)
{
    const int entries = s.n_pre + s.n_seq, per = entries <= (int)blockDim.x ? 1 : ceil_div(entries, (int)blockDim.x);
    e0 = threadIdx.x * per, e1 = min(e0 + per, entries);
}

// Adds up the entries of each thread, and those of a warp in sc (len0: the length of the thread's first one).
template <class K>
__device__ __forceinline__ Sums add_up(const Kv16Attn& a, const Kv16Sched& s, const Prefixes& pre, Scan* sc, bool bad, int len0)
{
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    Sums y;
    first_entry(s, y.e0, y.e1);
    y.x0.mt = y.x0.nu = 0;
    long long sum = 0;
    int items = 0, top = 0;
    if (!bad) {
        for (int e = y.e0; e < y.e1; e++) {
            const Entry x = entry_with<K>(a, s, pre, e, e == y.e0 || e < s.n_pre ? len0 : a.lens[e - s.n_pre]);
            const int k = a.Hkv * x.mt;
            if (e == y.e0) y.x0 = x;
            if (x.nu) sum += (long long)k * x.nu, items = min(items + k, 1 << 20), top = max(top, x.nu);
            else if (!s.finish && x.b >= 0 && blockIdx.x == 0)
                // no rows, which the merge is to know
                for (int g = 0; g < a.Hkv; g++) s.items[(size_t)(a.Hkv + g) * a.B * a.R + x.row0].n = 0;
        }
    }
    y.units = (int)min(sum, 0x7fff0000LL);  // (there, or nothing is done: see `huge`)
    y.items = items;
    int xu = y.units;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int z = __shfl_up_sync(0xffffffffu, xu, o);
        if (lane >= o) xu += z;
    }
    y.before = xu - y.units;
    const int w_big = __reduce_add_sync(0xffffffffu, (int)min(sum >> 16, 1LL << 20)), w_items = __reduce_add_sync(0xffffffffu, items),
              w_top = __reduce_max_sync(0xffffffffu, top);
    if (lane == 31) sc->units[warp] = xu, sc->big[warp] = w_big, sc->items[warp] = w_items, sc->top[warp] = w_top;
    return y;
}

// All entries' units, or -1 if they do not fit.  (Behind a barrier after add_up.)
__device__ __forceinline__ int all_units(const Scan* sc)
{
    const int lane = threadIdx.x & 31;
    const bool in = lane < (int)blockDim.x >> 5;
    const bool huge = __reduce_add_sync(0xffffffffu, in ? sc->big[lane] : 0) >= 0x7000;
    const int all = __reduce_add_sync(0xffffffffu, in ? sc->units[lane] : 0);
    return huge ? -1 : all;
}

// Word of whether all is well, by one thread of the call.
__device__ __forceinline__ void say_bad(const Kv16Attn& a, const Kv16Sched& s, bool bad, bool huge)
{
    if (blockIdx.x != 0 || threadIdx.x != 0) return;
    if (huge) kv4_raise(a.status, LA_ERR_ARG);
    if (s.bad) *s.bad = bad || huge;
}

// Where each of the teams of CTA `cta` of `ctas` begins; the shares go to sc.
template <class K>
__device__ __forceinline__ void share_out(const Kv16Attn& a, const Kv16Sched& s, const Prefixes& pre, const Sums& y, int all_u, Start* starts, Scan* sc,
                                          int cta, int ctas)
{
    const int n = s.per_cta, lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const bool in = lane < (int)blockDim.x >> 5;
    const int it = in ? sc->items[lane] : 0;
    const int before = __reduce_add_sync(0xffffffffu, lane < warp ? sc->units[lane] : 0) + y.before;
    const int all_i = __reduce_add_sync(0xffffffffu, it), top = __reduce_max_sync(0xffffffffu, in ? sc->top[lane] : 0);
    const bool huge = all_u < 0;
    const int room = min(s.nteams, ctas * n);
    Shares h;
    // Whole items leave no parts: worth `slack` units of the longest team's work.
    h.whole = !huge && all_i <= 4 * room && ceil_div(all_i, room) * top - K::slack <= (int)((unsigned)all_u / (unsigned)room);
    int bi = 0;
    if (h.whole) {
        // the same for whole items
        int xi = y.items;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int z = __shfl_up_sync(0xffffffffu, xi, o);
            if (lane >= o) xi += z;
        }
        bi = xi - y.items + __reduce_add_sync(0xffffffffu, lane < warp ? it : 0);
    }
    const int all = huge ? 0 : h.whole ? all_i : all_u;
    h.nteams = all == 0 ? 0 : h.whole ? min(all_i, room) : min(room, max(1, (int)((unsigned)all / (unsigned)K::min_run)));
    h.q = h.nteams ? (int)((unsigned)all / (unsigned)h.nteams) : 0;
    h.r = all - h.q * h.nteams;
    if (threadIdx.x == 0) sc->shares = h;
    if (h.nteams && y.units) {
        int at = h.whole ? bi : before;
        const int end = at + (h.whole ? y.items : y.units);
        // the CTAs' teams by turns: few teams are spread over the SMs
        int i = 0;
        auto team = [&](int j) { return j * ctas + cta; };
        // the teams that begin within this thread's entries
        while (i < n && team(i) < h.nteams && h.at(team(i)) < at) i++;
        if (i < n && team(i) < h.nteams && h.at(team(i)) < end)
            for (int e = y.e0; e < y.e1; e++) {
                const Entry x = e == y.e0 ? y.x0 : entry_of<K>(a, s, pre, e);
                const int c = a.Hkv * x.mt * (h.whole ? x.nu > 0 : x.nu);
                for (; i < n && team(i) < h.nteams; i++) {
                    const int u0 = h.at(team(i));
                    if (u0 >= at + c) break;
                    starts[i] = Start{e, u0 - at, h.at(team(i) + 1) - u0, team(i)};
                }
                at += c;
            }
    }
    __syncthreads();
}

// The length of the thread's first entry, asked for before anything else.
__device__ __forceinline__ int first_len(const Kv16Attn& a, const Kv16Sched& s)
{
    int e0, e1;
    first_entry(s, e0, e1);
    return !s.direct && e0 < e1 && e0 >= s.n_pre ? a.lens[e0 - s.n_pre] : 0;
}

// Where each of the CTA's teams begins, for a kernel of one schedule.
template <class K>
__device__ __forceinline__ Prefixes find_starts(const Kv16Attn& a, const Kv16Sched& s, Start* starts, Scan* sc, PreShared* ps)
{
    const int len0 = first_len(a, s), n = s.per_cta;
    Prefixes pre;
    if ((int)threadIdx.x < n) starts[threadIdx.x].count = 0;
    const bool bad = look_over(a, ps, pre);
    if (s.direct) {
        const int mt = (a.R + K::row_tile - 1) / K::row_tile, each = a.Hkv * mt, t = blockIdx.x * n + threadIdx.x;
        if (threadIdx.x == 0) sc->shares = Shares{1, 0, s.nteams, 1};
        if ((int)threadIdx.x < n && t < s.nteams && !bad) {
            const int e = (unsigned)t / (unsigned)each;
            starts[threadIdx.x] = Start{e, t - e * each, 1, t};
        }
        __syncthreads();
        return pre;
    }
    const Sums y = add_up<K>(a, s, pre, sc, bad, len0);
    __syncthreads();
    const int all_u = all_units(sc);
    say_bad(a, s, bad, all_u < 0);
    share_out<K>(a, s, pre, y, all_u, starts, sc, blockIdx.x, gridDim.x);
    return pre;
}

// For a kernel some of whose CTAs take the prefixes (schedule sp) and the others the
// sequences (ss): how many take prefixes, the same in every CTA.  starts: room for
// either's teams; sc: two.
template <int D>
__device__ __forceinline__ int find_starts_beside(const Kv16Attn& a, const Kv16Sched& sp, const Kv16Sched& ss, Start* starts, Scan* sc, PreShared* ps,
                                                  Prefixes& pre)
{
    const int len0 = first_len(a, ss);
    if ((int)threadIdx.x < max(sp.per_cta, ss.per_cta)) starts[threadIdx.x].count = 0;
    const bool bad = look_over(a, ps, pre);
    const Sums yp = add_up<WideKind>(a, sp, pre, sc, bad, 0), ys = add_up<RowsKind>(a, ss, pre, sc + 1, bad, len0);
    __syncthreads();
    const int up = all_units(sc), us = all_units(sc + 1);
    say_bad(a, sp, bad, up < 0 || us < 0);
    // (units that do not fit are not worked on)
    const int ctas = wide_sms((float)max(up, 0), (float)max(us, 0), D);
    if ((int)blockIdx.x < ctas) share_out<WideKind>(a, sp, pre, yp, up, starts, sc, blockIdx.x, ctas);
    else share_out<RowsKind>(a, ss, pre, ys, us, starts, sc + 1, blockIdx.x - ctas, gridDim.x - ctas);
    return ctas;
}

// The run of one item's units that a team works on: tiles t0 .. t1 - 1 of KV
// head g's rows from r0 of entry e.
template <class K>
struct Run {
    Entry x;
    int e, item, whole, u0, u1, nu, t0, t1;
    int left;
    __device__ __forceinline__ void cut(int from)
    {
        nu = whole ? 1 : x.nu;
        u0 = from;
        u1 = min(nu, u0 + left);
        left -= u1 - u0;
        t0 = whole ? 0 : tile_at<K>(x, u0);
        t1 = whole ? x.tiles : tile_at<K>(x, u1);
        if (x.nu == 0) t0 = t1 = 0;  // (a direct team's sequence may be none)
    }
    __device__ __forceinline__ void begin(const Kv16Attn& a, const Kv16Sched& s, const Prefixes& pre, const Start& st, const Shares& h)
    {
        left = st.count, whole = h.whole, e = st.e;
        x = entry_of<K>(a, s, pre, e);
        const int n = whole ? 1 : x.nu;
        item = (unsigned)st.off / (unsigned)max(n, 1);
        cut(st.off - item * n);
    }
    __device__ __forceinline__ bool next(const Kv16Attn& a, const Kv16Sched& s, const Prefixes& pre)
    {
        if (left <= 0) return false;
        if (++item == a.Hkv * x.mt) {
            item = 0;
            do {
                if (++e >= s.n_pre + s.n_seq) return false;  // only if the lengths change under the call
                x = entry_of<K>(a, s, pre, e);
            } while (x.nu == 0);
        }
        cut(0);
        return true;
    }
    // all of the item's units: no other team has a part of it
    __device__ __forceinline__ bool all() const { return u0 == 0 && u1 == nu; }
    // which of the team's two parts it is: 1 begins an item, 0 goes on with one
    __device__ __forceinline__ int slot() const { return u0 == 0; }
    // leaves word of where the item's parts are, if it begins here (one thread)
    __device__ __forceinline__ void note(const Kv16Attn& a, const Kv16Sched& s, const Prefixes& pre, const Shares& h, int team) const
    {
        if (u0 != 0 || (s.finish && all())) return;
        const int g = item / x.mt, r0 = (item - g * x.mt) * K::row_tile;
        Kv16Item it;
        it.t0 = team, it.n = all() ? 1 : h.team_of(h.at(team + 1) + (nu - u1) - 1) - team + 1;
        it.row = x.row0 + r0, it.rows = min(K::row_tile, x.rows - r0), it.g = g;
        it.pre_row = x.b >= 0 && x.p >= 0 && !a.concat ? pre.first[x.p] * a.R : -1;
        if (s.finish) s.items[team] = it;
        else s.items[(size_t)((x.b >= 0) * a.Hkv + g) * a.B * a.R + it.row] = it;
    }
};

// Floats of a part and of the results of whole items.  A thread per row writes
// columns ([D + 2][rows]: outputs, M, sum), so that a warp's stores are lines;
// fragments of 8 rows x 4 lanes write rows ([rows][D], then [rows][M, sum]).
constexpr int kWideRows = WideKind::row_tile;  // in two tiles
__host__ __device__ constexpr size_t wide_part(int D) { return (size_t)2 * 128 * (D + 2); }
__host__ __device__ constexpr size_t rows_part(int D, int R) { return ((size_t)R * (D + 2) + 3) / 4 * 4; }  // (16-byte aligned)

}  // namespace

}  // namespace la
