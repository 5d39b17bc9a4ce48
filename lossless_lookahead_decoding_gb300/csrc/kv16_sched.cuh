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

__device__ __forceinline__ void fence_acquire() { asm volatile("fence.acq_rel.gpu;" ::: "memory"); }

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

// An entry; n: the sequence's own tokens (not looked at for a prefix's entry).
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
    x.wide = x.rows > s.wide;
    x.tiles = (x.nb + (1 << s.blk_log2) - 1) >> s.blk_log2;
    x.mt = (x.rows + s.row_tile - 1) / s.row_tile;
    x.nu = x.rows ? s.extra + (x.tiles << x.wide) : 0;
    return x;
}

__device__ __forceinline__ Entry entry_of(const Kv16Attn& a, const Kv16Sched& s, const Prefixes& pre, int e)
{
    return entry_with(a, s, pre, e, e < s.n_pre ? 0 : a.lens[e - s.n_pre]);
}

// The first tile at or behind unit u of an item.
__device__ __forceinline__ int tile_at(const Kv16Sched& s, const Entry& x, int u) { return max(u - s.extra + x.wide, 0) >> x.wide; }

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
    int units[32], big[32], cost[32], items[32], top[32];
    Shares shares;
};

// Of two kernels that run at the same time, the SMs of the wide one: with uw units
// (a tile for a stream: 32 KB of a pair's tile, 0.95 us) and ur blocks (8 KB at D =
// 128, 0.126 us at what one SM can read) both end together.  Where HBM and not the
// SMs sets the pace, a wide unit waits for its tiles and takes 1.73 us.  (128 single
// tokens behind 1000, us in all, at 1.0, 1.4, 1.73 and 2.4 us a unit: 77, 67, 65, 64;
// 48 behind prefixes of up to 4000: 61, 56, 54, 56; one kernel after the other, the
// former: 89.)
__device__ __forceinline__ int wide_sms(float uw, float ur, int D)
{
    const float half = D == 128 ? 1.f : 0.6f, tw = 0.95f * half, tr = 0.126f * half;
    const float hbm = (uw * 32.f + ur * 8.f) * (D / 128.f) / 6600.f;
    const bool waits = hbm > (uw * tw + ur * tr) / kSMs;
    const float w = uw * (waits ? 1.73f * half : tw), r = ur * tr;
    return min(max((int)(w * kSMs / fmaxf(w + r, 1e-3f)) + 1, 4), kSMs - 8);
}

// Where each of the CTA's teams begins; the shares go to sc.  CTA 0 of the
// call's first kernel raises what is wrong with the sequences.
template <int D>
__device__ Prefixes find_starts(const Kv16Attn& a, const Kv16Sched& s, Start* starts, Scan* sc, PreShared* ps)
{
    const int n = s.per_cta, entries = s.n_pre + s.n_seq;
    const int per = entries <= (int)blockDim.x ? 1 : ceil_div(entries, (int)blockDim.x), e0 = threadIdx.x * per, e1 = min(e0 + per, entries);
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, nw = blockDim.x >> 5;
    // ---- all loads at once
    const int len0 = !s.direct && e0 < e1 && e0 >= s.n_pre ? a.lens[e0 - s.n_pre] : 0;
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
    if (blockIdx.x == 0 && s.first) {
        for (int b = threadIdx.x; b < a.B; b += blockDim.x) wrong |= a.lens[b] > a.max_len;
        if (wrong || bad) kv4_raise(a.status, LA_ERR_ARG);
    }
    const Prefixes pre = fits ? Prefixes{ps->first, ps->lens} : Prefixes{a.pfirst, a.plens};
    if ((int)threadIdx.x < n) starts[threadIdx.x].count = 0;
    bad = __syncthreads_or(bad);
    if (s.direct) {
        const int mt = (a.R + s.row_tile - 1) / s.row_tile, each = a.Hkv * mt, t = blockIdx.x * n + threadIdx.x;
        if (threadIdx.x == 0) sc->shares = Shares{1, 0, s.nteams, 1};
        if ((int)threadIdx.x < n && t < s.nteams && !bad) {
            const int e = (unsigned)t / (unsigned)each;
            starts[threadIdx.x] = Start{e, t - e * each, 1, t};
        }
        __syncthreads();
        return pre;
    }
    long long sum = 0;
    int items = 0, top = 0, cost = 0;
    Entry x0;
    x0.mt = x0.nu = 0;
    if (!bad) {
        for (int e = e0; e < e1; e++) {
            const Entry x = entry_with(a, s, pre, e, e == e0 || e < s.n_pre ? len0 : a.lens[e - s.n_pre]);
            const int k = a.Hkv * x.mt;
            if (e == e0) x0 = x;
            if (x.nu) sum += (long long)k * x.nu, items = min(items + k, 1 << 20), top = max(top, x.nu);
            else if (!s.finish && x.b >= 0 && blockIdx.x == 0)
                // no rows, which the merge is to know
                for (int g = 0; g < a.Hkv; g++) s.items[(size_t)(a.Hkv + g) * a.B * a.R + x.row0].n = 0;
        }
        if (s.beside) {
            // the other kernel's work, by KV heads
            if (s.n_pre)
                for (int b = threadIdx.x; b < a.B; b += blockDim.x) cost += blocks_of(min(max(a.lens[b], 0), a.max_len)) + 3;
            else
                for (int p = threadIdx.x; p < a.nP; p += blockDim.x) {
                    const int rows = (pre.first[p + 1] - pre.first[p]) * a.R, m = min(max(pre.lens[p], 0), a.max_plen);
                    cost += (rows + 255) / 256 * (4 + ((blocks_of(m) + 7) / 8 << (rows > 128)));
                }
        }
    }
    const int units = (int)min(sum, 0x7fff0000LL);  // (there, or nothing is done: see `huge`)
    int xu = units;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int y = __shfl_up_sync(0xffffffffu, xu, o);
        if (lane >= o) xu += y;
    }
    {
        const int w_big = __reduce_add_sync(0xffffffffu, (int)min(sum >> 16, 1LL << 20)), w_cost = __reduce_add_sync(0xffffffffu, cost),
                  w_items = __reduce_add_sync(0xffffffffu, items), w_top = __reduce_max_sync(0xffffffffu, top);
        if (lane == 31) sc->units[warp] = xu, sc->big[warp] = w_big, sc->items[warp] = w_items, sc->top[warp] = w_top, sc->cost[warp] = w_cost;
    }
    __syncthreads();
    const bool in = lane < nw;
    const int u = in ? sc->units[lane] : 0, it = in ? sc->items[lane] : 0;
    const int before = __reduce_add_sync(0xffffffffu, lane < warp ? u : 0) + xu - units, all_u = __reduce_add_sync(0xffffffffu, u);
    const int all_i = __reduce_add_sync(0xffffffffu, it);
    top = __reduce_max_sync(0xffffffffu, in ? sc->top[lane] : 0);
    const bool huge = __reduce_add_sync(0xffffffffu, in ? sc->big[lane] : 0) >= 0x7000;
    if (huge && blockIdx.x == 0 && threadIdx.x == 0) kv4_raise(a.status, LA_ERR_ARG);
    if (s.bad && blockIdx.x == 0 && threadIdx.x == 0) *s.bad = bad || huge;
    int ctas = gridDim.x;
    if (s.beside) {
        // (both kernels count alike)
        const float mine = (float)all_u, other = (float)__reduce_add_sync(0xffffffffu, in ? sc->cost[lane] : 0) * (float)a.Hkv;
        const int sms = s.n_pre ? wide_sms(mine, other, D) : wide_sms(other, mine, D);
        ctas = s.n_pre ? sms : kSMs - sms;
    }
    const int room = min(s.nteams, ctas * n);
    Shares h;
    // Whole items leave no parts: worth `slack` units of the longest team's work.
    h.whole = all_i <= 4 * room && ceil_div(all_i, room) * top - s.slack <= (int)((unsigned)all_u / (unsigned)room);
    int bi = 0;
    if (h.whole) {
        // the same for whole items
        int xi = items;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int y = __shfl_up_sync(0xffffffffu, xi, o);
            if (lane >= o) xi += y;
        }
        bi = xi - items + __reduce_add_sync(0xffffffffu, lane < warp ? it : 0);
    }
    const int all = huge ? 0 : h.whole ? all_i : all_u;
    h.nteams = all == 0 ? 0 : h.whole ? min(all_i, room) : min(room, max(1, (int)((unsigned)all / (unsigned)s.min_run)));
    h.q = h.nteams ? (int)((unsigned)all / (unsigned)h.nteams) : 0;
    h.r = all - h.q * h.nteams;
    if (threadIdx.x == 0) sc->shares = h;
    if (h.nteams && units) {
        int at = h.whole ? bi : before;
        const int end = at + (h.whole ? items : units);
        // the CTAs' teams by turns: few teams are spread over the SMs
        int i = 0;
        auto team = [&](int j) { return j * ctas + (int)blockIdx.x; };
        // the teams that begin within this thread's entries
        while (i < n && (int)blockIdx.x < ctas && team(i) < h.nteams && h.at(team(i)) < at) i++;
        if (i < n && (int)blockIdx.x < ctas && team(i) < h.nteams && h.at(team(i)) < end)
            for (int e = e0; e < e1; e++) {
                const Entry x = e == e0 ? x0 : entry_of(a, s, pre, e);
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
    return pre;
}

// The run of one item's units that a team works on: tiles t0 .. t1 - 1 of KV
// head g's rows from r0 of entry e.
struct Run {
    Entry x;
    int e, item, whole, u0, u1, nu, t0, t1;
    int left;
    __device__ __forceinline__ void cut(const Kv16Sched& s, int from)
    {
        nu = whole ? 1 : x.nu;
        u0 = from;
        u1 = min(nu, u0 + left);
        left -= u1 - u0;
        t0 = whole ? 0 : tile_at(s, x, u0);
        t1 = whole ? x.tiles : tile_at(s, x, u1);
        if (x.nu == 0) t0 = t1 = 0;  // (a direct team's sequence may be none)
    }
    __device__ __forceinline__ void begin(const Kv16Attn& a, const Kv16Sched& s, const Prefixes& pre, const Start& st, const Shares& h)
    {
        left = st.count, whole = h.whole, e = st.e;
        x = entry_of(a, s, pre, e);
        const int n = whole ? 1 : x.nu;
        item = (unsigned)st.off / (unsigned)max(n, 1);
        cut(s, st.off - item * n);
    }
    __device__ __forceinline__ bool next(const Kv16Attn& a, const Kv16Sched& s, const Prefixes& pre)
    {
        if (left <= 0) return false;
        if (++item == a.Hkv * x.mt) {
            item = 0;
            do {
                if (++e >= s.n_pre + s.n_seq) return false;  // only if the lengths change under the call
                x = entry_of(a, s, pre, e);
            } while (x.nu == 0);
        }
        cut(s, 0);
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
        const int g = item / x.mt, r0 = (item - g * x.mt) * s.row_tile;
        Kv16Item it;
        it.t0 = team, it.n = all() ? 1 : h.team_of(h.at(team + 1) + (nu - u1) - 1) - team + 1;
        it.row = x.row0 + r0, it.rows = min(s.row_tile, x.rows - r0), it.g = g;
        it.pre_row = x.b >= 0 && x.p >= 0 && !a.concat ? pre.first[x.p] * a.R : -1;
        if (s.finish) s.items[team] = it;
        else s.items[(size_t)((x.b >= 0) * a.Hkv + g) * a.B * a.R + it.row] = it;
    }
};

// Floats of a part and of the results of whole items.  A thread per row writes
// columns ([D + 2][rows]: outputs, M, sum), so that a warp's stores are lines;
// fragments of 8 rows x 4 lanes write rows ([rows][D], then [rows][M, sum]).
constexpr int kWideRows = 256;   // rows of an item of k_kv16_wide, in two tiles
__host__ __device__ constexpr size_t wide_part(int D) { return (size_t)2 * 128 * (D + 2); }
__host__ __device__ constexpr size_t rows_part(int D, int R) { return ((size_t)R * (D + 2) + 3) / 4 * 4; }  // (16-byte aligned)

}  // namespace

}  // namespace la
