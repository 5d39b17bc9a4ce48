// kv16_attn.cu -- the step's masked attention over the paged bf16 cache, for
// sequences that share prefixes: which kernels a call takes, and the merge of
// their parts.
//
// A row's keys are its prefix's tokens, its sequence's own and the step's rows
// that it sees: o = sum p_j v_j / sum p_j, p_j = exp2(s_j f - m) with f =
// log2(e) / sqrt(D) and m the running largest of s_j f.  Any two parts of the
// keys join by o = sum o_k 2^(m_k - m), l = sum l_k 2^(m_k - m).
#include <algorithm>
#include <mutex>

#include "kv16_sched.cuh"

namespace la {

bool kv16_rows_init();
int kv16_rows_teams();
cudaError_t launch_kv16_rows(cudaStream_t s, const Kv16Attn& a, const Kv16Sched& w, int D);
bool kv16_wide_init();
int kv16_wide_teams();
int launch_kv16_wide(cudaStream_t s, const Kv16Attn& a, const Kv16Sched& w, int D, int rows_all);

namespace {
// ------------------------------------------------------------------- merge ---

constexpr int kMergeRows = 8, kMergeThreads = 512;

struct Sum {
    float top, l, o[4];
    __device__ __forceinline__ void add(float m, float sum, const float (&v)[4])
    {
        const float t = fmaxf(top, m), f = ex2(top - t), h = ex2(m - t);
        top = t;
        l = l * f + sum * h;
#pragma unroll
        for (int i = 0; i < 4; i++) o[i] = o[i] * f + v[i] * h;
    }
};

// Row r of entry x and KV head g, of which every `step`-th part from `first`
// is added to y; false: nothing is to be done for this row (the item's team
// has written its output, or nobody works on it).
template <int D>
__device__ __forceinline__ bool add_parts(const Kv16Attn& a, const Kv16Sched& s, const float* whole, bool by_rows, int e, const Entry& x,
                                          int g, int r, int rows_all, int ch, int first, int step, Sum& y)
{
    const Kv16Shares h = *s.shares;
    if (h.nteams == 0 || x.nu == 0) return false;
    const int mt = r / s.row_tile, rr = r - mt * s.row_tile, nu = h.whole ? 1 : x.nu, gr = x.row0 + r;
    const long long u0 = s.base[e] + ((long long)g * x.mt + mt) * nu;
    const int t0 = team_of(h, u0), n = team_of(h, u0 + nu - 1) - t0 + 1;
    if (n == 1) {
        if (s.finish) return false;
        if (first) return true;
        float v[4];
        if (by_rows) {
            const size_t at = (size_t)g * rows_all + gr;
            const float4 o = *(const float4*)(whole + at * D + ch);
            const float2 ml = *(const float2*)(whole + (size_t)a.Hkv * rows_all * D + 2 * at);
            v[0] = o.x, v[1] = o.y, v[2] = o.z, v[3] = o.w;
            y.add(ml.x, ml.y, v);
        } else {
            const float* col = whole + (size_t)g * (D + 2) * rows_all + gr;
#pragma unroll
            for (int i = 0; i < 4; i++) v[i] = col[(size_t)(ch + i) * rows_all];
            y.add(col[(size_t)D * rows_all], col[(size_t)(D + 1) * rows_all], v);
        }
        return true;
    }
    constexpr int kBatch = 4;
#pragma unroll 1
    for (int k0 = first; k0 < n; k0 += kBatch * step) {
        float m[kBatch], l[kBatch], v[kBatch][4];
#pragma unroll
        for (int j = 0; j < kBatch; j++) {
            m[j] = kNoRef, l[j] = 0.f;
#pragma unroll
            for (int i = 0; i < 4; i++) v[j][i] = 0.f;
            const int k = k0 + j * step, t = t0 + k;
            if (k >= n) continue;
            const int f = (int)max(0LL, units_at(h, t) - u0), b = (int)min((long long)nu, units_at(h, t + 1) - u0);
            if (tile_at(s, x, b) <= tile_at(s, x, f)) continue;  // no keys, no part
            const size_t slot = (size_t)t * 2 + (f == 0);
            if (by_rows) {
                const float* part = s.slots + slot * rows_part(D, a.R);
                const float4 o = *(const float4*)(part + (size_t)rr * D + ch);
                const float2 ml = *(const float2*)(part + (size_t)a.R * D + 2 * rr);
                m[j] = ml.x, l[j] = ml.y, v[j][0] = o.x, v[j][1] = o.y, v[j][2] = o.z, v[j][3] = o.w;
            } else {
                const float* col = s.slots + slot * wide_part(D) + (rr >> 7) * (128 * (D + 2)) + (rr & 127);
                m[j] = col[D * 128], l[j] = col[(D + 1) * 128];
#pragma unroll
                for (int i = 0; i < 4; i++) v[j][i] = col[(ch + i) * 128];
            }
        }
#pragma unroll
        for (int j = 0; j < kBatch; j++) y.add(m[j], l[j], v[j]);
    }
    return true;
}

// A CTA: 8 rows of a KV head; a warp: 16 of their channels and every kGroups-th
// part (8 rows x 4 lanes of 4 channels: whole sectors of either kind of part).
template <int D>
__global__ void __launch_bounds__(kMergeThreads) k_kv16_merge(const __grid_constant__ Kv16Attn a, const __grid_constant__ Kv16Merge w)
{
    constexpr int kSlices = D / 16, kGroups = kMergeThreads / 32 / kSlices;
    __shared__ float sums[kGroups - 1][6][kSlices * 32];
    pdl_wait();
    pdl_trigger();
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, slice = warp % kSlices, part = warp / kSlices;
    const int gr = blockIdx.x * kMergeRows + (lane & 7), ch = slice * 16 + (lane >> 3) * 4, g = blockIdx.y;
    Sum y = {kNoRef, 0.f, {0.f, 0.f, 0.f, 0.f}};
    bool live = false;
    if (gr < w.rows_all) {
        const int b = gr / a.R, es = w.seq.n_pre + b;
        const Entry x = entry_of(a, w.seq, es);
        live = x.nu > 0 && add_parts<D>(a, w.seq, w.seq.whole, w.seq_rows, es, x, g, gr - x.row0, w.rows_all, ch, part, kGroups, y);
        if (live && w.pre.n_pre && x.p >= 0) {
            const Entry p = entry_of(a, w.pre, x.p);
            if (p.nu > 0) add_parts<D>(a, w.pre, w.pre.whole_pre, false, x.p, p, g, gr - p.row0, w.rows_all, ch, part, kGroups, y);
        }
    }
    if (!__syncthreads_or(live)) return;
    if (part) {
        float* to = &sums[part - 1][0][slice * 32 + lane];
        to[0] = y.top, to[kSlices * 32] = y.l;
#pragma unroll
        for (int i = 0; i < 4; i++) to[(2 + i) * kSlices * 32] = y.o[i];
    }
    __syncthreads();
    if (part || !live) return;
#pragma unroll
    for (int k = 0; k < kGroups - 1; k++) {
        const float* from = &sums[k][0][slice * 32 + lane];
        float v[4];
#pragma unroll
        for (int i = 0; i < 4; i++) v[i] = from[(2 + i) * kSlices * 32];
        y.add(from[0], from[kSlices * 32], v);
    }
    const float inv = 1.f / y.l;
    __nv_bfloat16* dst = a.out + ((size_t)(gr / a.group) * a.H + (size_t)g * a.group + gr % a.group) * D + ch;
    *(uint2*)dst = make_uint2(pack_bf16(y.o[0] * inv, y.o[1] * inv), pack_bf16(y.o[2] * inv, y.o[3] * inv));
}

// -------------------------------------------------------------------- plan ---

struct Plan {
    Kv16Attn k;
    Kv16Merge w;
    bool rows, wide, merge;
    size_t bytes;
};

// The call's kernels and where their parts are in a workspace at `ws` (or at 0: sizes alone).
Plan plan_of(const la_kv16_desc& c, const la_kv16_attn& a, uint8_t* ws)
{
    Plan p = {};
    Kv16Attn& k = p.k;
    k.B = a.batch, k.H = a.n_heads, k.Hkv = c.n_kv_heads;
    k.W = a.W, k.n1 = a.N - 1, k.T = 1 + (a.W + a.G) * k.n1;
    k.group = a.n_heads / c.n_kv_heads, k.R = k.T * k.group;
    k.n_pages = c.n_pages, k.max_pages = c.max_pages, k.page_log2 = log2_of(c.page);
    auto bound = [](int given, int room) { return given > 0 && given < room ? given : room; };
    k.max_len = bound(a.max_len, c.max_pages * c.page);
    k.nP = a.n_prefix, k.pp = a.prefix_pages;
    k.max_plen = a.n_prefix ? bound(a.max_prefix_len, a.prefix_pages * c.page) : 0;
    k.sl2 = 1.4426950408889634f / sqrtf((float)c.head_dim);
    k.concat = 1;
    const int D = c.head_dim;
    auto blocks = [](int n) { return (n + 15) / 16; };
    size_t at = 0;
    auto room = [&](size_t bytes) {
        uint8_t* x = ws + at;
        at += (bytes + 255) / 256 * 256;
        return x;
    };
    p.w.rows_all = k.B * k.R;
    const size_t all = (size_t)k.Hkv * p.w.rows_all * (D + 2) * 4;  // results of whole items
    // A prefix by itself, for all of its sequences at once, where reading it for each would cost
    // more than the further launches and parts (these bytes come from L2 at 8 TB/s: 2 us), and
    // where a sequence has too few rows to fill a tile.
    const long long again = (long long)k.B * k.Hkv * k.max_plen * D * 4;
    const bool apart = k.B > 1 && k.R <= 64 && again > (16 << 20);
    k.concat = !apart;
    p.rows = k.R <= 16;
    p.wide = !p.rows || apart;
    p.merge = apart;
    auto notes = [&](Kv16Sched& s, size_t part) {
        s.shares = (Kv16Shares*)room(sizeof(Kv16Shares)), s.base = (long long*)room(8 * (size_t)(s.n_pre + s.n_seq));
        s.slots = (float*)room((size_t)s.nteams * 2 * part);
    };
    if (p.wide) {
        Kv16Sched& s = p.w.pre;
        s.n_pre = apart ? k.nP : 0, s.n_seq = p.rows ? 0 : k.B;
        s.row_tile = kWideRows, s.blk_log2 = 3, s.wide = 128, s.extra = 4;
        s.nteams = kv16_wide_teams(), s.min_run = 6, s.slack = 12;
        s.finish = !apart, s.first = 1;
        const long long items = (long long)k.B * k.Hkv * ((k.R + kWideRows - 1) / kWideRows);
        const int most = (blocks(k.max_len) + blocks(k.max_plen) + blocks(k.T) + 7) / 8 * (k.R > 128 ? 2 : 1);
        if (!apart && items <= s.nteams && most <= s.slack) s.nteams = (int)items, s.slack = 1 << 30;
        else {
            p.merge = true;
            notes(s, wide_part(D) * 4);
        }
        if (apart) {
            s.whole_pre = (float*)room(all);
            if (!p.rows) s.whole = (float*)room(all);
        }
        if (!p.rows) p.w.seq = s;
        if (!apart) p.w.pre.n_pre = 0;
    }
    if (p.rows) {
        Kv16Sched& s = p.w.seq;
        s.n_seq = k.B, s.row_tile = 16, s.wide = 1 << 30, s.extra = 2;
        const long long items = (long long)k.B * k.Hkv;
        const int most = blocks(k.max_len) + blocks(k.max_plen) + 1;  // blocks of an item, at most
        s.nteams = kv16_rows_teams(), s.min_run = 16, s.slack = 16;
        s.finish = !apart, s.first = !apart;
        if (!apart && items <= s.nteams && most <= s.slack) s.nteams = (int)items, s.slack = 1 << 30;
        else {
            p.merge = true;
            notes(s, rows_part(D, k.R) * 4);
        }
        if (apart) s.whole = (float*)room(all);
        p.w.seq_rows = 1;
    }
    p.bytes = at;
    return p;
}

bool init()
{
    static std::once_flag once;
    static bool ok;
    std::call_once(once, [] { ok = kv16_rows_init() && kv16_wide_init(); });
    return ok;
}

}  // namespace

size_t kv16_attn_bytes(const la_kv16_desc& c, const la_kv16_attn& a) { return plan_of(c, a, nullptr).bytes; }

int launch_kv16_attn(cudaStream_t s, const la_kv16_desc& c, const la_kv16_attn& a)
{
    if (!init()) return LA_ERR_CUDA;
    Plan p = plan_of(c, a, (uint8_t*)a.workspace);
    Kv16Attn& k = p.k;
    k.q = (const __nv_bfloat16*)a.q, k.ks = (const __nv_bfloat16*)a.k_step, k.vs = (const __nv_bfloat16*)a.v_step;
    k.out = (__nv_bfloat16*)a.out;
    k.lens = a.lens, k.table = a.table, k.status = c.status;
    k.plens = a.prefix_lens, k.ptable = a.prefix_table, k.pfirst = a.prefix_first;
    k.kp = (const __nv_bfloat16*)c.k_pages, k.vp = (const __nv_bfloat16*)c.v_pages;
    k.q_ld = a.q_ld, k.k_ld = a.k_ld, k.v_ld = a.v_ld;
    const int D = c.head_dim;
    if (p.wide) {
        const int rc = launch_kv16_wide(s, k, p.w.pre, D, p.w.rows_all);
        if (rc != LA_OK) return rc;
    }
    cudaError_t e = cudaSuccess;
    if (p.rows) e = launch_kv16_rows(s, k, p.w.seq, D);
    if (e == cudaSuccess && p.merge) {
        const dim3 grid((p.w.rows_all + kMergeRows - 1) / kMergeRows, k.Hkv), block(kMergeThreads);
        e = D == 128 ? launch_pdl(k_kv16_merge<128>, grid, block, 0, s, k, p.w) : launch_pdl(k_kv16_merge<64>, grid, block, 0, s, k, p.w);
    }
    return e == cudaSuccess ? LA_OK : LA_ERR_CUDA;
}

}  // namespace la
