// kv16_attn.cu -- the step's masked attention over the paged bf16 cache, for
// sequences that share prefixes: which kernels a call takes, and the merge of
// their parts.
//
// A row's keys are its prefix's tokens, its sequence's own and the step's rows
// that it sees: o = sum p_j v_j / sum p_j, p_j = exp2((s_j - m) f) with f =
// log2(e) / sqrt(D) and m one of the s_j, about the largest.  Any two parts of the
// keys join by o = sum o_k exp2((m_k - m) f), l = sum l_k exp2((m_k - m) f).
// (Scores are subtracted before they are scaled: m f in fp32 is off by up to 2^-24 of
// itself, at 2^31 more than exp2 can hold.)
#include <algorithm>
#include <mutex>

#include "kv16_sched.cuh"

namespace la {

bool kv16_rows_init();
int kv16_rows_teams();
cudaError_t launch_kv16_rows(cudaStream_t s, const Kv16Attn& a, const Kv16Sched& w, int D);
bool kv16_wide_init();
int kv16_wide_teams();
int kv16_beside_teams();
int launch_kv16_wide(cudaStream_t s, const Kv16Attn& a, const Kv16Sched& w, const Kv16Sched* beside, int D, int rows_all);

namespace {
// ------------------------------------------------------------------- merge ---

struct MergeArgs {
    Kv16Attn a;
    const Kv16Item* items;
    const int* bad;
    const float *slots_pre, *slots_seq, *whole_pre, *whole_seq;
    int rows_pre_tile;        // rows of a prefix's item
    int by_rows;              // sequences' parts are rows (k_kv16_rows), else columns
    int teams, teams_pre;     // that may have parts (nothing else is read, whatever a workspace holds)
    int chunks;               // groups of rows of an item
};

template <int C>
struct Sum {
    float top = kNoRef, l = 0.f, o[C] = {};
    __device__ __forceinline__ void add(float sl2, float m, float sum, const float (&v)[C])
    {
        const float t = fmaxf(top, m), f = ex2((top - t) * sl2), h = ex2((m - t) * sl2);
        top = t;
        l = l * f + sum * h;
#pragma unroll
        for (int i = 0; i < C; i++) o[i] = o[i] * f + v[i] * h;
    }
};

// Row r's M, sum and C channels from ch, of a part or of whole items' results:
// columns `pitch` apart, or rows (of which there are `rows`).
template <int D, int C>
__device__ __forceinline__ void load_cols(const float* col, size_t pitch, int ch, float& m, float& l, float (&v)[C])
{
    m = col[D * pitch], l = col[(D + 1) * pitch];
#pragma unroll
    for (int i = 0; i < C; i++) v[i] = col[(ch + i) * pitch];
}
template <int D, int C>
__device__ __forceinline__ void load_rows(const float* part, size_t r, size_t rows, int ch, float& m, float& l, float (&v)[C])
{
#pragma unroll
    for (int i = 0; i < C; i += 4) *(float4*)(v + i) = *(const float4*)(part + r * D + ch + i);
    const float2 ml = *(const float2*)(part + rows * D + 2 * r);
    m = ml.x, l = ml.y;
}

// Of the parts of teams t0 .. t0 + n - 1, every `step`-th from `first` is added
// to y: row r of their item, channels ch .. ch + C - 1.  kBatch parts are on
// their way at once.
template <int D, int C, int kBatch>
__device__ __forceinline__ void add_parts(const Kv16Attn& a, const float* slots, bool by_rows, int t0, int n, int r, int ch, int first, int step, Sum<C>& y)
{
#pragma unroll 1
    for (int k0 = first; k0 < n; k0 += kBatch * step) {
        float m[kBatch], l[kBatch], v[kBatch][C];
#pragma unroll
        for (int j = 0; j < kBatch; j++) {
            const int k = k0 + j * step;
            const size_t slot = (size_t)(t0 + k) * 2 + (k == 0);
            m[j] = kNoRef, l[j] = 0.f;
#pragma unroll
            for (int i = 0; i < C; i++) v[j][i] = 0.f;
            if (k < n) {
                if (by_rows) load_rows<D, C>(slots + slot * rows_part(D, a.R), r, a.R, ch, m[j], l[j], v[j]);
                else load_cols<D, C>(slots + slot * wide_part(D) + (r >> 7) * (128 * (D + 2)) + (r & 127), 128, ch, m[j], l[j], v[j]);
            }
        }
#pragma unroll
        for (int j = 0; j < kBatch; j++) {
            // (a part without keys has no outputs, whatever is in their place)
            const bool none = m[j] == kNoRef && l[j] == 0.f;
#pragma unroll
            for (int i = 0; i < C; i++) v[j][i] = none ? 0.f : v[j][i];
            y.add(a.sl2, m[j], l[j], v[j]);
        }
    }
}

template <int D, int C>
__device__ __forceinline__ void put_row(const Kv16Attn& a, const Sum<C>& y, int g, int gr, int ch)
{
    const float inv = 1.f / y.l;
    uint32_t z[C / 2];
#pragma unroll
    for (int i = 0; i < C; i += 2) z[i / 2] = pack_bf16(y.o[i] * inv, y.o[i + 1] * inv);
    __nv_bfloat16* dst = a.out + ((size_t)(gr / a.group) * a.H + (size_t)g * a.group + gr % a.group) * D + ch;
    if (C == 8) *(uint4*)dst = make_uint4(z[0], z[1], z[C / 2 - 2], z[C / 2 - 1]);
    else *(uint2*)dst = make_uint2(z[0], z[1]);
}

// Joins the parts of items that several teams hold.  CTAs go through teams and
// groups of rows by turns, the next item's record on its way.  kRowParts: 8 rows
// x all channels, a warp 8 rows x 4 lanes of 4 channels (whole sectors of rows);
// else 32 rows x 64 channels, a warp 32 rows x 8 channels (lines of columns).  Bound
// by two dependent trips, record and parts: 35 MB of parts take 10 us behind the
// kernel that wrote them, none 5 us.
constexpr int kMergeThreads = 256;
template <int D, bool kRowParts>
__global__ void __launch_bounds__(kMergeThreads) k_kv16_merge(const __grid_constant__ MergeArgs w)
{
    constexpr int C = kRowParts ? 4 : 8, kHigh = kRowParts ? 8 : 32, kSlices = kRowParts ? 1 : D / 64;
    pdl_wait();
    pdl_trigger();
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, each = w.chunks * kSlices, all = w.teams * each;
    auto record = [&](int i) { return i < all ? w.items[i / each] : Kv16Item{}; };
    Kv16Item next = record(blockIdx.x);
#pragma unroll 1
    for (int i = blockIdx.x; i < all; i += gridDim.x) {
        const Kv16Item it = next;
        next = record(i + gridDim.x);
        const int part = i % each, r0 = part / kSlices * kHigh;
        if (it.n <= 0 || it.t0 < 0 || it.n > w.teams - it.t0 || r0 >= it.rows) continue;
        const int r = r0 + (kRowParts ? lane & 7 : lane), ch = kRowParts ? warp * 16 + (lane >> 3) * 4 : part % kSlices * 64 + warp * 8;
        if (r >= it.rows || ch >= D) continue;
        Sum<C> y;
        add_parts<D, C, kRowParts ? 4 : 2>(w.a, w.slots_seq, kRowParts, it.t0, it.n, r, ch, 0, 1, y);
        put_row<D, C>(w.a, y, it.g, it.row + r, ch);
    }
}

// Joins every row's own keys and its prefix's.  A CTA: 32 rows of a KV head x 64
// channels; a warp 8 of them and every groups-th part.  (128 sequences, 32 heads:
// 14 MB from L2, 7.6 us by itself.)
constexpr int kMaxGroups = 4;
template <int D>
__global__ void __launch_bounds__(256 * kMaxGroups) k_kv16_join(const __grid_constant__ MergeArgs w)
{
    __shared__ float sums[kMaxGroups - 1][10][256];
    pdl_wait();
    pdl_trigger();
    const Kv16Attn& a = w.a;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, part = warp >> 3, groups = blockDim.x >> 8, at = threadIdx.x & 255;
    const int gr = blockIdx.x * 32 + lane, ch = blockIdx.z * 64 + (warp & 7) * 8, g = blockIdx.y, rows_all = a.B * a.R;
    Sum<8> y;
    bool live = gr < rows_all;
    if (live) {
        const int row0 = gr / a.R * a.R;
        const Kv16Item it = w.items[(size_t)(a.Hkv + g) * rows_all + row0];
        live = !*w.bad && it.n > 0 && it.t0 >= 0 && it.n <= w.teams - it.t0;
        if (live) {
            float m, l, v[8];
            const bool shared = it.pre_row >= 0 && it.pre_row <= gr;
            Kv16Item p = {};
            int first = 0;
            if (shared) {
                first = it.pre_row + (gr - it.pre_row) / w.rows_pre_tile * w.rows_pre_tile;
                p = w.items[(size_t)g * rows_all + first];
            }
            if (it.n > 1) {
                add_parts<D, 8, 2>(a, w.slots_seq, w.by_rows, it.t0, it.n, gr - row0, ch, part, groups, y);
            } else if (part == 0) {
                if (w.by_rows) load_rows<D, 8>(w.whole_seq, (size_t)g * rows_all + gr, (size_t)a.Hkv * rows_all, ch, m, l, v);
                else load_cols<D, 8>(w.whole_seq + (size_t)g * (D + 2) * rows_all + gr, rows_all, ch, m, l, v);
                y.add(a.sl2, m, l, v);
            }
            if (shared && p.n > 1 && p.t0 >= 0 && p.n <= w.teams_pre - p.t0) {
                add_parts<D, 8, 3>(a, w.slots_pre, false, p.t0, p.n, gr - first, ch, part, groups, y);
            } else if (shared && part == groups - 1) {
                load_cols<D, 8>(w.whole_pre + (size_t)g * (D + 2) * rows_all + gr, rows_all, ch, m, l, v);
                y.add(a.sl2, m, l, v);
            }
        }
    }
    if (part) {
        float* to = &sums[part - 1][0][at];
        to[0] = y.top, to[256] = y.l;
#pragma unroll
        for (int i = 0; i < 8; i++) to[(2 + i) * 256] = y.o[i];
    }
    if (groups > 1) __syncthreads();
    if (part || !live) return;
#pragma unroll 1
    for (int k = 0; k < groups - 1; k++) {
        const float* from = &sums[k][0][at];
        float v[8];
#pragma unroll
        for (int i = 0; i < 8; i++) v[i] = from[(2 + i) * 256];
        y.add(a.sl2, from[0], from[256], v);
    }
    put_row<D, 8>(a, y, g, gr, ch);
}

// -------------------------------------------------------------------- plan ---

struct Plan {
    Kv16Attn k;
    Kv16Sched wide, rows;
    MergeArgs m;
    bool use_wide, use_rows, apart, merge;
    int groups;  // of the merge
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
    const int D = c.head_dim, rows_all = k.B * k.R;
    auto blocks = [](int n) { return (n + 15) / 16; };
    size_t at = 0;
    auto room = [&](size_t bytes) {
        uint8_t* x = ws + at;
        at += (bytes + 255) / 256 * 256;
        return x;
    };
    // A prefix by itself, for all of its sequences at once, where reading it for each would cost
    // more than the further launch and parts (these bytes come from L2 at 8 TB/s: 2 us), and
    // where a sequence has too few rows to fill a tile.  Both ways, in us, 8 KV heads over 50 to
    // 600 tokens at D 128: 32 sequences behind 4000, with 8, 17, 32, 64 and 80 rows each, 28, 40,
    // 46, 59, 70 by itself and 68, 67, 67, 70, 74 with each; behind 1000 24, 33, 36, 41, 45 and 32,
    // 36, 36, 37, 39; 2 behind 4000, 8 and 64 rows, 20, 19 and 26, 20, behind 1000 (8 MB) 20, 18
    // and 18, 18.  With 100 rows of each of 6 prompts behind 1024 56 against 44, with 456 of 8
    // steps 160 against 130.  (The table's width stands for the prefixes' lengths, which are on
    // the device, and any number of prefixes for one.)
    const long long again = (long long)k.B * k.Hkv * k.max_plen * D * 4;
    p.apart = k.B > 1 && k.R <= 64 && again > (16 << 20);
    k.concat = !p.apart;
    // k_kv16_rows holds up to 16 rows.  The other kernel for these, 8 KV heads at D 128, 8 rows: 200
    // sequences of 20 to 300 tokens 81 us and here 33, 32 of 500 to 4000 54 and 56, 4 of 4000 20 and
    // 28 (more parts to join here); at 16 rows 81, 54, 20 and 40, 61, 32.
    p.use_rows = k.R <= 16;
    p.use_wide = !p.use_rows || p.apart;
    // ---- who begins where
    const int most = blocks(k.max_len) + (p.apart ? 0 : blocks(k.max_plen)) + blocks(k.T);  // blocks of a sequence, at most
    if (p.use_wide) {
        Kv16Sched& s = p.wide;
        s.n_pre = p.apart ? k.nP : 0, s.n_seq = p.use_rows ? 0 : k.B;
        s.nteams = kv16_wide_teams(), s.per_cta = 1;
        const long long items = (long long)k.B * k.Hkv * ((k.R + kWideRows - 1) / kWideRows);
        if (!p.apart && items <= s.nteams && (most + 7) / 8 * (k.R > WideKind::twice ? 2 : 1) <= WideKind::slack) s.nteams = (int)items, s.direct = 1;
    }
    if (p.use_rows) {
        Kv16Sched& s = p.rows;
        s.n_seq = k.B;
        const long long items = (long long)k.B * k.Hkv;
        s.nteams = p.apart ? kv16_beside_teams() : kv16_rows_teams(), s.per_cta = s.nteams / kSMs;
        if (!p.apart && items <= s.nteams && most <= RowsKind::slack) s.nteams = (int)items, s.direct = 1;
    }
    // ---- where their results go
    Kv16Sched& last = p.use_rows ? p.rows : p.wide;
    const size_t all = (size_t)k.Hkv * rows_all * (D + 2) * 4;  // results of whole items
    if (p.apart) {
        p.m.bad = (int*)room(4);
        p.m.items = (Kv16Item*)room(2 * (size_t)k.Hkv * rows_all * sizeof(Kv16Item));
        p.m.whole_pre = (float*)room(all), p.m.whole_seq = (float*)room(all);
    } else {
        if (!last.direct) p.m.items = (Kv16Item*)room(last.nteams * sizeof(Kv16Item));
        last.finish = 1;
    }
    if (p.use_wide && !p.wide.direct) p.wide.slots = (float*)room((size_t)p.wide.nteams * 2 * wide_part(D) * 4);
    if (p.use_rows && !p.rows.direct) p.rows.slots = (float*)room((size_t)p.rows.nteams * 2 * rows_part(D, k.R) * 4);
    for (Kv16Sched* s : {&p.wide, &p.rows}) {
        s->items = (Kv16Item*)p.m.items;
        if (p.apart) s->bad = (int*)p.m.bad;
        s->whole = (float*)p.m.whole_seq, s->whole_pre = (float*)p.m.whole_pre;
    }
    p.m.slots_pre = p.wide.slots, p.m.slots_seq = last.slots;
    p.m.rows_pre_tile = kWideRows, p.m.by_rows = p.use_rows;
    p.merge = !last.direct;
    p.m.teams = last.nteams, p.m.teams_pre = p.wide.nteams, p.m.chunks = (std::min(p.use_rows ? RowsKind::row_tile : WideKind::row_tile, k.R) + (p.use_rows ? 7 : 31)) / (p.use_rows ? 8 : 32);
    // as many groups of warps as an item may have fours of parts
    const long long parts = (p.use_wide ? p.wide.nteams : p.rows.nteams) / std::max(1LL, (long long)k.Hkv * (p.apart ? (rows_all + 255) / 256 : k.B));
    p.groups = parts >= 9 ? 4 : parts >= 4 ? 2 : 1;
    p.bytes = at;
    return p;
}

template <int D>
cudaError_t launch_merge(cudaStream_t s, const Plan& p)
{
    if (p.apart) return launch_pdl(k_kv16_join<D>, dim3((p.k.B * p.k.R + 31) / 32, p.k.Hkv, D / 64), dim3(256 * p.groups), 0, s, p.m);
    const long long all = (long long)p.m.teams * p.m.chunks * (p.use_rows ? 1 : D / 64);
    const dim3 grid((unsigned)std::min(all, (long long)kSMs * 6));
    return p.use_rows ? launch_pdl(k_kv16_merge<D, true>, grid, dim3(kMergeThreads), 0, s, p.m)
                      : launch_pdl(k_kv16_merge<D, false>, grid, dim3(kMergeThreads), 0, s, p.m);
}

std::mutex g_mu;
unsigned char g_ready[256];

// The kernels' shared-memory limits, once per device.
bool attn_ready()
{
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 256) return false;
    std::lock_guard<std::mutex> lock(g_mu);
    if (!g_ready[dev]) g_ready[dev] = kv16_rows_init() && kv16_wide_init();
    return g_ready[dev] != 0;
}

}  // namespace

size_t kv16_attn_bytes(const la_kv16_desc& c, const la_kv16_attn& a) { return plan_of(c, a, nullptr).bytes; }

int launch_kv16_attn(cudaStream_t s, const la_kv16_desc& c, const la_kv16_attn& a)
{
    if (!attn_ready()) return LA_ERR_CUDA;
    Plan p = plan_of(c, a, (uint8_t*)a.workspace);
    Kv16Attn& k = p.k;
    k.q = (const __nv_bfloat16*)a.q, k.ks = (const __nv_bfloat16*)a.k_step, k.vs = (const __nv_bfloat16*)a.v_step;
    k.out = (__nv_bfloat16*)a.out;
    k.lens = a.lens, k.table = a.table, k.status = c.status;
    k.plens = a.prefix_lens, k.ptable = a.prefix_table, k.pfirst = a.prefix_first;
    k.kp = (const __nv_bfloat16*)c.k_pages, k.vp = (const __nv_bfloat16*)c.v_pages;
    k.q_ld = a.q_ld, k.k_ld = a.k_ld, k.v_ld = a.v_ld;
    p.m.a = k;
    const int D = c.head_dim;
    if (p.use_wide) {
        const int rc = launch_kv16_wide(s, k, p.wide, p.use_rows ? &p.rows : nullptr, D, k.B * k.R);
        if (rc != LA_OK) return rc;
    }
    cudaError_t e = p.use_rows && !p.use_wide ? launch_kv16_rows(s, k, p.rows, D) : cudaSuccess;
    if (e == cudaSuccess && p.merge) e = D == 128 ? launch_merge<128>(s, p) : launch_merge<64>(s, p);
    return e == cudaSuccess ? LA_OK : LA_ERR_CUDA;
}

}  // namespace la
