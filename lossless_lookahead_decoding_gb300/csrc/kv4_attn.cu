// kv4_attn.cu -- the step's masked attention over the paged 4-bit cache for
// few rows per KV head, on mma.sync: decode steps of single tokens, small
// lookahead steps, grouped heads.
//
// For one sequence and KV head ("item") the rows are the T step rows times the
// query heads that share the KV head, in tiles of 8 NB rows.  With a key's
// parameters s, z and codes c:
//   S = q . (c - z) s = s (q . (128 + c) - (128 + z) sum q)
//   O = sum_keys p (c - z) s = sum_keys (p s) (c - z)
// so scales multiply the few scores and probabilities and not the many codes.
// K's codes go to the tensor core as 128 + c, the form the unpacking gives
// for free; the sum over q is subtracted in fp32, where 128 |q| costs 2^-16 of
// a code step.  V's would lose more (O shrinks as the context grows, 128 sum p
// does not), so 128 + z is subtracted from each pair of codes: exact.
// Rounding: p s to bf16 (relative 2^-9 a key, unbiased), then the output;
// scores, sums and outputs stay in fp32.
//
// Both products have the keys (K: 16 keys x 16 channels) or the channels (V:
// 16 channels x 16 keys) as the 16-row side of m16n8k16 and the query rows as
// the 8-wide side: a single token of a group of up to 8 heads fills it, and
// the probabilities go from one product's accumulators to the other's operand
// by an 8 x 8 transpose in registers.  Channels and keys are permuted so that
// each lane's fragments are contiguous bytes (kv4_key).
//
// HBM bound: 2 D / 2 + 8 bytes a key and KV head.  Each warp streams blocks of
// 16 keys (one contiguous bulk copy each) into a ring of its own, so no warp
// waits for another inside an item.  The running maximum moves only when a
// score exceeds it by more than 8 (a vote, no reduction per tile): the sums
// then hold terms up to 2^8.
//
// Items are cut into equal runs of blocks over the teams (a warp, or a CTA of
// 8 warps whose partial results meet in shared memory), whatever the
// sequences' lengths; an item that falls to several teams leaves partial
// outputs, which k_kv4_merge joins in a fixed order.
#include <algorithm>
#include <climits>
#include <cmath>
#include <mutex>

#include "kv4.cuh"

namespace la {

namespace {

using namespace ptx;

constexpr int kWarps = 8;
constexpr int kSMs = 152;

// The key of a tile held in row i of a score fragment (and in slot i of the
// probabilities): with these, the four keys whose V a lane reads at once lie
// in different 32-byte rows modulo 128 bytes, and so do the K rows of a
// quarter warp.
__device__ __forceinline__ int kv4_key(int i)
{
    const int h = (i >> 1) & 3;
    return (i & 8) + ((i & 1) ? 4 + (h ^ 3) : h);
}

__device__ __forceinline__ void bulk_load(void* dst, const void* src, uint32_t bytes, uint64_t* bar, uint64_t pol)
{
    asm volatile(
        "cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes.L2::cache_hint [%0], [%1], %2, [%3], %4;" ::"r"(
            smem_u32(dst)),
        "l"(src), "r"(bytes), "r"(smem_u32(bar)), "l"(pol)
        : "memory");
}

__device__ __forceinline__ void mma16816(float* d, uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                         uint32_t b1)
{
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

__device__ __forceinline__ uint32_t transpose8(uint32_t x)
{
    uint32_t y;
    asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
    return y;
}

__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi)
{
    __nv_bfloat162 v = __floats2bfloat162_rn(lo, hi);
    return *reinterpret_cast<uint32_t*>(&v);
}

__device__ __forceinline__ uint32_t sub_bf16x2(uint32_t a, uint32_t b)
{
    __nv_bfloat162 v = __hsub2(*reinterpret_cast<__nv_bfloat162*>(&a), *reinterpret_cast<__nv_bfloat162*>(&b));
    return *reinterpret_cast<uint32_t*>(&v);
}

// bf16 pair with its NaNs and infinities replaced by 0; whether there were any
__device__ __forceinline__ bool drop_nonfinite(uint32_t& u)
{
    const bool lo = (u & 0x7f80u) == 0x7f80u, hi = (u & 0x7f800000u) == 0x7f800000u;
    if (lo) u &= 0xffff0000u;
    if (hi) u &= 0x0000ffffu;
    return lo || hi;
}

// two codes at bits 4i and 16 + 4i as bf16 128 + c
__device__ __forceinline__ uint32_t codes(uint32_t w, int i) { return ((w >> (4 * i)) & 0x000f000fu) | 0x43004300u; }

// ------------------------------------------------------------ the schedule ---

__device__ __forceinline__ int seq_len(const Kv4Attn& a, int b)
{
    const int len = a.lens[b];
    return len > a.max_len ? -1 : len;  // too long: raised by k_kv4_rows, left alone everywhere
}

__device__ __forceinline__ int item_tiles(const Kv4Attn& a, int len)
{
    return len < 0 ? 0 : (len + 15) / 16 + (a.T + 15) / 16;
}

struct Start {
    int b;
    long long off, count;  // offset in the tiles of sequence b's items; tiles of the team
};

// Where each of the CTA's teams begins: teams t0 .. t0 + n - 1 of a.nteams
// take equal runs of all items' tiles in (sequence, item) order.
__device__ void find_starts(const Kv4Attn& a, int t0, int n, Start* starts, long long* scratch)
{
    const int items = a.Hkv * a.mtiles, per = ceil_div(a.B, (int)blockDim.x), b0 = threadIdx.x * per;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, nw = blockDim.x >> 5;
    long long mine = 0;
    for (int b = b0; b < min(b0 + per, a.B); b++) mine += (long long)items * item_tiles(a, seq_len(a, b));
    if ((int)threadIdx.x < n) starts[threadIdx.x].count = 0;
    long long x = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const long long y = __shfl_up_sync(0xffffffffu, x, o);
        if (lane >= o) x += y;
    }
    if (lane == 31) scratch[warp] = x;
    __syncthreads();
    long long before = x - mine, total = 0;
    for (int w = 0; w < nw; w++) {
        if (w < warp) before += scratch[w];
        total += scratch[w];
    }
    if (mine) {
        for (int i = 0; i < n; i++) {
            const long long u0 = total * (t0 + i) / a.nteams, u1 = total * (t0 + i + 1) / a.nteams;
            if (u0 >= u1 || u0 < before || u0 >= before + mine) continue;
            long long at = before;
            for (int b = b0; b < min(b0 + per, a.B); b++) {
                const long long c = (long long)items * item_tiles(a, seq_len(a, b));
                if (u0 < at + c) {
                    starts[i] = Start{b, u0 - at, u1 - u0};
                    break;
                }
                at += c;
            }
        }
    }
    __syncthreads();
}

// The run of tiles of one item that a team works on.
struct Run {
    int b, item, len, nt, t0, t1;
    long long left;
    __device__ __forceinline__ void begin(const Kv4Attn& a, const Start& s)
    {
        left = s.count;
        if (left <= 0) return;
        b = s.b;
        len = seq_len(a, b);
        nt = item_tiles(a, len);
        item = (int)(s.off / nt);
        t0 = (int)(s.off - (long long)item * nt);
        t1 = (int)min((long long)nt, t0 + left);
        left -= t1 - t0;
    }
    __device__ __forceinline__ bool next(const Kv4Attn& a)
    {
        if (left <= 0) return false;
        if (++item == a.Hkv * a.mtiles) {
            item = 0;
            do {
                if (++b >= a.B) return false;  // only if the lengths change under the call
                len = seq_len(a, b);
                nt = item_tiles(a, len);
            } while (nt == 0);
        }
        t0 = 0;
        t1 = (int)min((long long)nt, left);
        left -= t1;
        return true;
    }
};

// Items that several teams hold, one record per team, filled by the team that
// holds the item's first tile.
struct MergeRec {
    int b, item, rest;  // rest: the item's tiles that other teams hold (0: none begins here)
};

__host__ __device__ constexpr size_t part_floats(int R, int D) { return (size_t)R * (D + 2); }

// ------------------------------------------------------------------ kernel ---

template <int D, int NB, int TW>
struct RowsSmem {
    static constexpr int kR = 8 * NB;
    static constexpr int kStages = NB == 1 && TW > 1 ? 4 : 6;
    static constexpr int kBlk = kv4_block_bytes(D);
    static constexpr int kRing = kWarps * kStages * kBlk;
    static constexpr int kBar = kRing;
    static constexpr int kMisc = kBar + kWarps * kStages * 8;                   // starts and scan scratch
    static constexpr int kMerge = kMisc + kWarps * (int)(sizeof(Start) + 8);
    static constexpr int kMergeBytes = TW == 1 ? 0 : kWarps * kR * (D + 4) * 4;  // [warp][row][D | max, sum]
    static constexpr int kBytes = kMerge + kMergeBytes;
};

template <int D, int NB, int TW>
__global__ void __launch_bounds__(kWarps * 32, NB == 1 ? 2 : 1) k_kv4_rows(Kv4Attn a)
{
    using L = RowsSmem<D, NB, TW>;
    constexpr int S = L::kStages, R = L::kR, PAN = D / 64, MB = D / 16, DV = D / 8;
    extern __shared__ __align__(128) uint8_t sm[];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
    const int wi = TW == 1 ? 0 : warp;  // this warp's place in its team
    uint8_t* ring = sm + warp * S * L::kBlk;
    uint64_t* bar = (uint64_t*)(sm + L::kBar) + warp * S;
    Start* starts = (Start*)(sm + L::kMisc);
    long long* scratch = (long long*)(starts + kWarps);
    const int team = TW == 1 ? blockIdx.x * kWarps + warp : blockIdx.x;
    if (lane == 0) {
        for (int s = 0; s < S; s++) mbar_init(bar + s, 1);
        mbar_fence_init();
    }
    pdl_wait();
    pdl_trigger();
    if (blockIdx.x == 0)
        for (int b = threadIdx.x; b < a.B; b += blockDim.x)
            if (a.lens[b] > a.max_len) kv4_raise(a.status, LA_ERR_ARG);
    find_starts(a, TW == 1 ? blockIdx.x * kWarps : blockIdx.x, TW == 1 ? kWarps : 1, starts, scratch);
    const Start st = starts[TW == 1 ? warp : 0];
    MergeRec rec{0, 0, 0};
    MergeRec* recs = (MergeRec*)(a.part + (size_t)a.nteams * 2 * part_floats(R, D));

    const uint64_t pol = policy_evict_first();
    const int group = a.H / a.Hkv;
    // ---- the producing side: which of this warp's tiles comes next
    Run pr;
    pr.left = 0;
    pr.t0 = pr.t1 = 0;
    pr.begin(a, st);
    int pt = st.count > 0 ? pr.t0 + wi : 0;
    bool more = st.count > 0;
    int pend_page = 0, pend_head = 0, pend_blk = 0, issued = 0, taken = 0;
    bool pend = false;
    uint32_t bad_mask = 0;  // stages whose page index is outside the pool
    auto find_next = [&]() {
        pend = false;
        while (more) {
            if (pt < pr.t1 && pt * 16 < pr.len) {
                const int pg = (pt * 16) >> (4 + a.blk_log2);
                pend_page = a.table[(size_t)pr.b * a.max_pages + pg];
                pend_head = pr.item / a.mtiles;
                pend_blk = pt & ((1 << a.blk_log2) - 1);
                pend = true;
                pt += TW;
                return;
            }
            more = pr.next(a);
            if (more) pt = pr.t0 + wi;
        }
    };
    auto issue = [&]() {
        if (!pend) return;
        const int s = issued % S;
        const bool ok = (unsigned)pend_page < (unsigned)a.n_pages;
        bad_mask = (bad_mask & ~(1u << s)) | (ok ? 0u : 1u << s);
        if (lane == 0) {
            if (!ok) kv4_raise(a.status, LA_ERR_ARG);
            mbar_expect_tx(bar + s, L::kBlk);
            bulk_load(ring + s * L::kBlk,
                      a.pages + kv4_block_at(ok ? pend_page : 0, pend_head, pend_blk, a.Hkv, a.blk_log2, D), L::kBlk,
                      bar + s, pol);
        }
        issued++;
        find_next();
    };
    __syncwarp();
    find_next();
    for (int i = 0; i < S - 1; i++) issue();

    bool alive = true;  // no wait has given up
    Run run;
    run.left = 0;
    run.begin(a, st);
    if (st.count > 0) {
        bool first = true;
        do {
            const int head = run.item / a.mtiles, mt = run.item - head * a.mtiles;
            // ---- this lane's part of the query rows: row 8 nb + g, channels 64 p + 16 t ..
            uint32_t q[NB][PAN][8];
            float qs[NB][2];  // sum over the channels of rows 2t, 2t + 1
#pragma unroll
            for (int nb = 0; nb < NB; nb++) {
                const int r = mt * R + nb * 8 + g;
                float sum = 0.f;
                const __nv_bfloat16* src =
                    a.q + (size_t)(run.b * (long long)a.T + r / group) * a.q_ld + (size_t)(head * group + r % group) * D + 16 * t;
#pragma unroll
                for (int p = 0; p < PAN; p++) {
                    uint4 u0 = make_uint4(0, 0, 0, 0), u1 = u0;
                    if (r < a.rows) {
                        u0 = *(const uint4*)(src + 64 * p);
                        u1 = *(const uint4*)(src + 64 * p + 8);
                    }
                    q[nb][p][0] = u0.x, q[nb][p][1] = u0.y, q[nb][p][2] = u0.z, q[nb][p][3] = u0.w;
                    q[nb][p][4] = u1.x, q[nb][p][5] = u1.y, q[nb][p][6] = u1.z, q[nb][p][7] = u1.w;
#pragma unroll
                    for (int i = 0; i < 8; i++)
                        sum += __uint_as_float(q[nb][p][i] << 16) + __uint_as_float(q[nb][p][i] & 0xffff0000u);
                }
                sum += __shfl_xor_sync(0xffffffffu, sum, 1);
                sum += __shfl_xor_sync(0xffffffffu, sum, 2);
                qs[nb][0] = __shfl_sync(0xffffffffu, sum, 8 * t);
                qs[nb][1] = __shfl_sync(0xffffffffu, sum, 8 * t + 4);
            }
            float o[NB][MB][4], m[NB][2], l[NB][2];
#pragma unroll
            for (int nb = 0; nb < NB; nb++) {
                m[nb][0] = m[nb][1] = -INFINITY;
                l[nb][0] = l[nb][1] = 0.f;
#pragma unroll
                for (int i = 0; i < MB; i++)
#pragma unroll
                    for (int j = 0; j < 4; j++) o[nb][i][j] = 0.f;
            }
            // scores x[nb][i]: key kv4_key(g + 8 (i >> 1)) of the tile, row 2t + (i & 1);
            // turned into probabilities; the running maximum follows when it must
            auto softmax = [&](float (&x)[NB][4]) {
                bool up = false;
#pragma unroll
                for (int nb = 0; nb < NB; nb++)
                    up |= fmaxf(x[nb][0], x[nb][2]) > m[nb][0] + 8.f || fmaxf(x[nb][1], x[nb][3]) > m[nb][1] + 8.f;
                if (__any_sync(0xffffffffu, up)) {
#pragma unroll
                    for (int nb = 0; nb < NB; nb++)
#pragma unroll
                        for (int r = 0; r < 2; r++) {
                            float mx = fmaxf(x[nb][r], x[nb][r + 2]);
                            mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 4));
                            mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 8));
                            mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 16));
                            mx = fmaxf(mx, m[nb][r]);
                            const float c = mx == m[nb][r] ? 1.f : ex2(m[nb][r] - mx);
                            m[nb][r] = mx;
                            l[nb][r] *= c;
#pragma unroll
                            for (int i = 0; i < MB; i++) o[nb][i][r] *= c, o[nb][i][r + 2] *= c;
                        }
                }
#pragma unroll
                for (int nb = 0; nb < NB; nb++)
#pragma unroll
                    for (int i = 0; i < 4; i++) {
                        const float mu = m[nb][i & 1] == -INFINITY ? 0.f : m[nb][i & 1];
                        x[nb][i] = ex2(x[nb][i] - mu);
                        l[nb][i & 1] += x[nb][i];
                    }
            };
            for (int tile = run.t0 + wi; tile < run.t1; tile += TW) {
                float x[NB][4];
#pragma unroll
                for (int nb = 0; nb < NB; nb++) x[nb][0] = x[nb][1] = x[nb][2] = x[nb][3] = 0.f;
                if (tile * 16 < run.len) {
                    // ------------------------------------------ cached keys
                    issue();
                    const int s = taken % S;
                    if (alive) {
                        const unsigned long long since = globaltimer();
                        while (!mbar_try_wait(bar + s, (taken / S) & 1))
                            if (globaltimer() - since > kWaitNs) {
                                alive = false;
                                kv4_raise(a.status, LA_ERR_TIMEOUT);
                                break;
                            }
                    }
                    const uint8_t* blk = ring + s * L::kBlk;
                    const int live = (bad_mask >> s) & 1 ? 0 : run.len - tile * 16;  // keys below it count
                    taken++;
                    const int k0 = kv4_key(g), k1 = kv4_key(g + 8);
#pragma unroll
                    for (int p = 0; p < PAN; p++) {
                        const uint2 w0 = *(const uint2*)(blk + p * 512 + k0 * 32 + t * 8);
                        const uint2 w1 = *(const uint2*)(blk + p * 512 + k1 * 32 + t * 8);
#pragma unroll
                        for (int i = 0; i < 4; i++) {
                            const uint32_t u0 = i < 2 ? w0.x : w0.y, u1 = i < 2 ? w1.x : w1.y;
                            const int j = (i & 1) * 2;
                            const uint32_t a0 = codes(u0, j), a1 = codes(u1, j), a2 = codes(u0, j + 1), a3 = codes(u1, j + 1);
#pragma unroll
                            for (int nb = 0; nb < NB; nb++)
                                mma16816(x[nb], a0, a1, a2, a3, q[nb][p][2 * i], q[nb][p][2 * i + 1]);
                        }
                    }
                    const uint32_t* kp = (const uint32_t*)(blk + 16 * D);
                    const uint32_t p0 = kp[k0], p1 = kp[k1];
                    const float s0 = __uint_as_float(p0 & 0xffff0000u) * a.sl2, s1 = __uint_as_float(p1 & 0xffff0000u) * a.sl2;
                    const float z0 = __uint_as_float(p0 << 16), z1 = __uint_as_float(p1 << 16);
#pragma unroll
                    for (int nb = 0; nb < NB; nb++)
#pragma unroll
                        for (int r = 0; r < 2; r++) {
                            x[nb][r] = k0 < live ? s0 * fmaf(-z0, qs[nb][r], x[nb][r]) : -INFINITY;
                            x[nb][r + 2] = k1 < live ? s1 * fmaf(-z1, qs[nb][r], x[nb][r + 2]) : -INFINITY;
                        }
                    softmax(x);
                    const uint32_t* vp = kp + 16;
                    const float v0 = k0 < live ? __uint_as_float(vp[k0] & 0xffff0000u) : 0.f;
                    const float v1 = k1 < live ? __uint_as_float(vp[k1] & 0xffff0000u) : 0.f;
                    uint32_t b0[NB], b1[NB];
#pragma unroll
                    for (int nb = 0; nb < NB; nb++) {
                        b0[nb] = transpose8(pack_bf16(x[nb][0] * v0, x[nb][1] * v0));
                        b1[nb] = transpose8(pack_bf16(x[nb][2] * v1, x[nb][3] * v1));
                    }
                    // V of keys A, B (probability slots 2t, 2t + 1) and C, E (8 + 2t, 9 + 2t)
                    const int kA = t, kB = 4 + (t ^ 3), kC = 8 + kA, kE = 8 + kB;
                    const uint32_t zAB = __byte_perm(kA < live ? vp[kA] : 0x4300u, kB < live ? vp[kB] : 0x4300u, 0x5410);
                    const uint32_t zCE = __byte_perm(kC < live ? vp[kC] : 0x4300u, kE < live ? vp[kE] : 0x4300u, 0x5410);
                    const uint8_t* vc = blk + 8 * D;
                    if (D == 128) {
                        const uint8_t* vb = vc + (g >> 2) * 512 + (g & 3) * 8;
                        const uint2 wA = *(const uint2*)(vb + kA * 32), wB = *(const uint2*)(vb + kB * 32);
                        const uint2 wC = *(const uint2*)(vb + kC * 32), wE = *(const uint2*)(vb + kE * 32);
#pragma unroll
                        for (int hf = 0; hf < 2; hf++) {
                            const uint32_t sel = hf ? 0x7632 : 0x5410;
                            const uint32_t ab0 = __byte_perm(wA.x, wB.x, sel), ab1 = __byte_perm(wA.y, wB.y, sel);
                            const uint32_t ce0 = __byte_perm(wC.x, wE.x, sel), ce1 = __byte_perm(wC.y, wE.y, sel);
#pragma unroll
                            for (int j = 0; j < 4; j++) {
                                const uint32_t a0 = sub_bf16x2(codes(ab0, j), zAB), a1 = sub_bf16x2(codes(ab1, j), zAB);
                                const uint32_t a2 = sub_bf16x2(codes(ce0, j), zCE), a3 = sub_bf16x2(codes(ce1, j), zCE);
#pragma unroll
                                for (int nb = 0; nb < NB; nb++)
                                    mma16816(o[nb][(hf * 4 + j) % MB], a0, a1, a2, a3, b0[nb], b1[nb]);
                            }
                        }
                    } else {
                        const uint32_t wA = *(const uint32_t*)(vc + kA * 32 + g * 4), wB = *(const uint32_t*)(vc + kB * 32 + g * 4);
                        const uint32_t wC = *(const uint32_t*)(vc + kC * 32 + g * 4), wE = *(const uint32_t*)(vc + kE * 32 + g * 4);
                        const uint32_t ab0 = __byte_perm(wA, wB, 0x5410), ab1 = __byte_perm(wA, wB, 0x7632);
                        const uint32_t ce0 = __byte_perm(wC, wE, 0x5410), ce1 = __byte_perm(wC, wE, 0x7632);
#pragma unroll
                        for (int j = 0; j < 4; j++) {
                            const uint32_t a0 = sub_bf16x2(codes(ab0, j), zAB), a1 = sub_bf16x2(codes(ab1, j), zAB);
                            const uint32_t a2 = sub_bf16x2(codes(ce0, j), zCE), a3 = sub_bf16x2(codes(ce1, j), zCE);
#pragma unroll
                            for (int nb = 0; nb < NB; nb++) mma16816(o[nb][j], a0, a1, a2, a3, b0[nb], b1[nb]);
                        }
                    }
                    __syncwarp();  // every lane has read the stage: issue() may fill it again
                } else {
                    // ------------------------------------- the step's own rows
                    const int j0 = (tile - (run.len + 15) / 16) * 16;
                    const size_t col = (size_t)head * D;
                    auto row = [&](const __nv_bfloat16* base, int j) {
                        return base + (size_t)(run.b * (long long)a.T + j) * a.kv_ld + col;
                    };
                    const int k0 = j0 + kv4_key(g), k1 = j0 + kv4_key(g + 8);
#pragma unroll
                    for (int p = 0; p < PAN; p++)
#pragma unroll
                        for (int i = 0; i < 2; i++) {
                            uint4 u0 = make_uint4(0, 0, 0, 0), u1 = u0;
                            if (k0 < a.T) u0 = *(const uint4*)(row(a.ks, k0) + 64 * p + 16 * t + 8 * i);
                            if (k1 < a.T) u1 = *(const uint4*)(row(a.ks, k1) + 64 * p + 16 * t + 8 * i);
#pragma unroll
                            for (int nb = 0; nb < NB; nb++) {
                                mma16816(x[nb], u0.x, u1.x, u0.y, u1.y, q[nb][p][4 * i], q[nb][p][4 * i + 1]);
                                mma16816(x[nb], u0.z, u1.z, u0.w, u1.w, q[nb][p][4 * i + 2], q[nb][p][4 * i + 3]);
                            }
                        }
#pragma unroll
                    for (int nb = 0; nb < NB; nb++)
#pragma unroll
                        for (int r = 0; r < 2; r++) {
                            const int i = (mt * R + nb * 8 + 2 * t + r) / group;  // the step row
                            x[nb][r] = k0 < a.T && kv4_sees(i, k0, a.W, a.n1) ? x[nb][r] * a.sl2 : -INFINITY;
                            x[nb][r + 2] = k1 < a.T && kv4_sees(i, k1, a.W, a.n1) ? x[nb][r + 2] * a.sl2 : -INFINITY;
                        }
                    softmax(x);
                    uint32_t b0[NB], b1[NB];
#pragma unroll
                    for (int nb = 0; nb < NB; nb++) {
                        b0[nb] = transpose8(pack_bf16(x[nb][0], x[nb][1]));
                        b1[nb] = transpose8(pack_bf16(x[nb][2], x[nb][3]));
                    }
                    // A NaN or an infinity among the values must reach the rows that see its key
                    // and no others, and zero times it is NaN: the product runs without it
                    bool odd = false;
                    const int key[4] = {j0 + t, j0 + 4 + (t ^ 3), j0 + 8 + t, j0 + 12 + (t ^ 3)};
#pragma unroll
                    for (int half = 0; half < DV / 8; half++) {
                        // channels DV g + 8 half ..
                        uint4 v[4];
#pragma unroll
                        for (int e = 0; e < 4; e++) {
                            v[e] = make_uint4(0, 0, 0, 0);
                            if (key[e] < a.T) v[e] = *(const uint4*)(row(a.vs, key[e]) + DV * g + 8 * half);
                            odd |= drop_nonfinite(v[e].x) | drop_nonfinite(v[e].y) | drop_nonfinite(v[e].z) | drop_nonfinite(v[e].w);
                        }
                        const uint32_t* vA = (const uint32_t*)&v[0];
                        const uint32_t* vB = (const uint32_t*)&v[1];
                        const uint32_t* vC = (const uint32_t*)&v[2];
                        const uint32_t* vE = (const uint32_t*)&v[3];
                        if (D == 128) {
                            // fragment rows g and g + 8 hold channels 16 g + 2j (+ 1) and 16 g + 8 + 2j (+ 1):
                            // half the fragment at a time, the other half zero
#pragma unroll
                            for (int j = 0; j < 8; j++) {
                                const uint32_t sel = j < 4 ? 0x5410 : 0x7632;
                                const uint32_t ab = __byte_perm(vA[j & 3], vB[j & 3], sel);
                                const uint32_t ce = __byte_perm(vC[j & 3], vE[j & 3], sel);
#pragma unroll
                                for (int nb = 0; nb < NB; nb++)
                                    mma16816(o[nb][j % MB], half ? 0u : ab, half ? ab : 0u, half ? 0u : ce, half ? ce : 0u,
                                             b0[nb], b1[nb]);
                            }
                        } else {
#pragma unroll
                            for (int j = 0; j < 4; j++) {
                                const uint32_t a0 = __byte_perm(vA[j], vB[j], 0x5410), a1 = __byte_perm(vA[j], vB[j], 0x7632);
                                const uint32_t a2 = __byte_perm(vC[j], vE[j], 0x5410), a3 = __byte_perm(vC[j], vE[j], 0x7632);
#pragma unroll
                                for (int nb = 0; nb < NB; nb++) mma16816(o[nb][j], a0, a1, a2, a3, b0[nb], b1[nb]);
                            }
                        }
                    }
                    if (__any_sync(0xffffffffu, odd)) {
                        for (int j = j0; j < min(j0 + 16, a.T); j++) {
#pragma unroll
                            for (int c = 0; c < DV; c++) {
                                const float v = __bfloat162float(row(a.vs, j)[DV * g + c]);
                                if (fabsf(v) < INFINITY) continue;
                                const int mb = D == 128 ? ((c & 7) >> 1) + 4 * (c & 1) : c >> 1, hi = D == 128 ? c >> 3 : c & 1;
#pragma unroll
                                for (int nb = 0; nb < NB; nb++)
#pragma unroll
                                    for (int r = 0; r < 2; r++)
                                        if (kv4_sees((mt * R + nb * 8 + 2 * t + r) / group, j, a.W, a.n1))
                                            o[nb][mb % MB][r + 2 * hi] += v;
                            }
                        }
                    }
                }
            }
            // ---- the item's (or the run's) result
#pragma unroll
            for (int nb = 0; nb < NB; nb++)
#pragma unroll
                for (int r = 0; r < 2; r++) {
                    l[nb][r] += __shfl_xor_sync(0xffffffffu, l[nb][r], 4);
                    l[nb][r] += __shfl_xor_sync(0xffffffffu, l[nb][r], 8);
                    l[nb][r] += __shfl_xor_sync(0xffffffffu, l[nb][r], 16);
                }
            const bool whole = run.t0 == 0 && run.t1 == run.nt;
            float* part = a.part + ((size_t)team * 2 + (run.t0 == 0 ? 1 : 0)) * part_floats(R, D);
            if (run.t0 == 0 && !whole) {
                rec = MergeRec{run.b, run.item, run.nt - run.t1};
            }
            // channel c (of DV, from DV g) of row 2t + r
            auto chan = [&](int nb, int r, int c) -> float {
                if (D == 128) {
                    const int mb = ((c & 7) >> 1) + 4 * (c & 1);
                    return o[nb][mb % MB][r + (c >= 8 ? 2 : 0)];
                }
                return o[nb][c >> 1][r + 2 * (c & 1)];
            };
            if (TW == 1) {
#pragma unroll
                for (int nb = 0; nb < NB; nb++)
#pragma unroll
                    for (int r = 0; r < 2; r++) {
                        const int lr = nb * 8 + 2 * t + r, gr = mt * R + lr;
                        if (gr >= a.rows) continue;
                        if (whole) {
                            const float inv = 1.f / l[nb][r];
                            uint32_t y[DV / 2];
#pragma unroll
                            for (int c = 0; c < DV; c += 2)
                                y[c / 2] = pack_bf16(chan(nb, r, c) * inv, chan(nb, r, c + 1) * inv);
                            __nv_bfloat16* dst = a.out + ((size_t)(run.b * (long long)a.T + gr / group) * a.H + head * group + gr % group) * D + DV * g;
#pragma unroll
                            for (int c = 0; c < DV / 2; c += 4) *(uint4*)(dst + 2 * c) = make_uint4(y[c], y[c + 1], y[c + 2], y[c + 3]);
                        } else {
                            float* dst = part + (size_t)lr * D + DV * g;
#pragma unroll
                            for (int c = 0; c < DV; c += 4)
                                *(float4*)(dst + c) = make_float4(chan(nb, r, c), chan(nb, r, c + 1), chan(nb, r, c + 2), chan(nb, r, c + 3));
                            if (g == 0) *(float2*)(part + (size_t)R * D + 2 * lr) = make_float2(m[nb][r], l[nb][r]);
                        }
                    }
            } else {
                float* mg = (float*)(sm + L::kMerge);
                if (!first) __syncthreads();  // the last item's results have been read
#pragma unroll
                for (int nb = 0; nb < NB; nb++)
#pragma unroll
                    for (int r = 0; r < 2; r++) {
                        float* dst = mg + ((size_t)warp * R + nb * 8 + 2 * t + r) * (D + 4);
#pragma unroll
                        for (int c = 0; c < DV; c += 4)
                            *(float4*)(dst + DV * g + c) = make_float4(chan(nb, r, c), chan(nb, r, c + 1), chan(nb, r, c + 2), chan(nb, r, c + 3));
                        if (g == 0) *(float2*)(dst + D) = make_float2(m[nb][r], l[nb][r]);
                    }
                __syncthreads();
                for (int e = threadIdx.x; e < R * D / 4; e += kWarps * 32) {
                    const int lr = e / (D / 4), c = (e % (D / 4)) * 4, gr = mt * R + lr;
                    if (gr >= a.rows) continue;
                    float2 ml[kWarps];
                    float mx = -INFINITY;
#pragma unroll
                    for (int w = 0; w < kWarps; w++) {
                        ml[w] = *(const float2*)(mg + ((size_t)w * R + lr) * (D + 4) + D);
                        mx = fmaxf(mx, ml[w].x);
                    }
                    const float mu = mx == -INFINITY ? 0.f : mx;
                    float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
                    float sum = 0.f;
#pragma unroll
                    for (int w = 0; w < kWarps; w++) {
                        const float f = ex2(ml[w].x - mu);
                        const float4 v = *(const float4*)(mg + ((size_t)w * R + lr) * (D + 4) + c);
                        sum += f * ml[w].y;
                        acc.x += f * v.x, acc.y += f * v.y, acc.z += f * v.z, acc.w += f * v.w;
                    }
                    if (whole) {
                        const float inv = 1.f / sum;
                        *(uint2*)(a.out + ((size_t)(run.b * (long long)a.T + gr / group) * a.H + head * group + gr % group) * D + c) =
                            make_uint2(pack_bf16(acc.x * inv, acc.y * inv), pack_bf16(acc.z * inv, acc.w * inv));
                    } else {
                        *(float4*)(part + (size_t)lr * D + c) = acc;
                        if (c == 0) *(float2*)(part + (size_t)R * D + 2 * lr) = make_float2(mx, sum);
                    }
                }
                first = false;
            }
        } while (run.next(a));
    }
    if (!alive)  // no copy may still be on its way when the CTA ends
        for (; taken < issued; taken++) mbar_drain(bar + taken % S, (taken / S) & 1);
    if (a.part && (TW == 1 ? lane == 0 : threadIdx.x == 0) && team < a.nteams) recs[team] = rec;
}

// ------------------------------------------------------------------- merge ---
//
// The item that team i begins and does not end: its parts are team i's second
// slot and the first slots of the teams after it, until the item's tiles are
// all accounted for.  Weights exp2(m - M) of the parts in team order.

template <int D, int R>
__global__ void __launch_bounds__(256) k_kv4_merge(Kv4Attn a)
{
    pdl_wait();
    pdl_trigger();
    const MergeRec* recs = (const MergeRec*)(a.part + (size_t)a.nteams * 2 * part_floats(R, D));
    const MergeRec rec = recs[blockIdx.x];
    if (rec.rest == 0) return;
    __shared__ long long red[8];
    const int items = a.Hkv * a.mtiles, lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    long long mine = 0;
    for (int b = threadIdx.x; b < a.B; b += blockDim.x) mine += (long long)items * item_tiles(a, seq_len(a, b));
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) mine += __shfl_xor_sync(0xffffffffu, mine, o);
    if (lane == 0) red[warp] = mine;
    __syncthreads();
    long long total = 0;
    for (int w = 0; w < 8; w++) total += red[w];
    const int i0 = blockIdx.x;
    const long long end = total * (i0 + 1) / a.nteams + rec.rest;  // where the item ends
    int last = i0 + 1;  // teams i0 .. last hold a part
    while (total * (last + 1) / a.nteams < end) last++;
    const int head = rec.item / a.mtiles, mt = rec.item % a.mtiles, group = a.H / a.Hkv;
    for (int e = threadIdx.x; e < R * D / 4; e += blockDim.x) {
        const int lr = e / (D / 4), c = (e % (D / 4)) * 4, gr = mt * R + lr;
        if (gr >= a.rows) continue;
        float mx = -INFINITY, sum = 0.f;
        float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
        for (int i = i0; i <= last; i++) {
            if (total * i / a.nteams == total * (i + 1) / a.nteams) continue;  // a team without tiles
            const float* part = a.part + ((size_t)i * 2 + (i == i0 ? 1 : 0)) * part_floats(R, D);
            mx = fmaxf(mx, part[(size_t)R * D + 2 * lr]);
        }
        const float mu = mx == -INFINITY ? 0.f : mx;
        for (int i = i0; i <= last; i++) {
            if (total * i / a.nteams == total * (i + 1) / a.nteams) continue;
            const float* part = a.part + ((size_t)i * 2 + (i == i0 ? 1 : 0)) * part_floats(R, D);
            const float2 ml = *(const float2*)(part + (size_t)R * D + 2 * lr);
            const float4 v = *(const float4*)(part + (size_t)lr * D + c);
            const float f = ex2(ml.x - mu);
            sum += f * ml.y;
            acc.x += f * v.x, acc.y += f * v.y, acc.z += f * v.z, acc.w += f * v.w;
        }
        const float inv = 1.f / sum;
        *(uint2*)(a.out + ((size_t)(rec.b * (long long)a.T + gr / group) * a.H + head * group + gr % group) * D + c) =
            make_uint2(pack_bf16(acc.x * inv, acc.y * inv), pack_bf16(acc.z * inv, acc.w * inv));
    }
}

// ---------------------------------------------------------------- launches ---

struct Plan {
    int nb, tw, grid, nteams, mtiles;
    bool merge;
    size_t bytes;
};

int max_len_of(const la_kv4_desc& c, const la_kv4_attn& a)
{
    const int room = c.max_pages * c.page;
    return a.max_len > 0 && a.max_len < room ? a.max_len : room;
}

Plan plan_of(const la_kv4_desc& c, const la_kv4_attn& a)
{
    Plan p;
    const int T = 1 + (a.W + a.G) * (a.N - 1), rows = T * (a.n_heads / c.n_kv_heads);
    p.nb = rows <= 8 ? 1 : 2;
    p.mtiles = ceil_div(rows, 8 * p.nb);
    const long long items = (long long)a.batch * c.n_kv_heads * p.mtiles;
    const long long tiles = items * ((max_len_of(c, a) + 15) / 16 + (T + 15) / 16);
    const int ctas = p.nb == 1 ? 2 * kSMs : kSMs;  // resident at once
    p.tw = items >= (long long)ctas * kWarps ? 1 : kWarps;
    const long long teams = (long long)ctas * (p.tw == 1 ? kWarps : 1);
    p.nteams = (int)std::max(1LL, std::min(teams, std::max(items, tiles / kWarps)));
    if (p.nteams > items && p.nteams < 2 * items) p.nteams = (int)items;
    p.grid = p.tw == 1 ? ceil_div(p.nteams, kWarps) : p.nteams;
    // one sequence: every item has the same tiles, so whole items a team stay whole
    p.merge = !(a.batch == 1 && items % p.nteams == 0);
    p.bytes = p.merge ? (size_t)p.nteams * (2 * part_floats(8 * p.nb, c.head_dim) * 4 + sizeof(MergeRec)) : 0;
    return p;
}

std::mutex g_mu;
unsigned char g_ready[256];

template <int D, int NB, int TW>
bool set_smem()
{
    return cudaFuncSetAttribute(k_kv4_rows<D, NB, TW>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                RowsSmem<D, NB, TW>::kBytes) == cudaSuccess &&
           cudaFuncSetAttribute(k_kv4_rows<D, NB, TW>, cudaFuncAttributePreferredSharedMemoryCarveout, 100) == cudaSuccess;
}

// The kernels' shared-memory limits, once per device.
int attn_ready()
{
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 256) return LA_ERR_CUDA;
    std::lock_guard<std::mutex> lock(g_mu);
    if (!g_ready[dev]) {
        if (!(set_smem<128, 1, 1>() && set_smem<128, 1, 8>() && set_smem<128, 2, 1>() && set_smem<128, 2, 8>() &&
              set_smem<64, 1, 1>() && set_smem<64, 1, 8>() && set_smem<64, 2, 1>() && set_smem<64, 2, 8>()))
            return LA_ERR_CUDA;
        g_ready[dev] = 1;
    }
    return LA_OK;
}

template <int D, int NB>
cudaError_t go(cudaStream_t s, const Plan& p, const Kv4Attn& k)
{
    cudaError_t e = p.tw == 1 ? launch_pdl(k_kv4_rows<D, NB, 1>, dim3(p.grid), dim3(kWarps * 32), RowsSmem<D, NB, 1>::kBytes, s, k)
                              : launch_pdl(k_kv4_rows<D, NB, 8>, dim3(p.grid), dim3(kWarps * 32), RowsSmem<D, NB, 8>::kBytes, s, k);
    if (e == cudaSuccess && p.merge) e = launch_pdl(k_kv4_merge<D, 8 * NB>, dim3(p.nteams), dim3(256), 0, s, k);
    return e;
}

}  // namespace

size_t kv4_attn_bytes(const la_kv4_desc& c, const la_kv4_attn& a) { return a.batch ? plan_of(c, a).bytes : 0; }

int launch_kv4_attn(cudaStream_t s, const la_kv4_desc& c, const la_kv4_attn& a)
{
    if (int rc = attn_ready()) return rc;
    const Plan p = plan_of(c, a);
    Kv4Attn k;
    k.pages = (const uint8_t*)c.pages;
    k.q = (const __nv_bfloat16*)a.q, k.ks = (const __nv_bfloat16*)a.k_step, k.vs = (const __nv_bfloat16*)a.v_step;
    k.out = (__nv_bfloat16*)a.out;
    k.lens = a.lens, k.table = a.table, k.status = c.status;
    k.part = p.merge ? (float*)a.workspace : nullptr;
    k.B = a.batch, k.H = a.n_heads, k.Hkv = c.n_kv_heads;
    k.W = a.W, k.n1 = a.N - 1, k.T = 1 + (a.W + a.G) * k.n1;
    k.q_ld = a.q_ld, k.kv_ld = a.kv_ld;
    k.n_pages = c.n_pages, k.max_pages = c.max_pages, k.max_len = max_len_of(c, a);
    k.blk_log2 = c.page == 16 ? 0 : c.page == 32 ? 1 : c.page == 64 ? 2 : 3;
    k.rows = k.T * (a.n_heads / c.n_kv_heads), k.mtiles = p.mtiles, k.nteams = p.nteams;
    k.sl2 = 1.4426950408889634f / sqrtf((float)c.head_dim);
    const cudaError_t e = c.head_dim == 128 ? (p.nb == 1 ? go<128, 1>(s, p, k) : go<128, 2>(s, p, k))
                                            : (p.nb == 1 ? go<64, 1>(s, p, k) : go<64, 2>(s, p, k));
    return e == cudaSuccess ? LA_OK : LA_ERR_CUDA;
}

}  // namespace la
