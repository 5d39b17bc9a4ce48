// kv4_attn.cu -- the step's masked attention over the paged 4-bit cache for
// few rows per KV head, on mma.sync: decode steps of single tokens, small
// lookahead steps, grouped heads.
//
// For one sequence and KV head ("item") the rows are the T step rows times the
// query heads that share the KV head, in tiles of 8 rows.  With a key's
// parameters s, z and codes c:
//   S = q . (c - z) s = s (q . c - z sum q)
//   O = sum_keys p (c - z) s = sum_keys (p s) (c - z)
// so scales multiply the few scores and probabilities and not the many codes.
// A code masked out of its word is an fp16 subnormal as it stands: bits 0-3 of
// a half are c 2^-24, bits 4-7 are c 2^-20.  So unpacking is one AND a pair
// and one shift per two pairs, and both products run in fp16 with fp32 sums:
//  * q is scaled by a power of two per row (largest magnitude in [2^11, 2^12))
//    and, for the channels at bits 4-7, by 1/16: exact for every element
//    within 2^-18 of the row's largest, and off by 2^-36 of it below;
//  * p s goes to fp16: relative 2^-11, or 2^-25 absolute, where the running
//    reference keeps a row's largest so far between 1 and 2^11 (bf16 would cost
//    2^-8);
//  * -z sum(p s) is a product of its own, with -z in place of the codes of all
//    channels, added to the outputs' sums after every tile: these return near
//    zero (they shrink as the context grows, z sum(p s) does not).  Added by
//    16 more products a tile it cost 6 % (16 long 34B sequences: 113 us
//    instead of 106).
//
// Both products have the keys (K: 16 keys x 16 channels) or the channels (V:
// 16 channels x 16 keys) as the 16-row side of m16n8k16 and the query rows as
// the 8-wide side: a single token of a group of up to 8 heads fills it, and
// the probabilities go from one product's accumulators to the other's operand
// by an 8 x 8 transpose in registers.  Channels and keys are permuted so that
// each lane's fragments are contiguous bytes (kv4_key).
//
// HBM bound by its bytes: D + 8 a key and KV head.  One warp of a CTA streams
// blocks of 16 keys (one contiguous bulk copy each) into a ring for each of the
// others, so no warp waits for another inside an item.  The running reference
// M moves only when a tile's p s sum to more than 2^11 (a vote, no reduction
// per tile).
//
// Items are cut into equal runs of tiles over the teams (a warp, or a CTA
// whose warps' partial results meet in shared memory), whatever the
// sequences' lengths; an item that falls to several teams leaves partial
// outputs, which k_kv4_merge joins in a fixed order.  Fewer or shorter items
// take a cluster of 1 to 8 CTAs each (cluster_of).
//
// Measured on one GB300: 16 sequences of 1 to 64 K tokens, 8 KV heads of 8 query
// heads, D = 128: 103 us = 5.6 TB/s (83 % of a plain copy's rate); 128 sequences
// of 31 to 768 tokens, 32 heads: 53.4 us = 4.2 TB/s; one sequence of 2 K tokens, 32
// heads: 7.1 us.  At two CTAs of 128 registers a thread on an SM the schedulers
// issue in 55 % of their cycles with 3.6 warps each to choose from, half the
// arithmetic being the masks of the codes on the half-rate integer pipe (50 %
// busy): latency between dependent instructions bounds it, not a pipe.  Codes
// in bf16 (more instructions to unpack) and tiles of 16 keys were slower.
#include <algorithm>
#include <climits>
#include <cmath>
#include <mutex>

#include "kv4_sched.cuh"

namespace la {

namespace {

constexpr int kWarps = 7;  // and one that fills their rings: 8 warps leave 128 registers each at two CTAs per SM
constexpr int kKeysLog2 = 5, kKeys = 1 << kKeysLog2;  // a tile: two blocks, for independent instructions and one vote per 32 keys

// The key of a tile held in row i of a score fragment (and in slot i of the
// probabilities): with these, the four keys whose V a lane reads at once lie
// in different 32-byte rows modulo 128 bytes, and so do the K rows of a
// quarter warp.
__device__ __forceinline__ int kv4_key(int i)
{
    const int h = (i >> 1) & 3;
    return (i & 8) + ((i & 1) ? 4 + (h ^ 3) : h);
}

#define LA_MMA16816(name, type)                                                                                        \
    __device__ __forceinline__ void name(float* d, uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,    \
                                         uint32_t b1)                                                                  \
    {                                                                                                                  \
        asm volatile("mma.sync.aligned.m16n8k16.row.col.f32." type "." type                                            \
                     ".f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"                                      \
                     : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])                                                  \
                     : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));                                          \
    }
LA_MMA16816(mma_f16, "f16")
LA_MMA16816(mma_b16, "bf16")
#undef LA_MMA16816

__device__ __forceinline__ uint32_t transpose8(uint32_t x)
{
    uint32_t y;
    asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
    return y;
}

__device__ __forceinline__ void prefetch_l1(const void* p) { asm volatile("prefetch.global.L1 [%0];" ::"l"(p)); }

// bf16 pair with its NaNs and infinities replaced by 0; whether there were any
__device__ __forceinline__ bool drop_nonfinite(uint32_t& u)
{
    const bool lo = (u & 0x7f80u) == 0x7f80u, hi = (u & 0x7f800000u) == 0x7f800000u;
    if (lo) u &= 0xffff0000u;
    if (hi) u &= 0x0000ffffu;
    return lo || hi;
}

// Added to V scales, so that their logarithm exists (values under 2^-50 differ).  Not smaller: a warp's
// reference over keys without a value is that of this scale, and beside one of values near 2^50 its keys
// must keep their weight in fp32.
constexpr float kMinScale = 0x1p-64f;

// ------------------------------------------------------------------ kernel ---

// Where a row of a KV head is, relative to its sequence and head, and which
// step rows it sees (bits).
constexpr int kMaxRows = 16;
struct RowAt {
    long long q;
    int out;
    uint32_t sees;
};

// A team's results meet in areas of their own, fewer than its warps, so that the rings have three stages
// (with two, 16 sequences of 1 to 64 K tokens took 107.0 us instead of 102.7); the last warps' results
// go through the first ones'.  A cluster has two stages and an area a warp: its few tiles a warp gain
// nothing from the third, and its one result a warp loses 0.3 us of 4.0 on the way.
template <int D, int TW, bool CL>
struct RowsSmem {
    static constexpr int kR = 8;
    static constexpr int kStages = CL ? 2 : 3;
    static constexpr int kAreas = CL ? kWarps : 5;
    static constexpr int kBlk = 2 * kv4_block_bytes(D);
    static constexpr int kRing = kWarps * kStages * kBlk;
    static constexpr int kBar = kRing;                                          // full, empty
    static constexpr int kLive = kBar + kWarps * kStages * 16;                  // keys of each stage's block
    static constexpr int kMisc = kLive + (kWarps * kStages * 4 + 15) / 16 * 16;  // starts and scan scratch
    static constexpr int kTab = kMisc + (kWarps * (int)sizeof(Start) + (kWarps + 2) * 8 + 15) / 16 * 16;
    static constexpr int kMerge = kTab + kMaxRows * (int)sizeof(RowAt);
    static constexpr int kMergeBytes = TW == 1 ? 0 : kAreas * kR * (D + 4) * 4;  // [area][row][D | M, sum]
    static constexpr int kBytes = kMerge + kMergeBytes;
    static_assert(kMisc % 8 == 0 && kMerge % 16 == 0, "alignment");
};

constexpr int kThreads = (kWarps + 1) * 32;

// Warp kWarps: lane w fills the ring of warp w, block by block in the order in
// which that warp takes them.  The lanes poll their rings' empty barriers in
// turn; the page of the next block is looked up a round ahead.
template <int D, bool CL, int S>
__device__ __forceinline__ void produce(const Kv4Attn& a, Run r, bool more, uint8_t* ring, uint64_t* full, uint64_t* empty,
                                        int* live, int wi, int stride)
{
    const uint64_t pol = policy_evict_first();
    constexpr int BLK = kv4_block_bytes(D);
    int t = r.t0 + wi, page = 0, page1 = 0, head = 0, left = 0, blk = 0, n = 0;
    bool pend = false;
    auto find = [&]() {
        pend = false;
        while (more) {
            if (t < r.t1 && t * kKeys < r.len) {
                // block 2t of the sequence and, when it has one, 2t + 1: in the same
                // page unless pages hold a single block
                const int* entry = a.table + (size_t)r.b * a.max_pages + ((2 * t) >> a.blk_log2);
                page = __ldg(entry);
                left = r.len - t * kKeys;
                page1 = left > 16 ? (a.blk_log2 ? page : __ldg(entry + 1)) : -2;
                head = r.item >> (a.mtiles >> 1);
                blk = (2 * t) & ((1 << a.blk_log2) - 1);
                pend = true;
                t += stride;
                return;
            }
            more = !CL && r.next(a);
            t = r.t0 + wi;
        }
    };
    find();
    unsigned long long since = 0;
    int s = 0, phase = 1;  // the first pass over the ring does not wait
    while (__any_sync(0xffffffffu, pend)) {
        bool moved = false;
        if (pend && (n < S || mbar_try_wait(empty + s, phase))) {
            // two numbers of keys: the first block's and the second's
            const bool ok0 = (unsigned)page < (unsigned)a.n_pages, ok1 = (unsigned)page1 < (unsigned)a.n_pages;
            if (!ok0 || (!ok1 && page1 != -2)) kv4_raise(a.status, LA_ERR_ARG);
            live[s] = (ok0 ? min(left, 16) : 0) | (ok1 ? left - 16 < 16 ? left - 16 : 16 : 0) << 8;
            uint8_t* dst = ring + s * 2 * BLK;
            const uint8_t* src = a.pages + kv4_block_at(ok0 ? page : 0, head, blk, a.Hkv, a.blk_log2, D);
            if (page1 == -2) {
                mbar_expect_tx(full + s, BLK);
                bulk_load(dst, src, BLK, full + s, pol);
            } else if (a.blk_log2) {
                mbar_expect_tx(full + s, 2 * BLK);
                bulk_load(dst, src, 2 * BLK, full + s, pol);
            } else {
                mbar_expect_tx(full + s, 2 * BLK);
                bulk_load(dst, src, BLK, full + s, pol);
                bulk_load(dst + BLK, a.pages + kv4_block_at(ok1 ? page1 : 0, head, 0, a.Hkv, 0, D), BLK, full + s, pol);
            }
            n++;
            if (++s == S) s = 0, phase ^= 1;
            find();
            moved = true;
        }
        if (__any_sync(0xffffffffu, moved)) {
            since = 0;
        } else {
            __nanosleep(40);
            const unsigned long long now = globaltimer();
            if (!since) since = now;
            if (now - since > 2 * kWaitNs) {  // the consumers gave up: they have reported it
                pend = false;
            }
        }
    }
    // no copy may still be on its way when the CTA ends: the last S of this
    // lane's, whichever of them were issued
    for (int i = 0; i < S && i < n; i++) {
        const int k = n - 1 - i;
        mbar_drain(full + k % S, (k / S) & 1);
    }
}

// CL: one item per cluster of CTAs, whose warps take its tiles in turn and whose results meet in
// distributed shared memory: one launch, no workspace.
template <int D, int TW, bool CL>
__global__ void __launch_bounds__(kThreads, 2) k_kv4_rows(Kv4Attn a)
{
    using L = RowsSmem<D, TW, CL>;
    constexpr int S = L::kStages, R = L::kR, PAN = D / 64, MB = D / 16, DV = D / 8, BLK = kv4_block_bytes(D);
    extern __shared__ __align__(128) uint8_t sm[];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
    uint64_t *full = (uint64_t*)(sm + L::kBar), *empty = full + kWarps * S;
    int* live_of = (int*)(sm + L::kLive);
    Start* starts = (Start*)(sm + L::kMisc);
    RowAt* tab = (RowAt*)(sm + L::kTab);
    const int group = a.H / a.Hkv;
    if (threadIdx.x < kWarps * S) {
        mbar_init(full + threadIdx.x, 1);
        mbar_init(empty + threadIdx.x, 1);
        mbar_fence_init();
    } else if (threadIdx.x >= 64 && threadIdx.x < 64 + kMaxRows) {
        const int r = threadIdx.x - 64, i = r / group;
        uint32_t see = 0;
        for (int j = 0; j < a.T; j++) see |= kv4_sees(i, j, a.W, a.n1) ? 1u << j : 0u;
        tab[r] = RowAt{(long long)i * a.q_ld + (r - i * group) * D, (i * a.H + r - i * group) * D, see};
    }
    pdl_wait();
    pdl_trigger();
    if (blockIdx.x == 0) raise_long(a);
    const int cs = CL ? (int)cluster_size() : 1, rank = CL ? (int)cluster_rank() : 0;
    // the lane's warp in the producer, this warp otherwise; its place in its team, and how many there are
    const int w = warp == kWarps ? min(lane, kWarps - 1) : warp;
    const int wi = TW == 1 ? 0 : rank * TW + w, stride = TW * cs;
    Run run;
    run.left = 0, run.t0 = run.t1 = 0;
    bool work;
    if (CL) {
        const int x = blockIdx.x / cs, items = a.Hkv * a.mtiles;
        run.b = x / items;
        run.item = x - run.b * items;
        run.len = seq_len(a, run.b);
        work = run.len >= 0;
        run.nu = run.u1 = run.t1 = (run.len + kKeys - 1) / kKeys + 1, run.u0 = 0;
        __syncthreads();  // the mbarriers and the table
    } else {
        // (its barriers also publish the mbarriers and the table)
        find_starts(a, TW == 1 ? blockIdx.x * kWarps : blockIdx.x, TW == 1 ? kWarps : 1, starts, (long long*)(starts + kWarps));
        const Start st = starts[TW == 1 ? w : 0];
        work = st.count > 0;
        if (work) run.begin(a, st);
    }
    if (warp == kWarps) {
        produce<D, CL, S>(a, run, work && lane < kWarps, sm + w * S * L::kBlk, full + w * S, empty + w * S, live_of + w * S, wi, stride);
        return;
    }
    const int team = TW == 1 ? blockIdx.x * kWarps + warp : blockIdx.x;
    full += warp * S, empty += warp * S, live_of += warp * S;
    MergeRec* rec = (MergeRec*)(a.part + (size_t)a.nteams * 2 * part_floats(R, D)) + team;
    const bool writes_rec = !CL && a.part && team < a.nteams && lane == 0 && wi == 0;
    if (writes_rec) rec->rest = 0;
    bool alive = true;  // no wait has given up
    int s = 0, phase = 0;
    if (work) {
        bool first = true;
        do {
            const int mt = run.item & (a.mtiles - 1), head = run.item >> (a.mtiles >> 1);  // 1 or 2 row tiles
            const int ntc = (run.len + kKeys - 1) / kKeys;
            const __nv_bfloat16* q_base = a.q + (size_t)run.b * a.T * a.q_ld + (size_t)head * group * D;
            // needed last: the step's rows of this KV head; then the next head's queries
            const size_t step_at = (size_t)run.b * a.T * a.kv_ld + (size_t)head * D;
            if (run.t1 > ntc && lane < a.T) {
                const size_t at = step_at + (size_t)lane * a.kv_ld;
                prefetch_l1(a.ks + at), prefetch_l1(a.vs + at);
                if (D == 128) prefetch_l1(a.ks + at + 64), prefetch_l1(a.vs + at + 64);
            }
            const bool q_here = mt * R + g < a.rows;
            const __nv_bfloat16* q_row = q_base + tab[mt * R + g].q + 16 * t;
            if (q_here && t < PAN && head + 1 < a.Hkv) prefetch_l1(q_row + group * D + 48 * t);
            float o[MB][4], m[2] = {kNoRef, kNoRef}, l[2] = {0.f, 0.f};  // rows 2t, 2t + 1
#pragma unroll
            for (int i = 0; i < MB; i++)
#pragma unroll
                for (int j = 0; j < 4; j++) o[i][j] = 0.f;
            // Move the references to the largest y = log2(p s) of the tile (y: of this lane's).
            auto raise_ref = [&](float y0, float y1) {
#pragma unroll
                for (int r = 0; r < 2; r++) {
                    float mx = r ? y1 : y0;
                    mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 4));
                    mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 8));
                    mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 16));
                    mx = fmaxf(mx, m[r]);
                    const float c = ex2(m[r] - mx);
                    m[r] = mx;
                    l[r] *= c;
#pragma unroll
                    for (int i = 0; i < MB; i++) o[i][r] *= c, o[i][r + 2] *= c;
                }
            };
            if (run.t0 + wi < min(run.t1, ntc)) {
                // ---------------------------------------------- cached keys
                // this lane's part of the query rows: row g, channels 64 p + 16 t ..
                uint32_t q[PAN][8];
                float qs[2], qf[2];  // rows 2t, 2t + 1: sum of q, what undoes q's and the codes' powers of two
                {
                    float sum = 0.f, top = 0.f;
#pragma unroll
                    for (int p = 0; p < PAN; p++) {
                        uint4 u0 = make_uint4(0, 0, 0, 0), u1 = u0;
                        if (q_here) {
                            u0 = *(const uint4*)(q_row + 64 * p);
                            u1 = *(const uint4*)(q_row + 64 * p + 8);
                        }
                        q[p][0] = u0.x, q[p][1] = u0.y, q[p][2] = u0.z, q[p][3] = u0.w;
                        q[p][4] = u1.x, q[p][5] = u1.y, q[p][6] = u1.z, q[p][7] = u1.w;
                    }
#pragma unroll
                    for (int p = 0; p < PAN; p++)
#pragma unroll
                        for (int i = 0; i < 8; i++) {
                            const float lo = __uint_as_float(q[p][i] << 16), hi = __uint_as_float(q[p][i] & 0xffff0000u);
                            sum += lo + hi;
                            top = fmaxf(top, fmaxf(fabsf(lo), fabsf(hi)));
                        }
                    sum += __shfl_xor_sync(0xffffffffu, sum, 1);
                    sum += __shfl_xor_sync(0xffffffffu, sum, 2);
                    top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 1));
                    top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 2));
                    // exponent of the row's largest, kept where both powers of two are normal numbers
                    const int e = min(max((int)(__float_as_uint(top) >> 23), 16), 236);
                    const float down = __uint_as_float((uint32_t)(127 + 11 + 127 - e) << 23);    // 2^(11 - (e - 127))
                    const float up = __uint_as_float((uint32_t)(e - 11 + 24 - 8) << 23) * 256.f;  // 2^(24 - 11 + e - 127)
#pragma unroll
                    for (int p = 0; p < PAN; p++)
#pragma unroll
                        for (int i = 0; i < 8; i++) {
                            const float f = i & 1 ? down * 0.0625f : down;
                            q[p][i] = pack_f16(__uint_as_float(q[p][i] << 16) * f, __uint_as_float(q[p][i] & 0xffff0000u) * f);
                        }
                    qs[0] = __shfl_sync(0xffffffffu, sum * a.sl2, 8 * t);
                    qs[1] = __shfl_sync(0xffffffffu, sum * a.sl2, 8 * t + 4);
                    qf[0] = __shfl_sync(0xffffffffu, up * a.sl2, 8 * t);
                    qf[1] = __shfl_sync(0xffffffffu, up * a.sl2, 8 * t + 4);
                }
                const int k0 = kv4_key(g), k1 = k0 + 8;
                const int kA = t, kB = 4 + (t ^ 3);  // V's keys: probability slots 2t, 2t + 1; + 8: slots 2t + 8, 2t + 9
                for (int tile = run.t0 + wi; tile < min(run.t1, ntc); tile += stride) {
                    if (alive && !mbar_try_wait(full + s, phase)) {
                        const unsigned long long since = globaltimer();
                        while (!mbar_try_wait(full + s, phase))
                            if (globaltimer() - since > kWaitNs) {
                                alive = false;
                                kv4_raise(a.status, LA_ERR_TIMEOUT);
                                break;
                            }
                    }
                    const uint8_t* stage = sm + (warp * S + s) * L::kBlk;
                    const int live = live_of[s];
                    float x[2][4], sv[2][2];  // per block: scores; V scales of the keys k0, k1
#pragma unroll
                    for (int u = 0; u < 2; u++) {
                        const uint8_t* blk = stage + u * BLK;
                        float y[4] = {0.f, 0.f, 0.f, 0.f};  // a second sum, to halve the chain of dependent products
                        x[u][0] = x[u][1] = x[u][2] = x[u][3] = 0.f;
#pragma unroll
                        for (int p = 0; p < PAN; p++) {
                            const uint2 w0 = *(const uint2*)(blk + p * 512 + k0 * 32 + t * 8);
                            const uint2 w1 = *(const uint2*)(blk + p * 512 + k1 * 32 + t * 8);
#pragma unroll
                            for (int i = 0; i < 4; i++) {
                                uint32_t u0 = i < 2 ? w0.x : w0.y, u1 = i < 2 ? w1.x : w1.y;
                                if (i & 1) u0 >>= 8, u1 >>= 8;
                                mma_f16(i & 1 ? y : x[u], u0 & kLo, u1 & kLo, u0 & kHi, u1 & kHi, q[p][2 * i], q[p][2 * i + 1]);
                            }
                        }
                        const uint32_t* par = (const uint32_t*)(blk + 16 * D);  // K, then V
                        const uint32_t p0 = par[k0], p1 = par[k1];
                        const float s0 = __uint_as_float(p0 & 0xffff0000u), s1 = __uint_as_float(p1 & 0xffff0000u);
                        const float z0 = 128.f - __uint_as_float(p0 << 16), z1 = 128.f - __uint_as_float(p1 << 16);  // -z
                        sv[u][0] = __uint_as_float(par[16 + k0] & 0xffff0000u) + kMinScale;
                        sv[u][1] = __uint_as_float(par[16 + k1] & 0xffff0000u) + kMinScale;
#pragma unroll
                        for (int r = 0; r < 2; r++) {
                            x[u][r] = s0 * fmaf(x[u][r] + y[r], qf[r], z0 * qs[r]);
                            x[u][r + 2] = s1 * fmaf(x[u][r + 2] + y[r + 2], qf[r], z1 * qs[r]);
                        }
                    }
                    if (live != 0x1010) {
                        // the last blocks of a sequence (or a bad page): the rest may hold anything
#pragma unroll
                        for (int u = 0; u < 2; u++) {
                            const int n = (live >> (8 * u)) & 255;
                            if (k0 >= n) x[u][0] = x[u][1] = -INFINITY, sv[u][0] = kMinScale;
                            if (k1 >= n) x[u][2] = x[u][3] = -INFINITY, sv[u][1] = kMinScale;
                        }
                    }
                    float e[2][4];              // probabilities
                    uint32_t b0[2], b1[2];      // p s of the keys k0 and k1, rows 2t and 2t + 1
                    auto weigh = [&]() {  // the sum of this lane's p s: while it is at most 2^11, none is above that
                        float all[2];
#pragma unroll
                        for (int u = 0; u < 2; u++) {
                            float w[4];
#pragma unroll
                            for (int i = 0; i < 4; i++) {
                                e[u][i] = ex2(x[u][i] - m[i & 1]);
                                w[i] = e[u][i] * sv[u][i >> 1];
                            }
                            all[u] = (w[0] + w[1]) + (w[2] + w[3]);
                            b0[u] = pack_f16(w[0], w[1]);
                            b1[u] = pack_f16(w[2], w[3]);
                        }
                        return all[0] + all[1];
                    };
                    if (__any_sync(0xffffffffu, weigh() > 2048.f)) {
                        float y[2];
#pragma unroll
                        for (int r = 0; r < 2; r++)
                            y[r] = fmaxf(fmaxf(x[0][r] + __log2f(sv[0][0]), x[0][r + 2] + __log2f(sv[0][1])),
                                         fmaxf(x[1][r] + __log2f(sv[1][0]), x[1][r + 2] + __log2f(sv[1][1])));
                        raise_ref(y[0], y[1]);
                        weigh();
                    }
                    float zs[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
                    for (int u = 0; u < 2; u++) {
                        const uint8_t* blk = stage + u * BLK;
                        const uint32_t* vpar = (const uint32_t*)(blk + 16 * D + 64);
                        const uint32_t vA = vpar[kA], vB = vpar[kB], vC = vpar[8 + kA], vE = vpar[8 + kB];
                        l[0] += e[u][0] + e[u][2];
                        l[1] += e[u][1] + e[u][3];
                        b0[u] = transpose8(b0[u]);
                        b1[u] = transpose8(b1[u]);
                        // -z of the same keys as fp16 2^-24 z
                        const uint32_t zAB = __byte_perm(vA, vB, 0x5410) & kLo, zCE = __byte_perm(vC, vE, 0x5410) & kLo;
                        const uint32_t zl0 = zAB | 0x80008000u, zl1 = zCE | 0x80008000u;
                        const uint8_t* vc = blk + 8 * D;
                        if (D == 128) {
                            const uint8_t* vb = vc + (g >> 2) * 512 + (g & 3) * 8;
                            const uint2 wA = *(const uint2*)(vb + kA * 32), wB = *(const uint2*)(vb + kB * 32);
                            const uint2 wC = *(const uint2*)(vb + kA * 32 + 256), wE = *(const uint2*)(vb + kB * 32 + 256);
#pragma unroll
                            for (int hf = 0; hf < 2; hf++) {
                                const uint32_t sel = hf ? 0x7632 : 0x5410;
                                uint32_t ab0 = __byte_perm(wA.x, wB.x, sel), ab1 = __byte_perm(wA.y, wB.y, sel);
                                uint32_t ce0 = __byte_perm(wC.x, wE.x, sel), ce1 = __byte_perm(wC.y, wE.y, sel);
#pragma unroll
                                for (int j = 0; j < 4; j++) {
                                    const uint32_t mk = j & 1 ? kHi : kLo;
                                    if (j == 2) ab0 >>= 8, ab1 >>= 8, ce0 >>= 8, ce1 >>= 8;
                                    mma_f16(o[(hf * 4 + j) % MB], ab0 & mk, ab1 & mk, ce0 & mk, ce1 & mk, b0[u], b1[u]);
                                }
                            }
                        } else {
                            const uint8_t* vb = vc + g * 4;
                            const uint32_t wA = *(const uint32_t*)(vb + kA * 32), wB = *(const uint32_t*)(vb + kB * 32);
                            const uint32_t wC = *(const uint32_t*)(vb + kA * 32 + 256), wE = *(const uint32_t*)(vb + kB * 32 + 256);
                            uint32_t ab0 = __byte_perm(wA, wB, 0x5410), ab1 = __byte_perm(wA, wB, 0x7632);
                            uint32_t ce0 = __byte_perm(wC, wE, 0x5410), ce1 = __byte_perm(wC, wE, 0x7632);
#pragma unroll
                            for (int j = 0; j < 4; j++) {
                                const uint32_t mk = j & 1 ? kHi : kLo;
                                if (j == 2) ab0 >>= 8, ab1 >>= 8, ce0 >>= 8, ce1 >>= 8;
                                mma_f16(o[j], ab0 & mk, ab1 & mk, ce0 & mk, ce1 & mk, b0[u], b1[u]);
                            }
                        }
                        mma_f16(zs, zl0, zl0, zl1, zl1, b0[u], b1[u]);
                    }
                    {
                        // the odd accumulators' codes are 16 times as large
                        const uint64_t lo = pair(zs[0], zs[1]), hi = pair(zs[0] * 16.f, zs[1] * 16.f);
#pragma unroll
                        for (int j = 0; j < MB; j++) {
                            unpair(add2(pair(o[j][0], o[j][1]), j & 1 ? hi : lo), o[j][0], o[j][1]);
                            unpair(add2(pair(o[j][2], o[j][3]), j & 1 ? hi : lo), o[j][2], o[j][3]);
                        }
                    }
                    __syncwarp();  // every lane has read the stage
                    if (lane == 0) mbar_arrive(empty + s);
                    if (++s == S) s = 0, phase ^= 1;
                }
            }
            // ------------------------------------------ the step's own rows (16 at most: one tile)
            // in bf16, with the probabilities brought to the codes' powers of two.  V is bf16 of any
            // exponent, so both operands of P V are, and P rounds by 2^-8 of itself (as in la_attention);
            // fp16 would need V scaled by the tile's largest first, for the few keys of a step.
            if (run.t1 > ntc && (TW == 1 || (ntc - run.t0) % stride == wi)) {
                const __nv_bfloat16 *ks = a.ks + step_at, *vs = a.vs + step_at;
                const int k0 = kv4_key(g), k1 = k0 + 8;
                float x[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
                for (int p = 0; p < PAN; p++)
#pragma unroll
                    for (int i = 0; i < 2; i++) {
                        const int c = 64 * p + 16 * t + 8 * i;
                        uint4 u0 = make_uint4(0, 0, 0, 0), u1 = u0, u = u0;
                        if (k0 < a.T) u0 = *(const uint4*)(ks + (size_t)k0 * a.kv_ld + c);
                        if (k1 < a.T) u1 = *(const uint4*)(ks + (size_t)k1 * a.kv_ld + c);
                        if (q_here) u = *(const uint4*)(q_row + 64 * p + 8 * i);
                        mma_b16(x, u0.x, u1.x, u0.y, u1.y, u.x, u.y);
                        mma_b16(x, u0.z, u1.z, u0.w, u1.w, u.z, u.w);
                    }
#pragma unroll
                for (int r = 0; r < 2; r++) {
                    const uint32_t see = tab[mt * R + 2 * t + r].sees;  // (rows beyond T see none)
                    x[r] = (see >> k0) & 1 ? x[r] * a.sl2 : -INFINITY;
                    x[r + 2] = (see >> k1) & 1 ? x[r + 2] * a.sl2 : -INFINITY;
                }
                raise_ref(fmaxf(x[0], x[2]), fmaxf(x[1], x[3]));
                uint32_t b0[2], b1[2];
                float e[4];
#pragma unroll
                for (int i = 0; i < 4; i++) e[i] = ex2(x[i] - m[i & 1]);
                l[0] += e[0] + e[2];
                l[1] += e[1] + e[3];
#pragma unroll
                for (int h = 0; h < 2; h++) {
                    const float f = h ? 0x1p-20f : 0x1p-24f;
                    b0[h] = transpose8(pack_bf16(e[0] * f, e[1] * f));
                    b1[h] = transpose8(pack_bf16(e[2] * f, e[3] * f));
                }
                bool odd = false;
                const int key[4] = {t, 4 + (t ^ 3), 8 + t, 12 + (t ^ 3)};
#pragma unroll
                for (int half = 0; half < DV / 8; half++) {
                    // channels DV g + 8 half ..
                    uint32_t v[4][4];
                    __nv_bfloat162 zero = __float2bfloat162_rn(0.f), nan = zero;
#pragma unroll
                    for (int i = 0; i < 4; i++) {
                        uint4 u = make_uint4(0, 0, 0, 0);
                        if (key[i] < a.T) u = *(const uint4*)(vs + (size_t)key[i] * a.kv_ld + DV * g + 8 * half);
                        v[i][0] = u.x, v[i][1] = u.y, v[i][2] = u.z, v[i][3] = u.w;
#pragma unroll
                        for (int k = 0; k < 4; k++) nan = __hfma2(*reinterpret_cast<__nv_bfloat162*>(&v[i][k]), zero, nan);
                    }
                    if (!__hbeq2(nan, zero)) {
                        // A NaN or an infinity among the values must reach the rows that see its key
                        // and no others, and zero times it is NaN: the product runs without it
                        odd = true;
#pragma unroll
                        for (int i = 0; i < 4; i++)
#pragma unroll
                            for (int k = 0; k < 4; k++) drop_nonfinite(v[i][k]);
                    }
                    if (D == 128) {
                        // fragment rows g and g + 8 hold channels 16 g + 2j (+ 1) and 16 g + 8 + 2j (+ 1):
                        // half the fragment at a time, the other half zero
#pragma unroll
                        for (int j = 0; j < 8; j++) {
                            const uint32_t sel = j < 4 ? 0x5410 : 0x7632;
                            const uint32_t ab = __byte_perm(v[0][j & 3], v[1][j & 3], sel);
                            const uint32_t ce = __byte_perm(v[2][j & 3], v[3][j & 3], sel);
                            mma_b16(o[j % MB], half ? 0u : ab, half ? ab : 0u, half ? 0u : ce, half ? ce : 0u, b0[j & 1], b1[j & 1]);
                        }
                    } else {
#pragma unroll
                        for (int j = 0; j < 4; j++) {
                            const uint32_t a0 = __byte_perm(v[0][j], v[1][j], 0x5410), a1 = __byte_perm(v[0][j], v[1][j], 0x7632);
                            const uint32_t a2 = __byte_perm(v[2][j], v[3][j], 0x5410), a3 = __byte_perm(v[2][j], v[3][j], 0x7632);
                            mma_b16(o[j], a0, a1, a2, a3, b0[j & 1], b1[j & 1]);
                        }
                    }
                }
                if (__any_sync(0xffffffffu, odd)) {
                    for (int j = 0; j < a.T; j++) {
#pragma unroll
                        for (int c = 0; c < DV; c++) {
                            const float v = __bfloat162float(vs[(size_t)j * a.kv_ld + DV * g + c]);
                            const int mb = D == 128 ? ((c & 7) >> 1) + 4 * (c & 1) : c >> 1, hi = D == 128 ? c >> 3 : c & 1;
                            if (!(fabsf(v) < INFINITY))
#pragma unroll
                                for (int r = 0; r < 2; r++)
                                    if ((tab[mt * R + 2 * t + r].sees >> j) & 1) o[mb % MB][r + 2 * hi] += v;
                        }
                    }
                }
            }
            // ---- the item's (or the run's) result
#pragma unroll
            for (int r = 0; r < 2; r++) {
                l[r] += __shfl_xor_sync(0xffffffffu, l[r], 4);
                l[r] += __shfl_xor_sync(0xffffffffu, l[r], 8);
                l[r] += __shfl_xor_sync(0xffffffffu, l[r], 16);
            }
            const bool whole = run.u0 == 0 && run.u1 == run.nu;
            float* part = a.part + ((size_t)team * 2 + (run.u0 == 0 ? 1 : 0)) * part_floats(R, D);
            if (run.u0 == 0 && !whole && writes_rec) *rec = MergeRec{run.b, run.item, run.nu - run.u1, 0, starts[TW == 1 ? warp : 0].sh};
            __nv_bfloat16* out_base = a.out + ((size_t)run.b * a.T * a.H + (size_t)head * group) * D;
            // channel c (of DV, from DV g) of row 2t + r, times f
            auto chan = [&](int r, int c, float f) -> float {
                const int mb = D == 128 ? ((c & 7) >> 1) + 4 * (c & 1) : c >> 1, hi = D == 128 ? c >> 3 : c & 1;
                return o[mb % MB][r + 2 * hi] * (mb & 1 ? f * 0x1p20f : f * 0x1p24f);
            };
            if (TW == 1 && whole) {
#pragma unroll
                for (int r = 0; r < 2; r++) {
                    const int lr = mt * R + 2 * t + r;
                    const float inv = 1.f / l[r];
                    uint32_t y[DV / 2];
#pragma unroll
                    for (int c = 0; c < DV; c += 2) y[c / 2] = pack_bf16(chan(r, c, 1.f) * inv, chan(r, c + 1, 1.f) * inv);
                    if (lr < a.rows) {
                        __nv_bfloat16* dst = out_base + tab[lr].out + DV * g;
#pragma unroll
                        for (int c = 0; c < DV / 2; c += 4) *(uint4*)(dst + 2 * c) = make_uint4(y[c], y[c + 1], y[c + 2], y[c + 3]);
                    }
                }
            } else {
                // [row][D], then the rows' references and sums: to a merge area of the team, or as a part
                constexpr int kLd = TW == 1 ? D : D + 4, kAreas = L::kAreas;
                constexpr bool kTwice = TW > 1 && kAreas < kWarps;
                const int area = warp < kAreas ? warp : warp - kAreas;
                float* to = TW == 1 ? part : (float*)(sm + L::kMerge) + (size_t)area * R * (D + 4);
                if (TW > 1 && !first) named_sync(1, kWarps * 32);  // the last item's results have been read
#pragma unroll 1
                for (int late = 0; late < (kTwice ? 2 : 1); late++) {  // the last warps' results first
                    if (kTwice && late == 1) {
                        named_sync(1, kWarps * 32);
                        if (warp < kWarps - kAreas) {
                            // the same lane of the late warp wrote the same elements
#pragma unroll
                            for (int r = 0; r < 2; r++) {
                                const float* row = to + (size_t)(2 * t + r) * kLd;
                                const float2 ml = *(const float2*)(row + D);
                                const float mx = fmaxf(m[r], ml.x), f = ex2(m[r] - mx), h = ex2(ml.x - mx);
                                l[r] = l[r] * f + ml.y * h;
                                m[r] = mx;
#pragma unroll
                                for (int c = 0; c < DV; c++) {
                                    const int mb = D == 128 ? ((c & 7) >> 1) + 4 * (c & 1) : c >> 1, hi = D == 128 ? c >> 3 : c & 1;
                                    float& x = o[mb % MB][r + 2 * hi];
                                    x = x * f + row[DV * g + c] * (mb & 1 ? h * 0x1p-20f : h * 0x1p-24f);
                                }
                            }
                            __syncwarp();  // every lane has read the references
                        }
                    }
                    if (kTwice && (warp < kAreas) != (late == 1)) continue;
#pragma unroll
                    for (int r = 0; r < 2; r++) {
                        const int lr = 2 * t + r;
                        if (TW > 1 || mt * R + lr < a.rows) {
#pragma unroll
                            for (int c = 0; c < DV; c += 4)
                                *(float4*)(to + (size_t)lr * kLd + DV * g + c) =
                                    make_float4(chan(r, c, 1.f), chan(r, c + 1, 1.f), chan(r, c + 2, 1.f), chan(r, c + 3, 1.f));
                            if (g == 0) *(float2*)(TW == 1 ? to + (size_t)R * D + 2 * lr : to + (size_t)lr * kLd + D) = make_float2(m[r], l[r]);
                        }
                    }
                }
            }
            if (TW > 1) {
                float* mg = (float*)(sm + L::kMerge);
                named_sync(1, kWarps * 32);
                for (int i = threadIdx.x; i < R * D / 4; i += kWarps * 32) {
                    const int lr = i / (D / 4), c = (i % (D / 4)) * 4;
                    if (mt * R + lr >= a.rows) continue;
                    float2 ml[L::kAreas];
                    float mx = kNoRef;
#pragma unroll
                    for (int w = 0; w < L::kAreas; w++) {
                        ml[w] = *(const float2*)(mg + ((size_t)w * R + lr) * (D + 4) + D);
                        mx = fmaxf(mx, ml[w].x);
                    }
                    float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
                    float sum = 0.f;
#pragma unroll
                    for (int w = 0; w < L::kAreas; w++) {
                        const float f = ex2(ml[w].x - mx);
                        const float4 v = *(const float4*)(mg + ((size_t)w * R + lr) * (D + 4) + c);
                        sum += f * ml[w].y;
                        acc.x += f * v.x, acc.y += f * v.y, acc.z += f * v.z, acc.w += f * v.w;
                    }
                    if (CL && cs > 1) {
                        // over the first warp's (no other thread reads these four); the rest of the row's padding
                        *(float4*)(mg + (size_t)lr * (D + 4) + c) = acc;
                        if (c == 0) *(float2*)(mg + (size_t)lr * (D + 4) + D + 2) = make_float2(mx, sum);
                    } else if (whole) {
                        const float inv = 1.f / sum;
                        *(uint2*)(out_base + tab[mt * R + lr].out + c) =
                            make_uint2(pack_bf16(acc.x * inv, acc.y * inv), pack_bf16(acc.z * inv, acc.w * inv));
                    } else {
                        *(float4*)(part + (size_t)lr * D + c) = acc;
                        if (c == 0) *(float2*)(part + (size_t)R * D + 2 * lr) = make_float2(mx, sum);
                    }
                }
                first = false;
            }
            if (CL && cs > 1) {
                // every CTA joins its share of the item's outputs
                __syncwarp();
                cluster_sync();
                const int share = R * D / 4 / cs;
                for (int i = threadIdx.x; i < share; i += kWarps * 32) {
                    const int at = rank * share + i, lr = at / (D / 4), c = (at % (D / 4)) * 4;
                    if (mt * R + lr >= a.rows) continue;
                    const float* row = (const float*)(sm + L::kMerge) + (size_t)lr * (D + 4);
                    float2 ml[8];
                    float4 v[8];
                    float mx = kNoRef, sum = 0.f;
#pragma unroll
                    for (int r = 0; r < 8; r++) {
                        ml[r] = make_float2(kNoRef, 0.f), v[r] = make_float4(0.f, 0.f, 0.f, 0.f);
                        if (r < cs) ml[r] = ld_peer2(peer(row + D + 2, r)), v[r] = ld_peer4(peer(row + c, r));
                    }
#pragma unroll
                    for (int r = 0; r < 8; r++) mx = fmaxf(mx, ml[r].x);
                    float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
                    for (int r = 0; r < 8; r++) {
                        const float f = ex2(ml[r].x - mx);
                        sum += f * ml[r].y;
                        acc.x += f * v[r].x, acc.y += f * v[r].y, acc.z += f * v[r].z, acc.w += f * v[r].w;
                    }
                    const float inv = 1.f / sum;
                    *(uint2*)(out_base + tab[mt * R + lr].out + c) =
                        make_uint2(pack_bf16(acc.x * inv, acc.y * inv), pack_bf16(acc.z * inv, acc.w * inv));
                }
                __syncwarp();
                cluster_sync();  // no CTA leaves while others read its results
            }
        } while (!CL && run.next(a));
    }
}

// ------------------------------------------------------------------- merge ---
//
// The item that team i begins and does not end: its parts are team i's second
// slot and the first slots of the teams after it, until the item's tiles are
// all accounted for.  Weights exp2(m - M) of the parts in team order.

// kBatch parts are loaded together: one after the other, each costs a trip to L2.  R = 128: 8 for items
// of many parts (100 rows over 32 K tokens: 26.1 us instead of 29.3), 4 where there are few (76 items of
// 4 K: 38.2 instead of 39.8).
template <int D, int R, int kBatch>
__global__ void __launch_bounds__(256) k_kv4_merge(Kv4Attn a)
{
    pdl_wait();
    pdl_trigger();
    // one warp per team and 128 floats of the item's rows, or (R = 128) 32 rows x 8 channels
    constexpr bool kCols = R == 128;
    const int rows = min(R, a.rows);
    const int groups = kCols ? (rows + 31) / 32 * (D / 8) : ceil_div(rows * D, 128);
    const int w = blockIdx.x * 8 + (threadIdx.x >> 5), i0 = w / groups, grp = w - i0 * groups, lane = threadIdx.x & 31;
    if (i0 >= a.nteams) return;
    const MergeRec* recs = (const MergeRec*)(a.part + (size_t)a.nteams * 2 * part_floats(R, D));
    const MergeRec rec = recs[i0];
    if (rec.rest == 0) return;
    const Shares sh = rec.sh;
    const long long end = sh.at(i0 + 1) + rec.rest;  // where the item ends
    const int head = rec.item / a.mtiles, mt = rec.item - head * a.mtiles, group = a.H / a.Hkv;
    const int lr = kCols ? grp / (D / 8) * 32 + lane : (grp * 128 + lane * 4) / D;
    const int c = kCols ? grp % (D / 8) * 8 : (grp * 128 + lane * 4) % D, gr = mt * R + lr;
    if (lr >= R || gr >= a.rows) return;
    constexpr int kV = kCols ? 8 : 4;
    float mx = kNoRef, sum = 0.f, acc[kV] = {};
    // the parts: team i0's second one, then the first ones of the teams after it up to the
    // item's end; joined in team order
#pragma unroll 1
    for (int i = i0; i == i0 || sh.at(i) < end; i += kBatch) {
        float m[kBatch], l[kBatch], v[kBatch][kV];
#pragma unroll
        for (int j = 0; j < kBatch; j++) {
            m[j] = kNoRef, l[j] = 0.f;
#pragma unroll
            for (int k = 0; k < kV; k++) v[j][k] = 0.f;
            const long long at = sh.at(i + j);
            if (at >= end || at == sh.at(i + j + 1)) continue;  // past the item, or a team without units
            const float* part = a.part + ((size_t)(i + j) * 2 + (i + j == i0 ? 1 : 0)) * part_floats(R, D);
            if (kCols) {
                m[j] = part[(size_t)R * D + lr], l[j] = part[(size_t)R * D + R + lr];
#pragma unroll
                for (int k = 0; k < kV; k++) v[j][k] = part[(size_t)(c + k) * R + lr];
            } else {
                const float2 ml = *(const float2*)(part + (size_t)R * D + 2 * lr);
                const float4 x = *(const float4*)(part + (size_t)lr * D + c);
                m[j] = ml.x, l[j] = ml.y, v[j][0] = x.x, v[j][1] = x.y, v[j][2] = x.z, v[j][3] = x.w;
            }
        }
#pragma unroll
        for (int j = 0; j < kBatch; j++) {
            const float top = fmaxf(mx, m[j]), f = ex2(mx - top), h = ex2(m[j] - top);
            mx = top;
            sum = sum * f + l[j] * h;
#pragma unroll
            for (int k = 0; k < kV; k++) acc[k] = acc[k] * f + v[j][k] * h;
        }
    }
    const float inv = 1.f / sum;
    uint32_t y[kV / 2];
#pragma unroll
    for (int k = 0; k < kV; k += 2) y[k / 2] = pack_bf16(acc[k] * inv, acc[k + 1] * inv);
    __nv_bfloat16* dst = a.out + ((size_t)(rec.b * (long long)a.T + gr / group) * a.H + head * group + gr % group) * D + c;
    if (kCols) *(uint4*)dst = make_uint4(y[0], y[1], y[kV / 2 - 2], y[kV / 2 - 1]);
    else *(uint2*)dst = make_uint2(y[0], y[1]);
}

// ---------------------------------------------------------------- launches ---

struct Plan {
    int tw, grid, nteams, mtiles, extra;
    int cluster;  // CTAs per item, 0: equal runs over the teams
    bool merge;
    size_t bytes;
};

int max_len_of(const la_kv4_desc& c, const la_kv4_attn& a)
{
    const int room = c.max_pages * c.page;
    return a.max_len > 0 && a.max_len < room ? a.max_len : room;
}

// CTAs per item, or 0 for equal runs, by what both cost in rounds of a tile per warp (1.55 us with two
// CTAs on an SM, about half of that while there is one).  A cluster goes as long as the longest item and 2
// rounds for queries and result, again for every 304 items; equal runs as long as all tiles and 7 rounds
// for the search of the starts, the parts and their merge.  Of a batch, three quarters of the longest
// length are taken for the average.  D = 128, 4 rows (us, clusters / runs):
//   1 sequence of 8 items: 400 tokens 4.5 / 8.3, 4 K 6.2 / 10.4, 16 K 11.3 / 15.0, 64 K 34.1 / 23.4
//   1 sequence of 100 items: 400 tokens 6.2 / 10.8, 4 K 18.0 / 18.0, 16 K 58.0 / 46.0
//   1/8 to full length, 250 sequences: to 400 tokens 6.1 / 12.1, to 4 K 28.5 / 24.1, to 16 K 103 / 62
//   likewise 900: to 400 tokens 15.1 / 18.6, 1200 to 1 K: 31.2 / 29.9, 2000 to 400: 31.3 / 28.4
int cluster_of(long long items, long long tiles, bool ragged)
{
    const double mean = ragged ? 0.75 : 1.0, ctas = 2.0 * kSMs;
    // (not all of a GPC's SMs fit into clusters of 4 and 8)
    int cs = items <= 32 ? 8 : items <= 64 ? 4 : items <= kSMs ? 2 : 1;
    while (cs > 1 && cs * kWarps >= 2 * tiles) cs /= 2;
    const double waves = std::ceil(items / ctas), shared = items * cs > kSMs / 2 ? 1.0 : 0.55;
    const double rounds = (double)tiles / (cs * kWarps) * shared * (waves > 1 ? waves * mean : 1.0);
    const double clusters = rounds + 2 * std::max(1.0, items / ctas), runs = items * tiles * mean / (ctas * kWarps) + 7;
    return clusters <= runs ? cs : 0;
}

Plan plan_of(const la_kv4_desc& c, const la_kv4_attn& a)
{
    Plan p;
    const int T = 1 + (a.W + a.G) * (a.N - 1), rows = T * (a.n_heads / c.n_kv_heads);
    p.mtiles = ceil_div(rows, 8);  // 1 or 2
    const long long items = (long long)a.batch * c.n_kv_heads * p.mtiles;
    const int ctas = 2 * kSMs;  // resident at once
    // A warp per team spares the CTA's barriers but splits few items too finely: 13B lookahead x 9 (720
    // items) 36 against 39 us, 7B greedy x 16 (512 items) 19.4 against 20.1, 34B greedy x 32 (256 items)
    // 45 against 28
    p.tw = items >= 512 ? 1 : kWarps;
    p.cluster = cluster_of(items, (max_len_of(c, a) + kKeys - 1) / kKeys + 1, a.batch > 1);
    // an item's queries and result take as long as so many tiles (32 keys); without them the teams
    // that get many short sequences finish last.  Warps: 128 greedy 7B sequences 64 us at 0, 57 at 1,
    // 61 at 4; CTAs: 16 long 34B sequences of 1 to 64 K tokens 132 us at 0, 121 at 14, 122 at 24
    p.extra = p.tw == 1 ? 1 : 14;
    const long long teams = (long long)ctas * (p.tw == 1 ? kWarps : 1);
    const long long tiles = items * ((max_len_of(c, a) + kKeys - 1) / kKeys + 1);  // at most
    p.nteams = (int)std::max(1LL, std::min(teams, std::max(items, tiles / kWarps)));
    p.grid = p.tw == 1 ? ceil_div(p.nteams, kWarps) : p.nteams;
    // one sequence: every item has the same tiles, so whole items a team stay whole
    p.merge = !p.cluster && !(a.batch == 1 && items % p.nteams == 0);
    p.bytes = p.merge ? (size_t)p.nteams * (2 * part_floats(8, c.head_dim) * 4 + sizeof(MergeRec)) : 0;
    return p;
}

std::mutex g_mu;
unsigned char g_ready[256];

template <int D, int TW, bool CL>
bool set_smem()
{
    auto kern = k_kv4_rows<D, TW, CL>;
    return cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, RowsSmem<D, TW, CL>::kBytes) == cudaSuccess &&
           cudaFuncSetAttribute(kern, cudaFuncAttributePreferredSharedMemoryCarveout, 100) == cudaSuccess;
}

// The kernels' shared-memory limits, once per device.
int attn_ready()
{
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 256) return LA_ERR_CUDA;
    std::lock_guard<std::mutex> lock(g_mu);
    if (!g_ready[dev]) {
        if (!(set_smem<128, 1, false>() && set_smem<128, kWarps, false>() && set_smem<128, kWarps, true>() &&
              set_smem<64, 1, false>() && set_smem<64, kWarps, false>() && set_smem<64, kWarps, true>() && kv4_tc_init()))
            return LA_ERR_CUDA;
        g_ready[dev] = 1;
    }
    return LA_OK;
}

template <int D>
cudaError_t go(cudaStream_t s, const Plan& p, const Kv4Attn& k)
{
    if (p.cluster)
        return launch_cluster(k_kv4_rows<D, kWarps, true>, (unsigned)(k.B * k.Hkv * k.mtiles), (unsigned)p.cluster, kThreads,
                              RowsSmem<D, kWarps, true>::kBytes, s, k);
    cudaError_t e = p.tw == 1 ? launch_pdl(k_kv4_rows<D, 1, false>, dim3(p.grid), dim3(kThreads), RowsSmem<D, 1, false>::kBytes, s, k)
                              : launch_pdl(k_kv4_rows<D, kWarps, false>, dim3(p.grid), dim3(kThreads), RowsSmem<D, kWarps, false>::kBytes, s, k);
    if (e == cudaSuccess && p.merge) e = launch_kv4_merge(s, k, D, 8);
    return e;
}

}  // namespace

cudaError_t launch_kv4_merge(cudaStream_t s, const Kv4Attn& k, int D, int R)
{
    const int rows = std::min(R, k.rows);
    const int groups = R == 128 ? (rows + 31) / 32 * (D / 8) : ceil_div(rows * D, 128);
    const bool many = k.nteams > 8LL * k.B * k.Hkv * k.mtiles;
    auto kern = R == 8 ? (D == 128 ? k_kv4_merge<128, 8, 8> : k_kv4_merge<64, 8, 8>)
                : many ? (D == 128 ? k_kv4_merge<128, 128, 8> : k_kv4_merge<64, 128, 8>)
                       : (D == 128 ? k_kv4_merge<128, 128, 4> : k_kv4_merge<64, 128, 4>);
    return launch_pdl(kern, dim3(ceil_div(k.nteams * groups, 8)), dim3(256), 0, s, k);
}

namespace {

// Rows of one KV head: up to 16, one or two tiles of the narrow side of
// mma.sync; more go to the 128-row tiles of tcgen05.
bool many_rows(const la_kv4_desc& c, const la_kv4_attn& a)
{
    return (1 + (a.W + a.G) * (a.N - 1)) * (a.n_heads / c.n_kv_heads) > 16;
}

}  // namespace

size_t kv4_attn_bytes(const la_kv4_desc& c, const la_kv4_attn& a)
{
    if (!a.batch) return 0;
    return many_rows(c, a) ? kv4_tc_bytes(c, a) : plan_of(c, a).bytes;
}

int launch_kv4_attn(cudaStream_t s, const la_kv4_desc& c, const la_kv4_attn& a)
{
    if (int rc = attn_ready()) return rc;
    Kv4Attn k;
    k.pages = (const uint8_t*)c.pages;
    k.q = (const __nv_bfloat16*)a.q, k.ks = (const __nv_bfloat16*)a.k_step, k.vs = (const __nv_bfloat16*)a.v_step;
    k.out = (__nv_bfloat16*)a.out;
    k.lens = a.lens, k.table = a.table, k.status = c.status;
    k.B = a.batch, k.H = a.n_heads, k.Hkv = c.n_kv_heads;
    k.W = a.W, k.n1 = a.N - 1, k.T = 1 + (a.W + a.G) * k.n1;
    k.q_ld = a.q_ld, k.kv_ld = a.kv_ld;
    k.n_pages = c.n_pages, k.max_pages = c.max_pages, k.max_len = max_len_of(c, a);
    k.blk_log2 = c.page == 16 ? 0 : c.page == 32 ? 1 : c.page == 64 ? 2 : 3;
    k.rows = k.T * (a.n_heads / c.n_kv_heads);
    k.sl2 = 1.4426950408889634f / sqrtf((float)c.head_dim);
    if (many_rows(c, a)) return launch_kv4_tc(s, c, a, k);
    const Plan p = plan_of(c, a);
    k.part = p.merge ? (float*)a.workspace : nullptr;
    k.mtiles = p.mtiles, k.nteams = p.nteams, k.extra = p.extra;
    k.tile_log2 = kKeysLog2;
    const cudaError_t e = c.head_dim == 128 ? go<128>(s, p, k) : go<64>(s, p, k);
    return e == cudaSuccess ? LA_OK : LA_ERR_CUDA;
}

}  // namespace la
