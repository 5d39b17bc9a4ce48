// kv4_attn.cu -- the step's masked attention over the paged 4-bit cache for
// few rows per KV head, on mma.sync: decode steps of single tokens, small
// lookahead steps, grouped heads.
//
// For one sequence and KV head ("item") the rows are the T step rows times the
// query heads that share the KV head, in tiles of 8 NB rows.  With a key's
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
//  * p s goes to fp16: relative 2^-11, or 2^-25 absolute where the running
//    reference keeps the largest between 1 and 2^8 (bf16 would cost 2^-8);
//  * z sum(p s) is subtracted by the tensor core too, by a second product
//    with -z in place of the codes: the outputs' sums return near zero in
//    every tile (they shrink as the context grows, z sum(p s) does not) and
//    no instruction per code is spent.
//
// Both products have the keys (K: 16 keys x 16 channels) or the channels (V:
// 16 channels x 16 keys) as the 16-row side of m16n8k16 and the query rows as
// the 8-wide side: a single token of a group of up to 8 heads fills it, and
// the probabilities go from one product's accumulators to the other's operand
// by an 8 x 8 transpose in registers.  Channels and keys are permuted so that
// each lane's fragments are contiguous bytes (kv4_key).
//
// HBM bound: D + 8 bytes a key and KV head.  One warp of a CTA streams blocks
// of 16 keys (one contiguous bulk copy each) into a ring for each of the
// others, so no warp waits for another inside an item.  The running reference
// M moves only when a p s exceeds 2^8 (a vote, no reduction per tile).
//
// Items are cut into equal runs of blocks over the teams (a warp, or a CTA
// whose warps' partial results meet in shared memory), whatever the
// sequences' lengths; an item that falls to several teams leaves partial
// outputs, which k_kv4_merge joins in a fixed order.
#include <algorithm>
#include <climits>
#include <cmath>
#include <cstdlib>
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

__device__ __forceinline__ float max_nan(float a, float b)
{
    float y;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(y) : "f"(a), "f"(b));
    return y;
}

// bf16 pair with its NaNs and infinities replaced by 0; whether there were any
__device__ __forceinline__ bool drop_nonfinite(uint32_t& u)
{
    const bool lo = (u & 0x7f80u) == 0x7f80u, hi = (u & 0x7f800000u) == 0x7f800000u;
    if (lo) u &= 0xffff0000u;
    if (hi) u &= 0x0000ffffu;
    return lo || hi;
}

constexpr float kMinScale = 0x1p-92f;  // V scales below it count as it (values under 2^-88)

// ------------------------------------------------------------------ kernel ---

template <int D, int NB, int TW>
struct RowsSmem {
    static constexpr int kR = 8 * NB;
    static constexpr int kStages = NB == 1 && TW > 1 ? 2 : 3;
    static constexpr int kBlk = 2 * kv4_block_bytes(D);
    static constexpr int kRing = kWarps * kStages * kBlk;
    static constexpr int kBar = kRing;                                          // full, empty
    static constexpr int kLive = kBar + kWarps * kStages * 16;                  // keys of each stage's block
    static constexpr int kMisc = kLive + (kWarps * kStages * 4 + 15) / 16 * 16;  // starts and scan scratch
    static constexpr int kMerge = kMisc + (kWarps * (int)sizeof(Start) + (kWarps + 2) * 8 + 15) / 16 * 16;
    static constexpr int kMergeBytes = TW == 1 ? 0 : kWarps * kR * (D + 4) * 4;  // [warp][row][D | M, sum]
    static constexpr int kBytes = kMerge + kMergeBytes;
    static_assert(kMisc % 8 == 0 && kMerge % 16 == 0, "alignment");
};

constexpr int kThreads = (kWarps + 1) * 32;

// Warp kWarps: lane w fills the ring of warp w, block by block in the order in
// which that warp takes them.  The lanes poll their rings' empty barriers in
// turn; the page of the next block is looked up a round ahead.
template <int D, int TW, int S>
__device__ __forceinline__ void produce(const Kv4Attn& a, const Start& st, uint8_t* ring, uint64_t* full, uint64_t* empty,
                                        int* live, int wi)
{
    const uint64_t pol = policy_evict_first();
    Run r;
    r.left = 0;
    r.t0 = r.t1 = 0;
    bool more = st.count > 0;
    if (more) r.begin(a, st);
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
                head = r.item / a.mtiles;
                blk = (2 * t) & ((1 << a.blk_log2) - 1);
                pend = true;
                t += TW;
                return;
            }
            more = r.next(a);
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

template <int D, int NB, int TW>
__global__ void __launch_bounds__(kThreads, NB == 1 ? 2 : 1) k_kv4_rows(Kv4Attn a)
{
    using L = RowsSmem<D, NB, TW>;
    constexpr int S = L::kStages, R = L::kR, PAN = D / 64, MB = D / 16, DV = D / 8, BLK = kv4_block_bytes(D);
    extern __shared__ __align__(128) uint8_t sm[];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
    uint64_t *full = (uint64_t*)(sm + L::kBar), *empty = full + kWarps * S;
    int* live_of = (int*)(sm + L::kLive);
    Start* starts = (Start*)(sm + L::kMisc);
    if (threadIdx.x < kWarps * S) {
        mbar_init(full + threadIdx.x, 1);
        mbar_init(empty + threadIdx.x, 1);
        mbar_fence_init();
    }
    pdl_wait();
    pdl_trigger();
    if (blockIdx.x == 0) raise_long(a);
    // (its barriers also publish the mbarriers)
    find_starts(a, TW == 1 ? blockIdx.x * kWarps : blockIdx.x, TW == 1 ? kWarps : 1, starts, (long long*)(starts + kWarps));
    if (warp == kWarps) {
        const int w = min(lane, kWarps - 1);
        Start st = starts[TW == 1 ? w : 0];
        if (lane >= kWarps) st.count = 0;
        produce<D, TW, S>(a, st, sm + w * S * L::kBlk, full + w * S, empty + w * S, live_of + w * S, TW == 1 ? 0 : w);
        return;
    }
    const int wi = TW == 1 ? 0 : warp;  // this warp's place in its team
    const int team = TW == 1 ? blockIdx.x * kWarps + warp : blockIdx.x;
    const Start st = starts[TW == 1 ? warp : 0];
    const uint8_t* ring = sm + warp * S * L::kBlk;
    full += warp * S, empty += warp * S, live_of += warp * S;
    MergeRec* rec = (MergeRec*)(a.part + (size_t)a.nteams * 2 * part_floats(R, D)) + team;
    const bool writes_rec = a.part && team < a.nteams && lane == 0 && wi == 0;
    if (writes_rec) rec->rest = 0;
    const int group = a.H / a.Hkv;
    bool alive = true;  // no wait has given up
    int s = 0, phase = 0;
    Run run;
    run.left = 0;
    if (st.count > 0) {
        run.begin(a, st);
        bool first = true;
        do {
            const int head = run.item / a.mtiles, mt = run.item - head * a.mtiles;
            const int ntc = (run.len + kKeys - 1) / kKeys;
            // the step's rows of this KV head are needed last: have them near by then
            if (run.t1 > ntc && lane < min(a.T, 16)) {
                const size_t at = (size_t)(run.b * (long long)a.T + lane) * a.kv_ld + (size_t)head * D;
                prefetch_l1(a.ks + at), prefetch_l1(a.vs + at);
                if (D == 128) prefetch_l1(a.ks + at + 64), prefetch_l1(a.vs + at + 64);
            }
            auto q_row = [&](int nb) {
                const int r = mt * R + nb * 8 + g;
                return a.q + (size_t)(run.b * (long long)a.T + r / group) * a.q_ld + (size_t)(head * group + r % group) * D + 16 * t;
            };
            float o[NB][MB][4], m[NB][2], l[NB][2];
#pragma unroll
            for (int nb = 0; nb < NB; nb++) {
                m[nb][0] = m[nb][1] = kNoRef;
                l[nb][0] = l[nb][1] = 0.f;
#pragma unroll
                for (int i = 0; i < MB; i++)
#pragma unroll
                    for (int j = 0; j < 4; j++) o[nb][i][j] = 0.f;
            }
            // Move the reference of row 2t + r to the largest y = log2(p s) of the tile; y(i) is
            // the largest of this lane's for row 2t + (i & 1) of row block i >> 1.
            auto raise_ref = [&](auto&& y) {
#pragma unroll
                for (int nb = 0; nb < NB; nb++)
#pragma unroll
                    for (int r = 0; r < 2; r++) {
                        float mx = y(nb, r);
                        mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 4));
                        mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 8));
                        mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 16));
                        mx = fmaxf(mx, m[nb][r]);
                        const float c = ex2(m[nb][r] - mx);
                        m[nb][r] = mx;
                        l[nb][r] *= c;
#pragma unroll
                        for (int i = 0; i < MB; i++) o[nb][i][r] *= c, o[nb][i][r + 2] *= c;
                    }
            };
            if (run.t0 + wi < min(run.t1, ntc)) {
                // ---------------------------------------------- cached keys
                // this lane's part of the query rows: row 8 nb + g, channels 64 p + 16 t ..
                uint32_t q[NB][PAN][8];
                float qs[NB][2], qf[NB][2];  // rows 2t, 2t + 1: sum of q, what undoes q's and the codes' powers of two
#pragma unroll
                for (int nb = 0; nb < NB; nb++) {
                    const bool valid = mt * R + nb * 8 + g < a.rows;
                    const __nv_bfloat16* src = q_row(nb);
                    uint32_t raw[PAN][8];
                    float sum = 0.f, top = 0.f;
#pragma unroll
                    for (int p = 0; p < PAN; p++) {
                        uint4 u0 = make_uint4(0, 0, 0, 0), u1 = u0;
                        if (valid) {
                            u0 = *(const uint4*)(src + 64 * p);
                            u1 = *(const uint4*)(src + 64 * p + 8);
                        }
                        raw[p][0] = u0.x, raw[p][1] = u0.y, raw[p][2] = u0.z, raw[p][3] = u0.w;
                        raw[p][4] = u1.x, raw[p][5] = u1.y, raw[p][6] = u1.z, raw[p][7] = u1.w;
#pragma unroll
                        for (int i = 0; i < 8; i++) {
                            const float lo = __uint_as_float(raw[p][i] << 16), hi = __uint_as_float(raw[p][i] & 0xffff0000u);
                            sum += lo + hi;
                            top = fmaxf(top, fmaxf(fabsf(lo), fabsf(hi)));
                        }
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
                            q[nb][p][i] = pack_f16(__uint_as_float(raw[p][i] << 16) * f,
                                                   __uint_as_float(raw[p][i] & 0xffff0000u) * f);
                        }
                    qs[nb][0] = __shfl_sync(0xffffffffu, sum * a.sl2, 8 * t);
                    qs[nb][1] = __shfl_sync(0xffffffffu, sum * a.sl2, 8 * t + 4);
                    qf[nb][0] = __shfl_sync(0xffffffffu, up * a.sl2, 8 * t);
                    qf[nb][1] = __shfl_sync(0xffffffffu, up * a.sl2, 8 * t + 4);
                }
                const int k0 = kv4_key(g), k1 = k0 + 8;
                const int kA = t, kB = 4 + (t ^ 3);  // V's keys: probability slots 2t, 2t + 1; + 8: slots 2t + 8, 2t + 9
                for (int tile = run.t0 + wi; tile < min(run.t1, ntc); tile += TW) {
                    if (alive && !mbar_try_wait(full + s, phase)) {
                        const unsigned long long since = globaltimer();
                        while (!mbar_try_wait(full + s, phase))
                            if (globaltimer() - since > kWaitNs) {
                                alive = false;
                                kv4_raise(a.status, LA_ERR_TIMEOUT);
                                break;
                            }
                    }
                    const uint8_t* stage = ring + s * L::kBlk;
                    const int live = live_of[s];
                    float x[2][NB][4], sv[2][2];  // per block: scores; V scales of the keys k0, k1
#pragma unroll
                    for (int u = 0; u < 2; u++) {
                        const uint8_t* blk = stage + u * BLK;
#pragma unroll
                        for (int nb = 0; nb < NB; nb++) x[u][nb][0] = x[u][nb][1] = x[u][nb][2] = x[u][nb][3] = 0.f;
#pragma unroll
                        for (int p = 0; p < PAN; p++) {
                            const uint2 w0 = *(const uint2*)(blk + p * 512 + k0 * 32 + t * 8);
                            const uint2 w1 = *(const uint2*)(blk + p * 512 + k1 * 32 + t * 8);
#pragma unroll
                            for (int i = 0; i < 4; i++) {
                                uint32_t u0 = i < 2 ? w0.x : w0.y, u1 = i < 2 ? w1.x : w1.y;
                                if (i & 1) u0 >>= 8, u1 >>= 8;
#pragma unroll
                                for (int nb = 0; nb < NB; nb++)
                                    mma_f16(x[u][nb], u0 & kLo, u1 & kLo, u0 & kHi, u1 & kHi, q[nb][p][2 * i], q[nb][p][2 * i + 1]);
                            }
                        }
                        const uint32_t* par = (const uint32_t*)(blk + 16 * D);  // K, then V
                        const uint32_t p0 = par[k0], p1 = par[k1];
                        const float s0 = __uint_as_float(p0 & 0xffff0000u), s1 = __uint_as_float(p1 & 0xffff0000u);
                        const float z0 = 128.f - __uint_as_float(p0 << 16), z1 = 128.f - __uint_as_float(p1 << 16);  // -z
                        sv[u][0] = max_nan(__uint_as_float(par[16 + k0] & 0xffff0000u), kMinScale);
                        sv[u][1] = max_nan(__uint_as_float(par[16 + k1] & 0xffff0000u), kMinScale);
#pragma unroll
                        for (int nb = 0; nb < NB; nb++)
#pragma unroll
                            for (int r = 0; r < 2; r++) {
                                x[u][nb][r] = s0 * fmaf(x[u][nb][r], qf[nb][r], z0 * qs[nb][r]);
                                x[u][nb][r + 2] = s1 * fmaf(x[u][nb][r + 2], qf[nb][r], z1 * qs[nb][r]);
                            }
                    }
                    if (live != 0x1010) {
                        // the last blocks of a sequence (or a bad page): the rest may hold anything
#pragma unroll
                        for (int u = 0; u < 2; u++) {
                            const int n = (live >> (8 * u)) & 255;
#pragma unroll
                            for (int nb = 0; nb < NB; nb++)
#pragma unroll
                                for (int r = 0; r < 2; r++) {
                                    if (k0 >= n) x[u][nb][r] = -INFINITY;
                                    if (k1 >= n) x[u][nb][r + 2] = -INFINITY;
                                }
                            if (k0 >= n) sv[u][0] = kMinScale;
                            if (k1 >= n) sv[u][1] = kMinScale;
                        }
                    }
                    float e[2][NB][4];              // probabilities
                    uint32_t b0[2][NB], b1[2][NB];  // p s of the keys k0 and k1, rows 2t and 2t + 1
                    auto weigh = [&]() {            // whether some p s is above 2^8
                        __half2 top = __float2half2_rn(0.f);
#pragma unroll
                        for (int u = 0; u < 2; u++)
#pragma unroll
                            for (int nb = 0; nb < NB; nb++) {
#pragma unroll
                                for (int i = 0; i < 4; i++) e[u][nb][i] = ex2(x[u][nb][i] - m[nb][i & 1]);
                                b0[u][nb] = pack_f16(e[u][nb][0] * sv[u][0], e[u][nb][1] * sv[u][0]);
                                b1[u][nb] = pack_f16(e[u][nb][2] * sv[u][1], e[u][nb][3] * sv[u][1]);
                                top = __hmax2(top, __hmax2(*(__half2*)&b0[u][nb], *(__half2*)&b1[u][nb]));
                            }
                        return !__hble2(top, __float2half2_rn(256.f));
                    };
                    if (__any_sync(0xffffffffu, weigh())) {
                        raise_ref([&](int nb, int r) {
                            float y = kNoRef;
#pragma unroll
                            for (int u = 0; u < 2; u++)
                                y = fmaxf(y, fmaxf(x[u][nb][r] + __log2f(sv[u][0]), x[u][nb][r + 2] + __log2f(sv[u][1])));
                            return y;
                        });
                        weigh();
                    }
#pragma unroll
                    for (int u = 0; u < 2; u++) {
                        const uint8_t* blk = stage + u * BLK;
                        const uint32_t* vpar = (const uint32_t*)(blk + 16 * D + 64);
                        const uint32_t vA = vpar[kA], vB = vpar[kB], vC = vpar[8 + kA], vE = vpar[8 + kB];
#pragma unroll
                        for (int nb = 0; nb < NB; nb++) {
                            l[nb][0] += e[u][nb][0] + e[u][nb][2];
                            l[nb][1] += e[u][nb][1] + e[u][nb][3];
                            b0[u][nb] = transpose8(b0[u][nb]);
                            b1[u][nb] = transpose8(b1[u][nb]);
                        }
                        // -z of the same keys as fp16 2^-24 z and 2^-20 z
                        const uint32_t zAB = __byte_perm(vA, vB, 0x5410) & kLo, zCE = __byte_perm(vC, vE, 0x5410) & kLo;
                        const uint32_t zl0 = zAB | 0x80008000u, zl1 = zCE | 0x80008000u;
                        const uint32_t zh0 = (zAB * 16) | 0x80008000u, zh1 = (zCE * 16) | 0x80008000u;
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
#pragma unroll
                                    for (int nb = 0; nb < NB; nb++)
                                        mma_f16(o[nb][(hf * 4 + j) % MB], ab0 & mk, ab1 & mk, ce0 & mk, ce1 & mk, b0[u][nb], b1[u][nb]);
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
#pragma unroll
                                for (int nb = 0; nb < NB; nb++)
                                    mma_f16(o[nb][j], ab0 & mk, ab1 & mk, ce0 & mk, ce1 & mk, b0[u][nb], b1[u][nb]);
                            }
                        }
#pragma unroll
                        for (int j = 0; j < MB; j++)
#pragma unroll
                            for (int nb = 0; nb < NB; nb++)
                                mma_f16(o[nb][j], j & 1 ? zh0 : zl0, j & 1 ? zh0 : zl0, j & 1 ? zh1 : zl1, j & 1 ? zh1 : zl1, b0[u][nb],
                                        b1[u][nb]);
                    }
                    __syncwarp();  // every lane has read the stage
                    if (lane == 0) mbar_arrive(empty + s);
                    if (++s == S) s = 0, phase ^= 1;
                }
            }
            // ------------------------------------------ the step's own rows
            // (in bf16, with their values brought to the codes' powers of two)
            int tile = run.t0 + wi;
            if (tile < ntc) tile += (ntc - tile + TW - 1) / TW * TW;
            for (; tile < run.t1; tile += TW) {
                const int j0 = (tile - ntc) * 16;
                const size_t col = (size_t)head * D;
                auto row = [&](const __nv_bfloat16* base, int j) {
                    return base + (size_t)(run.b * (long long)a.T + j) * a.kv_ld + col;
                };
                const int k0 = j0 + kv4_key(g), k1 = k0 + 8;
                float x[NB][4];
#pragma unroll
                for (int nb = 0; nb < NB; nb++) x[nb][0] = x[nb][1] = x[nb][2] = x[nb][3] = 0.f;
#pragma unroll
                for (int p = 0; p < PAN; p++)
#pragma unroll
                    for (int i = 0; i < 2; i++) {
                        uint4 u0 = make_uint4(0, 0, 0, 0), u1 = u0;
                        if (k0 < a.T) u0 = *(const uint4*)(row(a.ks, k0) + 64 * p + 16 * t + 8 * i);
                        if (k1 < a.T) u1 = *(const uint4*)(row(a.ks, k1) + 64 * p + 16 * t + 8 * i);
#pragma unroll
                        for (int nb = 0; nb < NB; nb++) {
                            uint4 u = make_uint4(0, 0, 0, 0);
                            if (mt * R + nb * 8 + g < a.rows) u = *(const uint4*)(q_row(nb) + 64 * p + 8 * i);
                            mma_b16(x[nb], u0.x, u1.x, u0.y, u1.y, u.x, u.y);
                            mma_b16(x[nb], u0.z, u1.z, u0.w, u1.w, u.z, u.w);
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
                raise_ref([&](int nb, int r) { return fmaxf(x[nb][r], x[nb][r + 2]); });
                uint32_t b0[NB][2], b1[NB][2];
#pragma unroll
                for (int nb = 0; nb < NB; nb++) {
                    float e[4];
#pragma unroll
                    for (int i = 0; i < 4; i++) e[i] = ex2(x[nb][i] - m[nb][i & 1]);
                    l[nb][0] += e[0] + e[2];
                    l[nb][1] += e[1] + e[3];
#pragma unroll
                    for (int h = 0; h < 2; h++) {
                        const float f = h ? 0x1p-20f : 0x1p-24f;
                        b0[nb][h] = transpose8(pack_bf16(e[0] * f, e[1] * f));
                        b1[nb][h] = transpose8(pack_bf16(e[2] * f, e[3] * f));
                    }
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
                    for (int i = 0; i < 4; i++) {
                        v[i] = make_uint4(0, 0, 0, 0);
                        if (key[i] < a.T) v[i] = *(const uint4*)(row(a.vs, key[i]) + DV * g + 8 * half);
                        odd |= drop_nonfinite(v[i].x) | drop_nonfinite(v[i].y) | drop_nonfinite(v[i].z) | drop_nonfinite(v[i].w);
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
                                mma_b16(o[nb][j % MB], half ? 0u : ab, half ? ab : 0u, half ? 0u : ce, half ? ce : 0u, b0[nb][j & 1],
                                        b1[nb][j & 1]);
                        }
                    } else {
#pragma unroll
                        for (int j = 0; j < 4; j++) {
                            const uint32_t a0 = __byte_perm(vA[j], vB[j], 0x5410), a1 = __byte_perm(vA[j], vB[j], 0x7632);
                            const uint32_t a2 = __byte_perm(vC[j], vE[j], 0x5410), a3 = __byte_perm(vC[j], vE[j], 0x7632);
#pragma unroll
                            for (int nb = 0; nb < NB; nb++) mma_b16(o[nb][j], a0, a1, a2, a3, b0[nb][j & 1], b1[nb][j & 1]);
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
            // ---- the item's (or the run's) result
#pragma unroll
            for (int nb = 0; nb < NB; nb++)
#pragma unroll
                for (int r = 0; r < 2; r++) {
                    l[nb][r] += __shfl_xor_sync(0xffffffffu, l[nb][r], 4);
                    l[nb][r] += __shfl_xor_sync(0xffffffffu, l[nb][r], 8);
                    l[nb][r] += __shfl_xor_sync(0xffffffffu, l[nb][r], 16);
                }
            const bool whole = run.u0 == 0 && run.u1 == run.nu;
            float* part = a.part + ((size_t)team * 2 + (run.u0 == 0 ? 1 : 0)) * part_floats(R, D);
            if (run.u0 == 0 && !whole && writes_rec) *rec = MergeRec{run.b, run.item, run.nu - run.u1, 0, starts[TW == 1 ? warp : 0].sh};
            // channel c (of DV, from DV g) of row 2t + r
            auto chan = [&](int nb, int r, int c) -> float {
                const int mb = D == 128 ? ((c & 7) >> 1) + 4 * (c & 1) : c >> 1, hi = D == 128 ? c >> 3 : c & 1;
                return o[nb][mb % MB][r + 2 * hi] * (mb & 1 ? 0x1p20f : 0x1p24f);
            };
            auto out_row = [&](int gr) {
                return a.out + ((size_t)(run.b * (long long)a.T + gr / group) * a.H + head * group + gr % group) * D;
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
                            __nv_bfloat16* dst = out_row(gr) + DV * g;
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
                if (!first) named_sync(1, kWarps * 32);  // the last item's results have been read
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
                named_sync(1, kWarps * 32);
                for (int i = threadIdx.x; i < R * D / 4; i += kWarps * 32) {
                    const int lr = i / (D / 4), c = (i % (D / 4)) * 4, gr = mt * R + lr;
                    if (gr >= a.rows) continue;
                    float2 ml[kWarps];
                    float mx = -INFINITY;
#pragma unroll
                    for (int w = 0; w < kWarps; w++) {
                        ml[w] = *(const float2*)(mg + ((size_t)w * R + lr) * (D + 4) + D);
                        mx = fmaxf(mx, ml[w].x);
                    }
                    const float mu = fmaxf(mx, kNoRef);
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
                        *(uint2*)(out_row(gr) + c) = make_uint2(pack_bf16(acc.x * inv, acc.y * inv), pack_bf16(acc.z * inv, acc.w * inv));
                    } else {
                        *(float4*)(part + (size_t)lr * D + c) = acc;
                        if (c == 0) *(float2*)(part + (size_t)R * D + 2 * lr) = make_float2(mx, sum);
                    }
                }
                first = false;
            }
        } while (run.next(a));
    }
}

// ------------------------------------------------------------------- merge ---
//
// The item that team i begins and does not end: its parts are team i's second
// slot and the first slots of the teams after it, until the item's tiles are
// all accounted for.  Weights exp2(m - M) of the parts in team order.

constexpr int kMergeChunks = 4;

template <int D, int R>
__global__ void __launch_bounds__(256) k_kv4_merge(Kv4Attn a)
{
    pdl_wait();
    pdl_trigger();
    // one warp per team and 128 floats of the item's rows (R <= 16: of 4 kMergeChunks channels),
    // or 32 rows x 8 channels (R = 128)
    constexpr bool kCols = R == 128;
    const int rows = min(R, a.rows);
    const int groups = kCols ? (rows + 31) / 32 * (D / 8) : ceil_div(ceil_div(rows * D, 128), kMergeChunks);
    const int w = blockIdx.x * 8 + (threadIdx.x >> 5), i0 = w / groups, lane = threadIdx.x & 31;
    if (i0 >= a.nteams) return;
    const MergeRec* recs = (const MergeRec*)(a.part + (size_t)a.nteams * 2 * part_floats(R, D));
    const MergeRec rec = recs[i0];
    if (rec.rest == 0) return;
    const Shares sh = rec.sh;
    const long long end = sh.at(i0 + 1) + rec.rest;  // where the item ends
    const int head = rec.item / a.mtiles, mt = rec.item % a.mtiles, group = a.H / a.Hkv;
    auto out_at = [&](int gr, int c) {
        return a.out + ((size_t)(rec.b * (long long)a.T + gr / group) * a.H + head * group + gr % group) * D + c;
    };
    // the parts: team i0's second one, then the first ones of the teams after it up to the item's end
    auto part_of = [&](int i) { return a.part + ((size_t)i * 2 + (i == i0 ? 1 : 0)) * part_floats(R, D); };
    if (kCols) {
        const int g = w % groups, lr = g / (D / 8) * 32 + lane, c = g % (D / 8) * 8, gr = mt * R + lr;
        if (gr >= a.rows) return;
        float mx = kNoRef, sum = 0.f, acc[8] = {};
        for (int i = i0; i == i0 || sh.at(i) < end; i++) {
            if (sh.at(i) == sh.at(i + 1)) continue;  // a team without units
            const float* part = part_of(i);
            const float m = part[(size_t)R * D + lr], l = part[(size_t)R * D + R + lr];
            float v[8];
#pragma unroll
            for (int k = 0; k < 8; k++) v[k] = part[(size_t)(c + k) * R + lr];
            const float top = fmaxf(mx, m), f = ex2(mx - top), h = ex2(m - top);
            mx = top;
            sum = sum * f + l * h;
#pragma unroll
            for (int k = 0; k < 8; k++) acc[k] = acc[k] * f + v[k] * h;
        }
        const float inv = 1.f / sum;
        *(uint4*)out_at(gr, c) = make_uint4(pack_bf16(acc[0] * inv, acc[1] * inv), pack_bf16(acc[2] * inv, acc[3] * inv),
                                            pack_bf16(acc[4] * inv, acc[5] * inv), pack_bf16(acc[6] * inv, acc[7] * inv));
        return;
    }
    const int c0 = (w % groups) * kMergeChunks;
#pragma unroll
    for (int ch = 0; ch < kMergeChunks; ch++) {
        const int at = (c0 + ch) * 128 + lane * 4, lr = at / D, c = at % D, gr = mt * R + lr;
        if (lr >= R || gr >= a.rows) return;
        float mx = kNoRef, sum = 0.f;
        float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
        for (int i = i0; i == i0 || sh.at(i) < end; i++) {
            if (sh.at(i) == sh.at(i + 1)) continue;
            const float* part = part_of(i);
            const float2 ml = *(const float2*)(part + (size_t)R * D + 2 * lr);
            const float4 v = *(const float4*)(part + (size_t)lr * D + c);
            const float top = fmaxf(mx, ml.x), f = ex2(mx - top), h = ex2(ml.x - top);
            mx = top;
            sum = sum * f + ml.y * h;
            acc.x = acc.x * f + v.x * h, acc.y = acc.y * f + v.y * h, acc.z = acc.z * f + v.z * h, acc.w = acc.w * f + v.w * h;
        }
        const float inv = 1.f / sum;
        *(uint2*)out_at(gr, c) = make_uint2(pack_bf16(acc.x * inv, acc.y * inv), pack_bf16(acc.z * inv, acc.w * inv));
    }
}

// ---------------------------------------------------------------- launches ---

struct Plan {
    int nb, tw, grid, nteams, mtiles, extra;
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
    const long long tiles = items * ((max_len_of(c, a) + kKeys - 1) / kKeys + (T + 15) / 16);  // at most
    const int ctas = p.nb == 1 ? 2 * kSMs : kSMs;  // resident at once
    p.tw = items >= (long long)ctas * kWarps ? 1 : kWarps;
    // an item's queries and result take as long as so many tiles (32 keys); without them the teams
    // that get many short sequences finish last.  128 greedy 7B sequences: 86 us at 0, 66 at 4, 71 at 8;
    // CTA teams on 16 long 34B sequences of 1 to 64 K: 124 us at 0, 117 at 21, 118 at 42
    p.extra = p.tw == 1 ? 4 : 18;
    const long long teams = (long long)ctas * (p.tw == 1 ? kWarps : 1);
    p.nteams = (int)std::max(1LL, std::min(teams, std::max(items, tiles / kWarps)));
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
        if (!(set_smem<128, 1, 1>() && set_smem<128, 1, kWarps>() && set_smem<128, 2, 1>() && set_smem<128, 2, kWarps>() &&
              set_smem<64, 1, 1>() && set_smem<64, 1, kWarps>() && set_smem<64, 2, 1>() && set_smem<64, 2, kWarps>() && kv4_tc_init()))
            return LA_ERR_CUDA;
        g_ready[dev] = 1;
    }
    return LA_OK;
}

template <int D, int NB>
cudaError_t go(cudaStream_t s, const Plan& p, const Kv4Attn& k)
{
    cudaError_t e = p.tw == 1 ? launch_pdl(k_kv4_rows<D, NB, 1>, dim3(p.grid), dim3(kThreads), RowsSmem<D, NB, 1>::kBytes, s, k)
                              : launch_pdl(k_kv4_rows<D, NB, kWarps>, dim3(p.grid), dim3(kThreads), RowsSmem<D, NB, kWarps>::kBytes, s, k);
    if (e == cudaSuccess && p.merge) e = launch_kv4_merge(s, k, D, 8 * NB);
    return e;
}

}  // namespace

cudaError_t launch_kv4_merge(cudaStream_t s, const Kv4Attn& k, int D, int R)
{
    const int rows = std::min(R, k.rows);
    const int groups = R == 128 ? (rows + 31) / 32 * (D / 8) : ceil_div(ceil_div(rows * D, 128), kMergeChunks);
    auto kern = D == 128 ? (R == 8 ? k_kv4_merge<128, 8> : R == 16 ? k_kv4_merge<128, 16> : k_kv4_merge<128, 128>)
                         : (R == 8 ? k_kv4_merge<64, 8> : R == 16 ? k_kv4_merge<64, 16> : k_kv4_merge<64, 128>);
    return launch_pdl(kern, dim3(ceil_div(k.nteams * groups, 8)), dim3(256), 0, s, k);
}

namespace {

// Rows of one KV head: up to 8 fill the narrow side of mma.sync; more go to
// the 128-row tiles of tcgen05.
bool many_rows(const la_kv4_desc& c, const la_kv4_attn& a)
{
    return (1 + (a.W + a.G) * (a.N - 1)) * (a.n_heads / c.n_kv_heads) > (getenv("KV_T") ? atoi(getenv("KV_T")) : 16);
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
    k.tile_log2 = kKeysLog2, k.step_tiles = (k.T + 15) / 16;
    const cudaError_t e = c.head_dim == 128 ? (p.nb == 1 ? go<128, 1>(s, p, k) : go<128, 2>(s, p, k))
                                            : (p.nb == 1 ? go<64, 1>(s, p, k) : go<64, 2>(s, p, k));
    return e == cudaSuccess ? LA_OK : LA_ERR_CUDA;
}

}  // namespace la
