// kv4_attn_tc.cu -- the step's masked attention over the paged 4-bit cache for
// many rows per KV head, on tcgen05: lookahead steps, prompt blocks, grouped
// heads with several step rows.
//
// An item is 128 rows (step rows x query heads of one KV head) of a sequence;
// its keys come in tiles of 128: cached ones, then one tile of the step's own
// rows under the mask.  Per tile, in fp16 with fp32 sums:
//   S = Q K^T          Q and K in shared memory, S in tensor memory
//   P = exp2(S f - M)  into columns of its own
//   O += P V           P from tensor memory, V in shared memory
// K and V are unpacked by 8 warps, one key row per two threads: masking two
// codes out of a word leaves fp16 subnormals (c 2^-24 or c 2^-20), and one
// fused multiply-add a pair gives (c - z) s, brought to the tile's own power
// of two: with E the largest scale's, s 2^-E < 2^-8, so a code step has at
// least 11 bits where the scale is within 2^-6 of the tile's largest and loses
// 2^-25 absolute below.  Rounding: q exact (a power of two per row), K and V
// values 2^-11 relative, P 2^-11, the output to bf16; S, the softmax sums and
// O stay in fp32.  The tiles' powers of two go into the exponent of exp2 and,
// for V, into the running reference M, which moves only when a row's P of a
// tile sum to more than 2^15.
//
// Tensor and exponential bound for full row tiles (128 x 128 x D x 2 products
// and 128 x 128 exponentials a tile: about 1024 cycles each at D = 128), HBM and
// unpacking bound for few rows.  All roles run at once on neighbouring tiles,
// one CTA per SM: warps 0-7 softmax (a row per thread; warps 0-3 the even
// tiles, 4-7 the odd ones, so that one group's exponentials run while the
// other waits), 8-11 unpack K, 12-15 V, 16 issues the MMAs, 17 copies code
// blocks ahead, 18 finds the tiles' powers of two.  S, P, K and V are double
// buffered, codes triple.
//
// Two ways to share an item's tiles: equal runs of all items' units over the
// SMs, parts joined by k_kv4_merge (many items, long ragged batches); or a
// cluster of 1 to 8 CTAs per item that join their outputs through distributed
// shared memory (up to 152 items: one launch, no workspace).
//
// Measured on one GB300.  121 rows of 32 heads over 2048 tokens (128 CTAs, 4 or
// 5 tiles each): 17.0 us in a graph, 2.1 of them by the tensor cores' rate; the rest is a
// chain of latencies (launch and first loads 3 us, 6 us a CTA for queries, first
// tile and unpacking, 2.5 us for the cluster's join).  6 such sequences: 52 us,
// 0.24 of the tensor cores' rate in steady state (1.6 us a tile): the softmax
// groups and the unpacking warps alternate on the schedulers (45 % of issue
// slots, tensor pipe 25 %); short prompt blocks: 128 rows over at most 11 tokens,
// 1872 items, 119 us = 9.7 us an item, the step's rows' way through bf16 to fp16
// and the queries' being the longest chain.
#include <algorithm>
#include <cmath>

#include "kv4_sched.cuh"

namespace la {

namespace {

constexpr int kTcThreads = 608;
constexpr int kTileLog2 = 7, kTile = 128;
constexpr int kRowsTc = 128;
constexpr int kRing = 3;

constexpr uint32_t idesc_f16(int M, int N, bool b_mn)
{
    return idesc_bf16(M, N, b_mn) & ~((1u << 7) | (1u << 10));  // A and B in fp16
}

// The MMAs of one product of a tile, by one elected lane.  The operands'
// descriptors advance by constants; the warp keeps everything uniform, so that
// nothing but an add goes before each instruction (issued by a single lane's
// code path with addresses of its own, an MMA cost 165 cycles).
__device__ __forceinline__ bool elect_one()
{
    uint32_t p;
    asm volatile("{\n .reg .pred p;\n elect.sync _|p, 0xffffffff;\n selp.u32 %0, 1, 0, p;\n}\n" : "=r"(p));
    return p != 0;
}

// D += A B, A and B in shared memory
__device__ __forceinline__ void mma_ss(uint32_t d_tmem, uint32_t a_lo, uint32_t b_lo, uint32_t hi, uint32_t idesc, bool acc)
{
    asm volatile(
        "{\n .reg .pred p;\n .reg .b64 x, y;\n setp.ne.b32 p, %5, 0;\n mov.b64 x, {%1, %3};\n mov.b64 y, {%2, %3};\n"
        " tcgen05.mma.cta_group::1.kind::f16 [%0], x, y, %4, p;\n}\n" ::"r"(d_tmem),
        "r"(a_lo), "r"(b_lo), "r"(hi), "r"(idesc), "r"((uint32_t)acc));
}

// D += A B with A (fp16 pairs, K along the columns) in tensor memory
__device__ __forceinline__ void mma_ts(uint32_t d_tmem, uint32_t a_tmem, uint32_t b_lo, uint32_t hi, uint32_t idesc, bool acc)
{
    asm volatile(
        "{\n .reg .pred p;\n .reg .b64 y;\n setp.ne.b32 p, %5, 0;\n mov.b64 y, {%2, %3};\n"
        " tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], y, %4, p;\n}\n" ::"r"(d_tmem),
        "r"(a_tmem), "r"(b_lo), "r"(hi), "r"(idesc), "r"((uint32_t)acc));
}

__device__ __forceinline__ void tmem_st16(uint32_t taddr, const uint32_t* r)
{
    asm volatile("tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};" ::"r"(
                     taddr),
                 "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]),
                 "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
                 : "memory");
}
__device__ __forceinline__ void tmem_ld8(uint32_t taddr, uint32_t* r)
{
    asm volatile("tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];\n tcgen05.wait::ld.sync.aligned;"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7])
                 : "r"(taddr)
                 : "memory");
}
__device__ __forceinline__ void tmem_st8(uint32_t taddr, const uint32_t* r)
{
    asm volatile("tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"r"(taddr), "r"(r[0]), "r"(r[1]),
                 "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7])
                 : "memory");
}
__device__ __forceinline__ void tmem_st_wait() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

// mbar_try_wait that may sleep up to 0.1 ms: a dozen warps that poll take the
// issue slots of those that work.
__device__ __forceinline__ bool try_wait_long(uint64_t* bar, uint32_t parity)
{
    uint32_t ok;
    asm volatile(
        "{\n .reg .pred p;\n mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2, %3;\n selp.u32 %0, 1, 0, p;\n}\n"
        : "=r"(ok)
        : "r"(smem_u32(bar)), "r"(parity), "r"(100000u)
        : "memory");
    return ok != 0;
}

__device__ __forceinline__ void prefetch_l1(const void* p) { asm volatile("prefetch.global.L1 [%0];" ::"l"(p)); }
__device__ __forceinline__ void prefetch_l2(const void* p) { asm volatile("prefetch.global.L2 [%0];" ::"l"(p)); }

__device__ __forceinline__ float pow2i(int e)  // 2^e, e in -126 .. 127
{
    return __uint_as_float((uint32_t)(e + 127) << 23);
}

// x 2^e for any e that two such factors reach
__device__ __forceinline__ float scale2(float x, int e) { return x * pow2i(e >> 1) * pow2i(e - (e >> 1)); }

// What the softmax needs to know of a tile; four in turn.  The unpacking warps fill tile n + 4's in when
// tile n + 2's scores (K's side: all but `odd`, and a step tile's `ev`) or products (V's side: those) are
// done.  By then tile n's weights are taken, and for V's side, as a step tile is its run's last, the run's
// results are out, which is when `odd` is read.  What is known of a cached tile's codes comes with their
// ring stage: the warp that finds it runs ahead of the others, by any number of tiles where items without
// cached ones are passed.
struct alignas(16) TileInfo {
    int live, bad;        // keys, and a bit per block of 16 whose page is not in the pool
    int ek, ev;           // powers of two of K and V
    uint32_t odd[4];      // step rows with a NaN or an infinity among their values
};
constexpr int kInfos = 4;

template <int D>
struct TcSmem {
    static constexpr int kAtoms = D / 64;
    static constexpr int kOperand = kAtoms * 128 * 128;       // [atom][128 rows][128 bytes]
    static constexpr int kQ = 0, kK = kOperand, kV = kK + 2 * kOperand;
    static constexpr int kCodes = kV + 2 * kOperand;
    static constexpr int kStage = 8 * kv4_block_bytes(D);
    static constexpr int kVis = kCodes + kRing * kStage;      // [step row][4]: step rows it sees
    static constexpr int kRowF = kVis + 128 * 16;             // [2 runs] per row: what undoes q's power of two
    static constexpr int kRowM = kRowF + 2 * 128 * 4;         // per row: the reference M
    static constexpr int kRowL = kRowM + 128 * 4;             // [2 groups] per row: sums
    static constexpr int kInfo = kRowL + 2 * 128 * 4;         // TileInfo[kInfos]
    static constexpr int kBar = kInfo + kInfos * (int)sizeof(TileInfo);
    static constexpr int kMisc = kBar + 32 * 8;               // ring info, reduction words, start, scan scratch
    static constexpr int kBytes = kMisc + 512 + 1024;         // 1024: to align the base
    static_assert(kInfo % 16 == 0 && kMisc % 16 == 0, "alignment");
};

enum {  // barriers
    kFull = 0, kEmpty = 3, kInfoReady = 6, kKReady = 9, kVReady = 11, kSDone = 13, kODone = 15, kPReady = 17, kQReady = 19,
    kOFree = 20, kEnd = 21, kStepReady = 22  // (22, 23: a step tile's power of two of V, by the tile's parity)
};
constexpr uint32_t kColO = 256, kColP = 384;  // tensor memory: S [2][128], O [D], P [2][64]

// Byte offset of 16-byte piece i of a row in an operand, with the 128-byte swizzle.
__device__ __forceinline__ int piece_at(int i, int row)
{
    return (i >> 3) * (128 * 128) + row * 128 + (((i & 7) ^ (row & 7)) << 4);
}

// the larger exponent of a bf16 pair, in place (bits 7 - 14)
__device__ __forceinline__ uint32_t high_exp(uint32_t w) { return max(w & 0x7f80u, (w >> 16) & 0x7f80u); }

// a bf16 pair times f, in fp16
__device__ __forceinline__ uint32_t to_f16(uint32_t w, float f)
{
    return pack_f16(__uint_as_float(w << 16) * f, __uint_as_float(w & 0xffff0000u) * f);
}

// 8 codes of a word as fp16 (c - z) s 2^-E: pairs 0, 2 by lo, 1, 3 by hi.
__device__ __forceinline__ uint4 unpack8(uint32_t w, __half2 lo, __half2 hi, __half2 off)
{
    auto one = [&](uint32_t bits, __half2 f) {
        const __half2 v = __hfma2(*reinterpret_cast<const __half2*>(&bits), f, off);
        return *reinterpret_cast<const uint32_t*>(&v);
    };
    const uint32_t h = w >> 8;
    return make_uint4(one(w & kLo, lo), one(w & kHi, hi), one(h & kLo, lo), one(h & kHi, hi));
}

// Adds what is not finite among the values of the step rows (bits of odd and see
// both set) to 32 channels from col.
__device__ __noinline__ void add_odd_to(const Kv4Attn& a, const uint32_t* odd, const uint32_t* see, int b, int col, float* o)
{
    for (int key = 0; key < a.T; key++) {
        if (!(((odd[key >> 5] & see[key >> 5]) >> (key & 31)) & 1)) continue;
        const __nv_bfloat16* v = a.vs + (size_t)(b * (long long)a.T + key) * a.kv_ld + col;
        for (int i = 0; i < 32; i++) {
            const float x = __bfloat162float(v[i]);
            if (!(fabsf(x) < INFINITY)) o[i] += x;
        }
    }
}

__device__ __forceinline__ void add_odd(const Kv4Attn& a, const uint32_t* odd, const uint32_t* see, int b, int col, float (&o)[32])
{
    float t[32];  // (in memory for the call; o stays in registers)
#pragma unroll
    for (int i = 0; i < 32; i++) t[i] = o[i];
    add_odd_to(a, odd, see, b, col, t);
#pragma unroll
    for (int i = 0; i < 32; i++) o[i] = t[i];
}

__device__ __forceinline__ float ld_peer(uint32_t addr)
{
    float v;
    asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(v) : "r"(addr) : "memory");
    return v;
}
__device__ __forceinline__ void st_peer4(uint32_t addr, float x, float y, float z, float w)
{
    asm volatile("st.shared::cluster.v4.f32 [%0], {%1, %2, %3, %4};" ::"r"(addr), "f"(x), "f"(y), "f"(z), "f"(w) : "memory");
}

template <int D>
__device__ __forceinline__ MergeRec* merge_rec(const Kv4Attn& a)
{
    return (MergeRec*)(a.part + (size_t)a.nteams * 2 * part_floats(kRowsTc, D)) + blockIdx.x;
}

// CL: one item per cluster; its CTAs take equal runs of the item's tiles.
template <int D, bool CL>
__global__ void __launch_bounds__(kTcThreads, 1) k_kv4_tc(Kv4Attn a)
{
    using L = TcSmem<D>;
    extern __shared__ uint8_t smem_raw[];
    uint8_t* sm = smem_raw + (-smem_u32(smem_raw) & 1023);  // (by an offset: a pointer made from an integer is generic)
    uint64_t* bar = (uint64_t*)(sm + L::kBar);
    TileInfo* info = (TileInfo*)(sm + L::kInfo);
    uint32_t* vis = (uint32_t*)(sm + L::kVis);
    float *rowf = (float*)(sm + L::kRowF), *row_m = (float*)(sm + L::kRowM), *row_l = (float*)(sm + L::kRowL);
    int* ring_info = (int*)(sm + L::kMisc);                // [3]: live | bad << 16
    uint32_t* red_e = (uint32_t*)(sm + L::kMisc + 16);     // [2][4]: largest exponents of the unpacking warps
    uint32_t* tmem_slot = (uint32_t*)(sm + L::kMisc + 80);
    volatile int* abort_flag = (volatile int*)(sm + L::kMisc + 84);
    Start* start = (Start*)(sm + L::kMisc + 96);
    long long* scratch = (long long*)(sm + L::kMisc + 160);  // one per warp
    int4* stage_info = (int4*)(sm + L::kMisc + 320);         // [3]: live, bad, ek, ev of the stage's tile
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int group = a.H / a.Hkv;

    if (warp == 16) tmem_alloc(tmem_slot, 512);
    if (threadIdx.x == 0) {
        for (int i = 0; i < 3; i++) mbar_init(bar + kFull + i, 1), mbar_init(bar + kEmpty + i, 8), mbar_init(bar + kInfoReady + i, 1);
        for (int i = 0; i < 2; i++) {
            mbar_init(bar + kKReady + i, 4);
            mbar_init(bar + kVReady + i, 4);
            mbar_init(bar + kSDone + i, 1);
            mbar_init(bar + kODone + i, 1);
            mbar_init(bar + kPReady + i, 4);
            mbar_init(bar + kStepReady + i, 1);
        }
        mbar_init(bar + kQReady, 8);
        mbar_init(bar + kOFree, 8);
        mbar_init(bar + kEnd, 1);
        *abort_flag = 0;
        mbar_fence_init();
    }
    for (int i = threadIdx.x - 32; i >= 0 && i < a.T; i += kTcThreads) {
        // the step rows that step row i sees (the mask), as bits
        uint32_t m[4];
        const int nl = a.W * a.n1;
        int lo, hi;  // besides row 0: lo .. hi, and column c of the levels up to lv
        int lv = 0, c = 0;
        if (i <= nl) lv = i ? (i - 1) / a.W : 0, c = i ? (i - 1) % a.W : 0, lo = 1, hi = i ? 1 + c : 0;
        else lo = i - (i - 1 - nl) % a.n1, hi = i;
#pragma unroll
        for (int w = 0; w < 4; w++) {
            const int x = max(lo - 32 * w, 0), y = min(hi - 32 * w, 31);
            m[w] = x <= y ? (~0u << x) & (~0u >> (31 - y)) : 0u;
        }
        m[0] |= 1u;
        for (int v = 1; v <= lv; v++) {
            const int j = 1 + v * a.W + c;
#pragma unroll
            for (int w = 0; w < 4; w++) m[w] |= j >> 5 == w ? 1u << (j & 31) : 0u;
        }
        *(uint4*)(vis + 4 * i) = make_uint4(m[0], m[1], m[2], m[3]);
    }
    pdl_wait();
    pdl_trigger();
    if (blockIdx.x == 0) raise_long(a);
    tc_fence_before();
    Run first;
    first.left = 0;
    bool work;
    int stride = 1;  // between the CTA's tiles of an item
    if (CL) {
        // tiles rank, rank + cs, ...: the first one does not depend on the length
        const int cs = (int)cluster_size(), rank = (int)cluster_rank();
        const int x = blockIdx.x / cs, items = a.Hkv * a.mtiles;
        first.b = x / items;
        first.item = x - first.b * items;
        if (warp >= 8 && warp < 16) {
            // what the unpacking warps read first and last
            const int head = first.item / a.mtiles, kv = warp >= 12, i = (threadIdx.x - 256) & 127;
            const int gr = (first.item - head * a.mtiles) * kRowsTc + ((threadIdx.x - 256) >> 1);
            if (gr < a.rows)
                prefetch_l1(a.q + (size_t)(first.b * (long long)a.T + gr / group) * a.q_ld + (size_t)(head * group + gr % group) * D +
                            (D == 128 ? 64 * (threadIdx.x & 1) : 0));
            if (i < a.T) {
                const __nv_bfloat16* src = (kv ? a.vs : a.ks) + (size_t)(first.b * (long long)a.T + i) * a.kv_ld + (size_t)head * D;
                prefetch_l2(src);
                if (D == 128) prefetch_l2(src + 64);
            }
        } else if (warp == 17 && (rank * 8 + lane) >> a.blk_log2 < a.max_pages) {
            prefetch_l1(a.table + (size_t)first.b * a.max_pages + ((rank * 8 + lane) >> a.blk_log2));
        }
        first.len = seq_len(a, first.b);
        const int nt = first.len < 0 ? 0 : (first.len + kTile - 1) / kTile + 1;
        first.nu = first.u1 = first.t1 = nt, first.u0 = 0, first.t0 = rank;
        stride = cs;
        __syncthreads();
        work = first.t1 > first.t0;
    } else {
        find_starts(a, blockIdx.x, 1, start, scratch);
        const Start st = *start;
        work = st.count > 0;
        if (work) first.begin(a, st);
        if (a.part && threadIdx.x == 0) merge_rec<D>(a)->rest = 0;
    }
    tc_fence_after();
    const uint32_t tmem = *tmem_slot;

    // A wait that gives up ends every later one at once, but no role leaves its
    // loops: the named barriers keep their counts.
    bool ok = true;
    auto wait = [&](int b, int parity) {
        if (!ok || try_wait_long(bar + b, parity)) return;
        const unsigned long long t0 = globaltimer();
        while (!try_wait_long(bar + b, parity)) {
            if (*abort_flag || globaltimer() - t0 > kWaitNs) {
                ok = false;
                *abort_flag = 1;
                kv4_raise(a.status, LA_ERR_TIMEOUT);
                return;
            }
        }
    };
    int n = 0;     // tiles so far: n & 1 is the buffer, (n >> 1) & 1 its phase
    int segs = 0;  // runs with tiles so far
    float out_m = kNoRef, out_l = 0.f;  // CL: this thread's row
    Run run = first;
    if (work && warp < 8) {
        // ------------------------------------------------------------ softmax
        const int q = warp & 3, grp = warp >> 2, row = q * 32 + lane;
        const uint32_t trow = tmem + ((uint32_t)(q * 32) << 16);
        int steps = 0;  // this group's step tiles so far
        do {
            const int head = run.item / a.mtiles, mt = run.item - head * a.mtiles;
            const int ntc = (run.len + kTile - 1) / kTile, gr = mt * kRowsTc + row;
            const bool any = mt * kRowsTc + q * 32 < a.rows;  // some row of this warp is there
            const int n0 = n;
            float m = kNoRef, l = 0.f;
            for (int tile = run.t0; tile < run.t1; tile += stride, n++) {
                if ((n & 1) != grp) continue;
                const bool step = tile >= ntc;
                const int b = grp, ph = (n >> 1) & 1;
                wait(kSDone + b, ph);  // (so K's part of the tile's entry is there; V's of a step tile may not be)
                // A barrier a group: V's part of tile n + 2 waits for tile n's products, so for this wait
                if (step) wait(kStepReady + grp, steps & 1), steps++;
                tc_fence_after();
                if (any) {
                    const TileInfo* ti = info + (n & (kInfos - 1));
                    const int live = ti->live, bad = ti->bad, iev = ti->ev;
                    const float f = fmaxf(scale2(rowf[(segs & 1) * 128 + row], ti->ek), 1e-37f), ev = (float)iev;
                    const bool part = step || live < kTile || bad;
                    const uint32_t* see = vis + 4 * min(gr / group, a.T - 1);
                    const int n32 = (live + 31) >> 5;  // groups of 32 scores that hold any (P V stops there, too)
                    auto counts = [&](int c) -> uint32_t {  // which of the scores 32 c .. count
                        if (step) return see[c];
                        const int left = live - c * 32, off = bad >> (2 * c);
                        const uint32_t s = left >= 32 ? ~0u : (1u << left) - 1u;
                        return s & ~((off & 1 ? 0xffffu : 0u) | (off & 2 ? 0xffff0000u : 0u));
                    };
                    const uint32_t ts = trow + b * 128;
                    // Weigh with the reference as it is, P going to its own columns; only where
                    // a row outgrows it (a sum above 2^15, so that no P overflows) find the
                    // row's largest and weigh again.  The first tile starts from the largest of
                    // its first 32 scores.  The other group may have moved the reference in the
                    // tile before: its decision is waited for with the results in hand.
                    const bool lead = n == n0;
                    float sum = 0.f;
                    int look = 0;  // scores / 32 to look for a row's largest in before weighing
                    if (lead) {
                        look = 1;
                    } else if (n == n0 + 1) {
                        wait(kPReady + (b ^ 1), ((n - 1) >> 1) & 1);
                        m = row_m[row];
                    }
#pragma unroll 1
                    while (true) {
                        if (look) {
                            float t0 = -INFINITY, t1 = -INFINITY;
#pragma unroll 1
                            for (int c = 0; c < min(look, n32); c++) {
                                float x[32];
                                tmem_ld32(ts + c * 32, x);
                                if (part) {
                                    const uint32_t s = counts(c);
#pragma unroll
                                    for (int j = 0; j < 32; j++)
                                        if (!((s >> j) & 1)) x[j] = -INFINITY;
                                }
#pragma unroll
                                for (int j = 0; j < 32; j += 4) {
                                    t0 = fmaxf(t0, fmaxf(x[j], x[j + 1]));
                                    t1 = fmaxf(t1, fmaxf(x[j + 2], x[j + 3]));
                                }
                            }
                            const float y = fmaxf(t0, t1) * f + ev;
                            const bool up = y > m + 8.f;
                            const float c = up ? ex2(m - y) : 1.f;
                            if (up) m = y;
                            l *= c;
                            row_m[row] = m;
                            if (!lead && __any_sync(0xffffffffu, up)) {
                                wait(kODone + (b ^ 1), ((n - 1) >> 1) & 1);
                                tc_fence_after();
#pragma unroll 1
                                for (int j = 0; j < D; j += 8) {
                                    uint32_t o[8];
                                    tmem_ld8(trow + kColO + j, o);
#pragma unroll
                                    for (int i = 0; i < 8; i++) o[i] = __float_as_uint(__uint_as_float(o[i]) * c);
                                    tmem_st8(trow + kColO + j, o);
                                }
                            }
                        }
                        const float c0 = ev - m;
                        uint64_t s2 = 0;  // two sums
                        const uint64_t f2 = pair(f, f), c2 = pair(c0, c0);
                        auto weigh = [&](int c, float (&x)[32]) {
                            uint32_t p[16];
#pragma unroll
                            for (int j = 0; j < 32; j += 2) {
                                float e0, e1;
                                unpair(fma2(pair(x[j], x[j + 1]), f2, c2), e0, e1);
                                e0 = ex2(e0), e1 = ex2(e1);
                                s2 = add2(s2, pair(e0, e1));
                                p[j / 2] = pack_f16(e0, e1);
                            }
                            tmem_st16(trow + kColP + b * 64 + c * 16, p);
                        };
#pragma unroll 1
                        for (int c = 0; c < n32; c++) {
                            float x[32];
                            tmem_ld32(ts + c * 32, x);
                            if (part) {
                                const uint32_t s = counts(c);
#pragma unroll
                                for (int j = 0; j < 32; j++)
                                    if (!((s >> j) & 1)) x[j] = -INFINITY;
                            }
                            weigh(c, x);
                        }
                        float s0, s1;
                        unpair(s2, s0, s1);
                        sum = s0 + s1;
                        if (look == 4) break;
                        bool again = sum > 32768.f || m == kNoRef;
                        if (!look && n > n0 + 1) {
                            wait(kPReady + (b ^ 1), ((n - 1) >> 1) & 1);
                            const float mm = row_m[row];
                            if (mm != m) l *= ex2(m - mm), m = mm, again = true;
                        }
                        if (!__any_sync(0xffffffffu, again)) break;
                        look = 4;
                    }
                    l += scale2(sum, -iev);
                    tmem_st_wait();
                } else if (n > n0) {
                    wait(kPReady + (b ^ 1), ((n - 1) >> 1) & 1);  // in tile order, like the others
                }
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(bar + kPReady + b);
            }
            // ---- the run's result: group grp takes half of the channels
            const bool tiles = run.t1 > run.t0, whole = run.u0 == 0 && run.u1 == run.nu;
            const int last = n - 1;
            if (tiles) {
                wait(kODone + (last & 1), (last >> 1) & 1);
                tc_fence_after();
            }
            if (any) {
                const float mm = tiles ? row_m[row] : kNoRef;
                row_l[grp * 128 + row] = l * (m == mm ? 1.f : ex2(m - mm));
                m = mm;
                named_sync(1 + q, 64);
                const float sum = row_l[row] + row_l[128 + row];
                named_sync(1 + q, 64);
                if (CL) {
                    out_m = m, out_l = sum;
                } else {
                    float* part = a.part + ((size_t)blockIdx.x * 2 + (run.u0 == 0 ? 1 : 0)) * part_floats(kRowsTc, D);
                    const float inv = 1.f / sum;
                    __nv_bfloat16* orow = a.out + ((size_t)(run.b * (long long)a.T + gr / group) * a.H + head * group + gr % group) * D;
                    // the step tile, if it is there, is the last one; its products are done, so its entry is complete
                    const uint32_t* odd = info[last & (kInfos - 1)].odd;
                    const bool fix = run.t1 > ntc && (odd[0] | odd[1] | odd[2] | odd[3]) != 0;
#pragma unroll 1
                    for (int j = 0; j < D / 2; j += 32) {
                        float o[32];
                        const int c = grp * (D / 2) + j;
                        __syncwarp();
                        if (tiles) {
                            tmem_ld32(trow + kColO + c, o);
                        } else {
#pragma unroll
                            for (int i = 0; i < 32; i++) o[i] = 0.f;
                        }
                        if (fix && gr < a.rows) add_odd(a, odd, vis + 4 * (gr / group), run.b, head * D + c, o);
                        if (gr < a.rows && whole) {
#pragma unroll
                            for (int i = 0; i < 32; i += 8)
                                *(uint4*)(orow + c + i) =
                                    make_uint4(pack_bf16(o[i] * inv, o[i + 1] * inv), pack_bf16(o[i + 2] * inv, o[i + 3] * inv),
                                               pack_bf16(o[i + 4] * inv, o[i + 5] * inv), pack_bf16(o[i + 6] * inv, o[i + 7] * inv));
                        } else if (gr < a.rows) {
#pragma unroll
                            for (int i = 0; i < 32; i++) part[(size_t)(c + i) * kRowsTc + row] = o[i];  // a line per warp
                        }
                    }
                    if (!whole && grp == 0 && gr < a.rows)
                        part[(size_t)kRowsTc * D + row] = m, part[(size_t)kRowsTc * (D + 1) + row] = sum;
                }
            }
            if (!CL && run.u0 == 0 && !whole && a.part && threadIdx.x == 0)
                *merge_rec<D>(a) = MergeRec{run.b, run.item, run.nu - run.u1, 0, start->sh};
            if (tiles) {
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(bar + kOFree);
                segs++;
            }
        } while (!CL && run.next(a));
    } else if (work && warp < 16) {
        // ------------------------------------------------------------- unpack
        const int kv = warp >= 12, tid = threadIdx.x - 256 - kv * 128, h = tid & 1, uw = warp & 3;
        int fills = 0;  // ring stages taken
        do {
            const int head = run.item / a.mtiles, mt = run.item - head * a.mtiles;
            const int ntc = (run.len + kTile - 1) / kTile;
            if (run.t1 <= run.t0) continue;
            // the step's rows are needed last: into L2 by then
            if (!CL && run.t1 > ntc && tid < a.T) {
                const __nv_bfloat16* src = (kv ? a.vs : a.ks) + (size_t)(run.b * (long long)a.T + tid) * a.kv_ld + (size_t)head * D;
                prefetch_l2(src);
                if (D == 128) prefetch_l2(src + 64);
            }
            // ---- the rows' queries, each by a power of two
            if (n > 0) wait(kSDone + ((n - 1) & 1), ((n - 1) >> 1) & 1);  // the last tile's S has read the old ones
            {
                // Neighbouring threads take neighbouring 16-byte pieces of a row (spread over
                // rows, each load would touch 32 lines); short loops, because code that runs
                // once costs 8 cycles an instruction to fetch.
                constexpr int kPieces = D / 8, kPass = 256 / kPieces;
                const int pc = (threadIdx.x - 256) % kPieces, r0 = (threadIdx.x - 256) / kPieces;
                uint8_t* q0 = sm + L::kQ;
                // step row and head of the group, advanced by kPass rows at a time
                int si = (mt * kRowsTc + r0) / group, sj = mt * kRowsTc + r0 - si * group;
                const int di = kPass / group, dj = kPass - di * group;
#pragma unroll 1
                for (int i0 = 0; i0 < 128 / kPass; i0 += 4) {
                    // (loads first: none moves above a store to shared memory by itself)
                    uint4 u[4];
#pragma unroll
                    for (int i = 0; i < 4; i++) {
                        const int gr = mt * kRowsTc + r0 + (i0 + i) * kPass;
                        u[i] = make_uint4(0, 0, 0, 0);
                        if (gr < a.rows)
                            u[i] = *(const uint4*)(a.q + ((size_t)run.b * a.T + si) * a.q_ld + (size_t)(head * group + sj) * D + 8 * pc);
                        si += di, sj += dj;
                        if (sj >= group) sj -= group, si++;
                    }
#pragma unroll
                    for (int i = 0; i < 4; i++) {
                        const int row = r0 + (i0 + i) * kPass;
                        uint32_t top = max(max(high_exp(u[i].x), high_exp(u[i].y)), max(high_exp(u[i].z), high_exp(u[i].w)));
#pragma unroll
                        for (int o = 1; o < kPieces; o <<= 1) top = max(top, __shfl_xor_sync(0xffffffffu, top, o));
                        const int e = min(max((int)(top >> 7), 16), 236);
                        const float down = pow2i(11 + 127 - e);  // the largest comes to [2^11, 2^12)
                        *(uint4*)(q0 + piece_at(pc, row)) = make_uint4(to_f16(u[i].x, down), to_f16(u[i].y, down), to_f16(u[i].z, down), to_f16(u[i].w, down));
                        if (pc == 0) rowf[(segs & 1) * 128 + row] = pow2i(e - 127 - 11) * a.sl2;
                    }
                }
                fence_proxy_async();
                __syncwarp();
                if (lane == 0) mbar_arrive(bar + kQReady);
                segs++;
            }
            for (int tile = run.t0; tile < run.t1; tile += stride, n++) {
                const int b = n & 1, ph = (n >> 1) & 1;
                uint8_t* dst = sm + (kv ? L::kV : L::kK) + b * L::kOperand;
                TileInfo* ti = info + (n & (kInfos - 1));
                if (tile < ntc) {
                    const int s = fills % kRing, sp = (fills / kRing) & 1;
                    wait(kInfoReady + s, sp);
                    wait(kFull + s, sp);
                    const uint8_t* stage = sm + L::kCodes + s * L::kStage;
                    const int4 known = stage_info[s];
                    const int live = known.x, bad = known.y, E = kv ? known.w : known.z;
                    if (n >= 2) wait((kv ? kODone : kSDone) + b, ph ^ 1);  // tile n - 2's product has read the buffer
                    if (tid == 0 && !kv) *(int4*)ti = known;
                    // key rows tid / 2 and 64 + tid / 2, half of each 64-channel panel
#pragma unroll 1
                    for (int r2 = 0; r2 < 2; r2++) {
                        const int row = (tid >> 1) + 64 * r2;
                        if ((row & ~15) >= live) break;
                        const uint8_t* blk = stage + (row >> 4) * kv4_block_bytes(D);
                        const uint32_t par = ((const uint32_t*)(blk + 16 * D))[16 * kv + (row & 15)];
                        const bool here = row < live && !((bad >> (row >> 4)) & 1);
                        const float sc = here ? scale2(__uint_as_float(par & 0xffff0000u), -E) : 0.f;
                        const __half2 lo = __float2half2_rn(sc * 0x1p24f), hi = __float2half2_rn(sc * 0x1p20f),
                                      off = __float2half2_rn(-(float)(par & 15u) * sc);
                        uint4 w[L::kAtoms];
#pragma unroll
                        for (int p = 0; p < L::kAtoms; p++)
                            w[p] = *(const uint4*)(blk + kv * 8 * D + p * 512 + (row & 15) * 32 + h * 16);
#pragma unroll
                        for (int p = 0; p < L::kAtoms; p++) {
                            const uint32_t* u = (const uint32_t*)&w[p];
#pragma unroll
                            for (int i = 0; i < 4; i++)
                                *(uint4*)(dst + p * (128 * 128) + row * 128 + (((4 * h + i) ^ (row & 7)) << 4)) = unpack8(u[i], lo, hi, off);
                        }
                    }
                    fence_proxy_async();
                    __syncwarp();
                    if (lane == 0) {
                        mbar_arrive(bar + (kv ? kVReady : kKReady) + b);
                        mbar_arrive(bar + kEmpty + s);
                    }
                    fills++;
                } else {
                    // the step's own rows: bf16 to fp16 by the tile's largest finite exponent
                    constexpr int kPieces = D / 8, kPass = 128 / kPieces;
                    const int pc = tid % kPieces, r0 = tid / kPieces;  // as the queries
                    const __nv_bfloat16* src = (kv ? a.vs : a.ks) + ((size_t)run.b * a.T + r0) * a.kv_ld + (size_t)head * D + 8 * pc;
                    uint32_t odd_rows = 0;  // bit i: of row r0 + i kPass
                    if (n >= 2) wait((kv ? kODone : kSDone) + b, ph ^ 1);  // tile n - 2's product has read the buffer
                    auto place = [&](int i) { return (uint4*)(dst + piece_at(pc, r0 + i * kPass)); };
                    // to their places as they are; the largest finite exponent, and whether there are others
                    uint32_t e = 0, all = 0;
#pragma unroll 1
                    for (int i0 = 0; i0 < 128 / kPass; i0 += 8) {
                        uint4 u[8];
#pragma unroll
                        for (int i = 0; i < 8; i++)
                            u[i] = r0 + (i0 + i) * kPass < a.T ? *(const uint4*)(src + (size_t)((i0 + i) * kPass) * a.kv_ld) : make_uint4(0, 0, 0, 0);
#pragma unroll
                        for (int i = 0; i < 8; i++) {
                            const uint32_t x = max(max(high_exp(u[i].x), high_exp(u[i].y)), max(high_exp(u[i].z), high_exp(u[i].w)));
                            all = max(all, x);
                            if (x < 0x7f80u) e = max(e, x);
                            *place(i0 + i) = u[i];
                        }
                    }
                    e >>= 7;
                    if (__any_sync(0xffffffffu, all >= 0x7f80u)) {
                        // (rare) per element: largest finite exponent; of V's, which rows have others
#pragma unroll 1
                        for (int i = 0; i < 128 / kPass; i++) {
                            uint4* at = place(i);
                            uint32_t w[4] = {at->x, at->y, at->z, at->w};
                            bool found = false;
#pragma unroll
                            for (int k = 0; k < 4; k++) {
                                const uint32_t x0 = (w[k] >> 7) & 255u, x1 = (w[k] >> 23) & 255u;
                                e = max(e, max(x0 < 255 ? x0 : 0u, x1 < 255 ? x1 : 0u));
                                found |= x0 == 255 || x1 == 255;
                                // zero times these is NaN: the product of V runs without them (TileInfo::odd)
                                if (kv) w[k] &= (x0 == 255 ? 0xffff0000u : ~0u) & (x1 == 255 ? 0xffffu : ~0u);
                            }
                            *at = make_uint4(w[0], w[1], w[2], w[3]);
                            if (found) odd_rows |= 1u << i;
                        }
                    }
                    e = __reduce_max_sync(0xffffffffu, e);
                    if (lane == 0) red_e[kv * 4 + uw] = e;
                    if (kv && tid < 4) ti->odd[tid] = 0;
                    named_sync(5 + kv, 128);
#pragma unroll
                    for (int i = 0; i < 4; i++) e = max(e, red_e[kv * 4 + i]);
                    named_sync(5 + kv, 128);  // red_e may be written again
                    // The largest comes to [2^-4, 2^-3), as the cached tiles' do: P carries the tiles'
                    // powers of two of V, and a step tile far from the others would push its P (or
                    // theirs) to where fp16 has fewer bits.
                    const int E = max((int)e, kv ? 82 : 28) - 123;
                    if (tid == 0) {
                        // K's part is waited for with the scores, which need all of K
                        if (kv) ti->ev = E, mbar_arrive(bar + kStepReady + b);
                        else ti->ek = E, ti->live = a.T, ti->bad = 0;
                    }
                    const float f = scale2(1.f, -E);
#pragma unroll 1
                    for (int i0 = 0; i0 < 128 / kPass; i0 += 4) {
                        uint4 u[4];
#pragma unroll
                        for (int i = 0; i < 4; i++) u[i] = *place(i0 + i);
#pragma unroll
                        for (int i = 0; i < 4; i++)
                            *place(i0 + i) = make_uint4(to_f16(u[i].x, f), to_f16(u[i].y, f), to_f16(u[i].z, f), to_f16(u[i].w, f));
                    }
                    if (kv)
                        for (uint32_t left = odd_rows; left; left &= left - 1) {
                            const int row = r0 + (__ffs(left) - 1) * kPass;
                            atomicOr(&ti->odd[row >> 5], 1u << (row & 31));
                        }
                    fence_proxy_async();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(bar + (kv ? kVReady : kKReady) + b);
                }
            }
        } while (!CL && run.next(a));
    } else if (work && warp == 16) {
        // ---------------------------------------------------------------- MMA
        constexpr uint32_t id_s = idesc_f16(128, kTile, false), id_o = idesc_f16(128, D, true);
        const uint32_t base = smem_u32(sm);
        const uint64_t dk = desc_sw128_kmajor(base), dv = desc_sw128_mnmajor(base, 128 * 128);
        const uint32_t k_lo = (uint32_t)dk, k_hi = (uint32_t)(dk >> 32), v_lo = (uint32_t)dv, v_hi = (uint32_t)(dv >> 32);
        const bool chosen = elect_one();
        auto scores = [&](int b, int ph, bool lead) {
            wait(kKReady + b, ph);
            if (lead) wait(kQReady, segs & 1);
            tc_fence_after();
            if (chosen && ok) {
#pragma unroll
                for (int k = 0; k < D / 16; k++) {
                    const uint32_t at = ((k >> 2) * (128 * 128) + (k & 3) * 32) >> 4;
                    mma_ss(tmem + b * 128, k_lo + (L::kQ >> 4) + at, k_lo + ((L::kK + b * L::kOperand) >> 4) + at, k_hi, id_s, k > 0);
                }
                mma_commit(bar + kSDone + b);
            }
            __syncwarp();
        };
        auto outputs = [&](int b, int ph, bool lead) {
            wait(kPReady + b, ph);
            wait(kVReady + b, ph);
            if (lead && segs > 0) wait(kOFree, (segs - 1) & 1);
            const int live = info[n & (kInfos - 1)].live;  // only these keys' products
            tc_fence_after();
            if (chosen && ok) {
                auto step16 = [&](int k) {
                    mma_ts(tmem + kColO, tmem + kColP + b * 64 + k * 8, v_lo + ((L::kV + b * L::kOperand + k * 16 * 128) >> 4), v_hi,
                           id_o, !lead || k > 0);
                };
                if (live > kTile - 16) {
#pragma unroll
                    for (int k = 0; k < kTile / 16; k++) step16(k);
                } else {
#pragma unroll 1
                    for (int k = 0; k * 16 < live; k++) step16(k);
                }
                mma_commit(bar + kODone + b);
            }
            __syncwarp();
        };
        do {
            const int tiles = (run.t1 - run.t0 + stride - 1) / stride;
            if (tiles <= 0) continue;
            scores(n & 1, (n >> 1) & 1, true);
            for (int i = 0; i < tiles; i++, n++) {
                // the next tile's scores go first: they run while this one's softmax does
                if (i + 1 < tiles) scores((n + 1) & 1, ((n + 1) >> 1) & 1, false);
                outputs(n & 1, (n >> 1) & 1, i == 0);
            }
            segs++;
        } while (!CL && run.next(a));
        if (!ok && chosen) {
            // let the products that were issued finish before the memory goes
            mma_commit(bar + kEnd);
            mbar_drain(bar + kEnd, 0);
        }
        __syncwarp();
    } else if (work && warp == 17) {
        // -------------------------------------------------------------- copies
        const uint64_t pol = policy_evict_first();
        int fills = 0;
        do {
            const int head = run.item / a.mtiles, ntc = (run.len + kTile - 1) / kTile;
            // the pages of four tiles' blocks at a time, and of the next four ahead
            const int* pages = a.table + (size_t)run.b * a.max_pages;
            auto look_up = [&](int tile) {
                const int blk = (tile + (lane >> 3) * stride) * 8 + (lane & 7);
                return blk * 16 < run.len ? __ldg(pages + (blk >> a.blk_log2)) : 0;
            };
            int pg = look_up(run.t0), pg_next = look_up(run.t0 + 4 * stride), turn = -1;
            for (int tile = run.t0; tile < min(run.t1, ntc); tile += stride) {
                const int s = fills % kRing, blk = tile * 8 + lane, live = min(run.len - tile * kTile, kTile);
                const bool mine = lane < 8 && lane * 16 < live;
                turn = (turn + 1) & 3;
                if (turn == 0 && tile > run.t0) pg = pg_next, pg_next = look_up(tile + 4 * stride);
                const int page_of = __shfl_sync(0xffffffffu, pg, (8 * turn + lane) & 31), page = mine ? page_of : 0;
                const bool bad = (unsigned)page >= (unsigned)a.n_pages;
                const uint32_t bads = __ballot_sync(0xffffffffu, bad), who = __ballot_sync(0xffffffffu, mine);
                if (fills >= kRing) wait(kEmpty + s, (fills / kRing - 1) & 1);
                if (!__all_sync(0xffffffffu, ok)) continue;
                if (lane == 0) {
                    if (bads) kv4_raise(a.status, LA_ERR_ARG);
                    ring_info[s] = live | (int)bads << 16;
                    mbar_expect_tx(bar + kFull + s, __popc(who) * kv4_block_bytes(D));
                }
                __syncwarp();
                if (mine)
                    bulk_load(sm + L::kCodes + s * L::kStage + lane * kv4_block_bytes(D),
                              a.pages + kv4_block_at(bad ? 0 : page, head, blk & ((1 << a.blk_log2) - 1), a.Hkv, a.blk_log2, D),
                              kv4_block_bytes(D), bar + kFull + s, pol);
                __syncwarp();
                fills++;
            }
        } while (!CL && run.next(a));
        // no copy may still be on its way when the CTA ends
        for (int i = 1; i <= kRing && i <= fills; i++) mbar_drain(bar + kFull + (fills - i) % kRing, ((fills - i) / kRing) & 1);
    } else if (work) {
        // ------------------------------------------------- the powers of two
        // (and, with time to spare, the next item's queries and step rows into L2)
        int fills = 0;
        do {
            const int ntc = (run.len + kTile - 1) / kTile;
            if (!CL && run.left > 0 && run.item + 1 < a.Hkv * a.mtiles) {
                const int item = run.item + 1, head = item / a.mtiles, r0 = (item - head * a.mtiles) * kRowsTc;
                for (int r = lane; r < min(kRowsTc, a.rows - r0); r += 32) {
                    const int i = (r0 + r) / group, j = r0 + r - i * group;
                    const __nv_bfloat16* src = a.q + ((size_t)run.b * a.T + i) * a.q_ld + (size_t)(head * group + j) * D;
                    prefetch_l2(src);
                    if (D == 128) prefetch_l2(src + 64);
                }
                if (r0 == 0)
                    for (int r = lane; r < a.T; r += 32) {
                        const size_t at = ((size_t)run.b * a.T + r) * a.kv_ld + (size_t)head * D;
                        prefetch_l2(a.ks + at), prefetch_l2(a.vs + at);
                        if (D == 128) prefetch_l2(a.ks + at + 64), prefetch_l2(a.vs + at + 64);
                    }
            }
            for (int tile = run.t0; tile < min(run.t1, ntc); tile += stride) {
                const int s = fills % kRing;
                wait(kFull + s, (fills / kRing) & 1);
                const uint8_t* stage = sm + L::kCodes + s * L::kStage;
                const int ri = ring_info[s], live = ri & 0xffff, bad = ri >> 16;
                uint32_t ek = 0, ev = 0;  // the largest scales' exponents (of keys that count)
#pragma unroll
                for (int i = 0; i < 4; i++) {
                    const int key = lane + 32 * i;
                    const uint32_t* par = (const uint32_t*)(stage + (key >> 4) * kv4_block_bytes(D) + 16 * D) + (key & 15);
                    const uint32_t k0 = par[0] >> 23, v0 = par[16] >> 23;
                    const bool here = key < live && !((bad >> (key >> 4)) & 1);
                    ek = max(ek, here && k0 < 255 ? k0 : 0u);
                    ev = max(ev, here && v0 < 255 ? v0 : 0u);
                }
                ek = __reduce_max_sync(0xffffffffu, ek), ev = __reduce_max_sync(0xffffffffu, ev);
                if (lane == 0) {
                    // s 2^-E < 2^-8.  V's not below 2^-41, where the values under 2^-50 lose bits: the weights of
                    // a tile without values must still be fp32 numbers beside one of values near 2^50.
                    stage_info[s] = make_int4(live, bad, max((int)ek, 20) - 118, max((int)ev, 77) - 118);
                    mbar_arrive(bar + kInfoReady + s);
                }
                __syncwarp();
                fills++;
            }
        } while (!CL && run.next(a));
    }
    __syncwarp();
    if (CL) {
        // ---- the cluster's parts meet: every CTA sums its share of the channels
        const int cs = (int)cluster_size(), rank = (int)cluster_rank(), row = threadIdx.x & 127, grp = threadIdx.x >> 7;
        const int head = first.item / a.mtiles, mt = first.item - head * a.mtiles, gr = mt * kRowsTc + row;
        const int ntc = (first.len + kTile - 1) / kTile;
        const int slice_log2 = __ffs(D / cs) - 1, slice = 1 << slice_log2;  // (cs is a power of two)
        const bool mine = warp < 8 && gr < a.rows && first.len >= 0;
        if (warp < 4) row_m[row] = out_m, row_l[row] = out_l;
        cluster_sync();  // also: no CTA's products read K any more, where the parts go
        float* parts = (float*)(sm + L::kK);  // [rank][slice / 4][128 rows][4]
        if (warp < 8) {
            float top = kNoRef, sum = 0.f, ms[8], ls[8];
#pragma unroll
            for (int r = 0; r < 8; r++) {
                ms[r] = kNoRef, ls[r] = 0.f;
                if (r < cs) ms[r] = ld_peer(peer(row_m + row, r)), ls[r] = ld_peer(peer(row_l + row, r));
            }
#pragma unroll
            for (int r = 0; r < 8; r++) top = fmaxf(top, ms[r]);
#pragma unroll
            for (int r = 0; r < 8; r++) sum += ls[r] * ex2(ms[r] - top);
            const float w = ex2(out_m - top) / sum;
            const uint32_t trow = tmem + ((uint32_t)((warp & 3) * 32) << 16);
            const uint32_t* odd = info[(n - 1) & (kInfos - 1)].odd;
            const bool fix = work && (ntc & (cs - 1)) == rank && (odd[0] | odd[1] | odd[2] | odd[3]) != 0;
            tc_fence_after();
#pragma unroll 1
            for (int j = 0; j < D / 2; j += 32) {
                float o[32];
                const int c = grp * (D / 2) + j;
                __syncwarp();
                if (work) {
                    tmem_ld32(trow + kColO + c, o);
                } else {
#pragma unroll
                    for (int i = 0; i < 32; i++) o[i] = 0.f;
                }
                if (fix && mine) add_odd(a, odd, vis + 4 * (gr / group), first.b, head * D + c, o);
                if (mine)
#pragma unroll
                    for (int i = 0; i < 32; i += 4)
                        st_peer4(peer(parts + (((size_t)rank * slice + ((c + i) & (slice - 1))) * 32 + row) * 4, (c + i) >> slice_log2), o[i] * w,
                                 o[i + 1] * w, o[i + 2] * w, o[i + 3] * w);
            }
        }
        cluster_sync();
        if (mine) {
            __nv_bfloat16* orow = a.out + ((size_t)(first.b * (long long)a.T + gr / group) * a.H + head * group + gr % group) * D + rank * slice;
            for (int c = grp * (slice / 2); c < (grp + 1) * (slice / 2); c += 4) {
                float4 v[8], y = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
                for (int r = 0; r < 8; r++)
                    if (r < cs) v[r] = *(const float4*)(parts + (((size_t)r * slice + c) * 32 + row) * 4);
#pragma unroll
                for (int r = 0; r < 8; r++)
                    if (r < cs) y.x += v[r].x, y.y += v[r].y, y.z += v[r].z, y.w += v[r].w;
                *(uint2*)(orow + c) = make_uint2(pack_bf16(y.x, y.y), pack_bf16(y.z, y.w));
            }
        }
    }
    tc_fence_before();
    __syncthreads();
    if (warp == 16) {
        tc_fence_after();
        tmem_dealloc(tmem, 512);
    }
}

struct TcPlan {
    int nteams, mtiles, cluster;  // cluster: CTAs per item, 0: equal runs over the SMs
    long long items;
    bool merge;
    size_t bytes;
};

// An item's queries and result take as long as so many tiles: 30 sequences of 30 to 2000 tokens, 57 rows
// of 8 heads each: 230 us at 0, 156 at 2, 142 at 4, 146 at 9; 6 sequences of 2303: 55.6, 53.6, 53.3, 55.0.
constexpr int kTcExtra = 4;

TcPlan tc_plan(const la_kv4_desc& c, const la_kv4_attn& a)
{
    TcPlan p;
    const int T = 1 + (a.W + a.G) * (a.N - 1), rows = T * (a.n_heads / c.n_kv_heads);
    p.mtiles = ceil_div(rows, kRowsTc);
    p.items = (long long)a.batch * c.n_kv_heads * p.mtiles;
    const int room = c.max_pages * c.page, max_len = a.max_len > 0 && a.max_len < room ? a.max_len : room;
    const int tiles = (max_len + kTile - 1) / kTile + 1;  // of an item, at most
    // Clusters of 4 and 8 leave some of a GPC's SMs over: 38 items of 1 K tokens in fours took two rounds
    // (25.9 us against 15.7 in twos), 16 in eights, too (24.5; 14: 13.2).  32 and 14 fit.  A cluster's time goes with the longest item, equal runs' with all tiles, and 10 tiles'
    // time on top for parts and their merge; of a batch, three quarters of the longest length are
    // taken for the average.  D = 128, 100 rows (us, cluster / runs): 8 items of 4 K tokens 15.8 / 20.8,
    // of 32 K 44.6 / 37.1; 28 of 16 K 45.5 / 44.1, of 32 K 77.5 / 71.4; 28 of 4 to 32 K 76.4 / 48.3;
    // 70 of 16 K 78.4 / 85.5; 114 sequences (one CTA each) of 60 to 500 tokens 16.9 / 24.2, of 250 to 2 K
    // 29.2 / 31.2, of 500 to 4 K 45.8 / 38.1.  Where every run is a whole item, runs need no parts: 152
    // items of 130 tokens 14.7 us, in clusters of one 15.7.
    p.cluster = p.items <= 14 ? 8 : p.items <= 32 ? 4 : 2 * p.items <= kSMs ? 2 : p.items <= kSMs ? 1 : 0;
    while (p.cluster > 2 && p.cluster >= 2 * tiles) p.cluster /= 2;
    if (p.cluster) {
        const long long all = p.items * tiles * (a.batch > 1 ? 3 : 4) / 4;
        if (tiles / p.cluster > all / kSMs + 10) p.cluster = 0;
    }
    const long long units = p.items * (kTcExtra + tiles);
    p.nteams = (int)std::max(1LL, std::min((long long)kSMs, std::max(p.items, units / (kTcExtra + 2))));
    if (p.cluster == 1 && a.batch == 1 && p.nteams == p.items) p.cluster = 0;
    p.merge = !p.cluster && !(a.batch == 1 && p.items % p.nteams == 0);
    p.bytes = p.merge ? (size_t)p.nteams * (2 * part_floats(kRowsTc, c.head_dim) * 4 + sizeof(MergeRec)) : 0;
    return p;
}

template <int D>
cudaError_t go(cudaStream_t s, const TcPlan& p, const Kv4Attn& k)
{
    if (!p.cluster) return launch_pdl(k_kv4_tc<D, false>, dim3(p.nteams), dim3(kTcThreads), TcSmem<D>::kBytes, s, k);
    return launch_cluster(k_kv4_tc<D, true>, (unsigned)p.items, (unsigned)p.cluster, kTcThreads, TcSmem<D>::kBytes, s, k);
}

template <typename K>
bool set_smem(K kern, int bytes)
{
    return cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes) == cudaSuccess;
}

}  // namespace

size_t kv4_tc_bytes(const la_kv4_desc& c, const la_kv4_attn& a) { return tc_plan(c, a).bytes; }

bool kv4_tc_init()
{
    return set_smem(k_kv4_tc<128, false>, TcSmem<128>::kBytes) && set_smem(k_kv4_tc<128, true>, TcSmem<128>::kBytes) &&
           set_smem(k_kv4_tc<64, false>, TcSmem<64>::kBytes) && set_smem(k_kv4_tc<64, true>, TcSmem<64>::kBytes);
}

int launch_kv4_tc(cudaStream_t s, const la_kv4_desc& c, const la_kv4_attn& a, Kv4Attn k)
{
    const TcPlan p = tc_plan(c, a);
    k.mtiles = p.mtiles, k.nteams = p.nteams, k.extra = kTcExtra;
    k.tile_log2 = kTileLog2;
    k.part = p.merge ? (float*)a.workspace : nullptr;
    cudaError_t e = c.head_dim == 128 ? go<128>(s, p, k) : go<64>(s, p, k);
    if (e == cudaSuccess && p.merge) e = launch_kv4_merge(s, k, c.head_dim, kRowsTc);
    return e == cudaSuccess ? LA_OK : LA_ERR_CUDA;
}

}  // namespace la
