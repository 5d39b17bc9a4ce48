// kv16_wide.cu -- the step's masked attention over the paged bf16 cache for
// many rows per KV head, on tcgen05: lookahead steps, prompt blocks, and the
// rows of all sequences that share a prefix.
//
// An item is up to 256 rows of a KV head.  Its keys come in tiles of 128: 8
// blocks of 16, each from a page of the prefix or of the sequence or from the
// step's rows, each two boxes (64 channels x 16 keys) of a tensor map.  Two
// streams of 128 rows work at once, so that one's products run while the other
// weighs: with more than 128 rows each has its own rows and both use every
// tile (a tile is read once for 256 rows: 128 rows a tile would need all that an
// SM can read from L2); with fewer, both have the same rows and take every
// second tile, and join their results at the end.  Per stream and tile
//   S = Q K^T          Q and K in shared memory, S in tensor memory
//   P = exp2((S - M) f)  in bf16, in the place of S
//   O += P V           P from tensor memory, V in shared memory
// with S, M, the sums and O in fp32, half a tile at a time.  The reference M is
// the largest score of a row's first half tile and moves, to the largest since,
// only when a row's P of a half tile sum to more than a bound: weights above 1
// lose no more in bf16 than smaller ones, and O is read back once in many thousand
// tiles.  The half's weights stay in registers until that is known.  The bound is
// 2^15 for a tile's first half and 2^30 for its second (O has room for 2^17 tiles
// of values up to 2^70): a move in the second rounds the first one's weights, in
// their place already, once more, when they are less than 2^-15 of the sum.
//
// Keys that are not there: their scores count as -inf, and their values, of
// which a product would take 0 x NaN, are cleared in shared memory, as are the
// step rows' that are not finite; these are added to the rows that see them at
// the end.
//
// One CTA per SM: warps 0-3 and 4-7 the streams' softmax (a row per thread), 8
// issues the products, 9 and 11 the copies of keys and of values, 10 clears values.
//
// What bounds it.  A tile of 256 rows takes 1.7 us: 1.1 us of a stream's softmax
// and the two products after it (0.27 us each, with the hand-overs 0.6 us), which
// the other stream's softmax only hides in part: tensor pipe 54 %, issue slots
// 41 %, special functions 26 %.  8 steps of 57 rows x 8 heads, 8 KV heads, over
// 8.3 to 9.5 K keys (133 GFLOP): 128 us, 1.04 PFLOP/s.  Measured for that call and not taken:
// 16 softmax warps (147 against 122 us for the kernel: twice the loads from tensor
// memory), streams strictly by turns (150), loads from tensor memory ahead of their
// use (165), sums of unrounded weights (126 against 120), sums by a product (152),
// the next scores made half by half behind the weights' own half (168 against 130),
// values' products by halves (161), more registers for the softmax by setmaxnreg
// (spills).  With up to 128 rows a tile takes what an SM can read: 64 KB in 1.2 us
// where pages are 16 tokens.
#include <cudaTypedefs.h>

#include "kv16_rows.cuh"

namespace la {
namespace {

constexpr int kThreads = 384;
constexpr int kInfos = 8;
constexpr uint32_t kColO = 256;  // tensor memory: S [2][128] (P in their place), O [2][128]

// What is known of a tile; eight in turn, of its keys and of its values (which may
// be there first).
struct alignas(16) TileInfo {
    uint32_t code[2];  // a byte for each block: keys, or 128 + number of the step's block; 0: none
    int blocks, part;  // blocks; are scores to be left out
};

template <int S>
struct Bars {
    uint64_t full[S], empty[S];  // of the ring's stages
    uint64_t s[2], p[2];         // of a stream's tile: scores; weights, its values cleared and the next one's keys
    uint64_t q, o, end;          // of a run: queries; the last products
};

template <int D>
struct WideSmem {
    static constexpr int kAtoms = D / 64;
    static constexpr int kOperand = kAtoms * 128 * 128;  // [atom][128 rows][128 bytes]
    static constexpr int kStages = D == 128 ? 5 : 9;     // K and V by turns: odd, so that each use is known by the fill
    static constexpr int kQ = 0, kRing = 2 * kOperand;
    static constexpr int kVis = kRing + kStages * kOperand;  // [step row][4]: step rows it sees
    static constexpr int kBar = kVis + 128 * 16;
    static constexpr int kInfo = (kBar + (int)sizeof(Bars<kStages>) + 15) / 16 * 16;
    static constexpr int kOdd = kInfo + 2 * kInfos * (int)sizeof(TileInfo);  // [run][4]: step rows whose values are not finite
    static constexpr int kMisc = kOdd + 8 * 16;
    static constexpr int kPre = kMisc + 16;
    static constexpr int kBytes = kPre + (int)sizeof(PreShared);
    static_assert(kBytes <= 227 * 1024, "shared memory");
};

__device__ __forceinline__ int piece_at(int i, int row)
{
    return (i >> 3) * (128 * 128) + row * 128 + (((i & 7) ^ (row & 7)) << 4);
}

// Adds what is not finite among the values of the step rows (bits of odd and see
// both set) to 32 channels from col.
__device__ __noinline__ void add_odd_to(const Kv16Attn& a, const uint32_t* odd, const uint32_t* see, int b, int col, float* o)
{
    for (int key = 0; key < a.T; key++) {
        if (!(((odd[key >> 5] & see[key >> 5]) >> (key & 31)) & 1)) continue;
        const __nv_bfloat16* v = a.vs + (size_t)(b * (long long)a.T + key) * a.v_ld + col;
        for (int i = 0; i < 32; i++) {
            const float x = __bfloat162float(v[i]);
            if (!(fabsf(x) < INFINITY)) o[i] += x;
        }
    }
}

// Which of a tile's scores 32 c .. 32 c + 31 count for a row that sees the step rows `see`.
__device__ __forceinline__ uint32_t counted(const TileInfo& ti, int c, const uint32_t* see)
{
    const uint32_t code = ti.code[c >> 1] >> (16 * (c & 1));
    auto half = [&](uint32_t k) -> uint32_t {
        if (k & 128) return see[(k & 127) >> 1] >> (16 * (k & 1)) & 0xffffu;
        return (1u << k) - 1u;
    };
    return half(code & 255) | half(code >> 8 & 255) << 16;
}

// 64 scores x of a row as weights p = exp2(x f - m), in bf16; returns their sum
// (of the rounded ones: what a weight loses is then lost above and below).
__device__ __forceinline__ float weigh64(const uint32_t (&x)[64], float f, float m, uint32_t (&p)[32])
{
    const uint64_t f2 = la::pair(f, f), c2 = la::pair(-m, -m);
    uint64_t s0 = 0, s1 = 0;
    auto values = [](uint32_t u) { return la::pair(__uint_as_float(u << 16), __uint_as_float(u & 0xffff0000u)); };
#pragma unroll
    for (int j = 0; j < 64; j += 4) {
        float e0, e1, e2, e3;
        unpair(fma2(la::pair(__uint_as_float(x[j]), __uint_as_float(x[j + 1])), f2, c2), e0, e1);
        unpair(fma2(la::pair(__uint_as_float(x[j + 2]), __uint_as_float(x[j + 3])), f2, c2), e2, e3);
        p[j / 2] = pack_bf16(ex2(e0), ex2(e1)), p[j / 2 + 1] = pack_bf16(ex2(e2), ex2(e3));
        s0 = add2(s0, values(p[j / 2])), s1 = add2(s1, values(p[j / 2 + 1]));
    }
    float t0, t1, t2, t3;
    unpair(s0, t0, t1), unpair(s1, t2, t3);
    return (t0 + t1) + (t2 + t3);
}

// 16 bytes, or zeros (then nothing is read)
__device__ __forceinline__ void cp16(uint32_t dst, const void* src, bool there)
{
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(there ? 16 : 0) : "memory");
}

// A wait that gives up ends every later one at once, but no role leaves its
// loops: the named barriers keep their counts.  From then on the role tells the
// others nothing, so that none goes on with what is not there: their own waits end.
struct Wait {
    volatile int* abort_flag;
    int* status;
    bool ok;
    __device__ __forceinline__ void operator()(uint64_t* b, int parity)
    {
        if (!ok || mbar_try_wait(b, parity & 1)) return;
        const unsigned long long t0 = globaltimer();
        while (!try_wait_long(b, parity & 1)) {
            if (*abort_flag || globaltimer() - t0 > kWaitNs) {
                ok = false;
                *abort_flag = 1;
                kv4_raise(status, LA_ERR_TIMEOUT);
                return;
            }
        }
    }
};

// A reference m, as f times a score, does for |m| < 512: it is off by no more than
// 2^-16 then.  Where it is further from 0 (what it is off by grows with it, at 2^31
// past what exp2 can hold) m is kFar, with which any score's weight is past every
// bound, and the score itself is taken away from the others before they are scaled.
// (So it is before a run's first score that counts.)  x - m for every score would be
// one instruction more for two of them: 145 us, not 130, for the call above.
constexpr float kFar = kNoRef;
__device__ __forceinline__ float near_of(float score, float f) { return fabsf(score * f) < 512.f ? score * f : kFar; }

// Takes `far` away from 64 scores, where they are.
__device__ __noinline__ void take_away(uint32_t ts, float far)
{
#pragma unroll 1
    for (int j = 0; j < 64; j += 8) {
        uint32_t y[8];
        tmem_ld8(ts + j, y);
#pragma unroll
        for (int e = 0; e < 8; e++) y[e] = __float_as_uint(__uint_as_float(y[e]) - far);
        tmem_st8(ts + j, y);
    }
    tmem_st_wait();
}


// A stream's tiles of a run, `step` apart from tile n (`done` before them): the
// scores become weights where they are.  Returns the row's reference and sum.  A
// function, so that what its caller keeps over it leaves the registers once and
// not in every tile (spilt around the loop's body, a tile took 2.2 us, not 1.7).
// 64 scores at a time: by 32 the call above took 147 us, by 16 177.
template <int D>
__device__ __noinline__ float2 weigh_tiles(uint8_t* sm, uint32_t trow, int str, int n, int step, int tiles, int done, bool any, const uint32_t* see,
                                           float f, int* status)
{
    using L = WideSmem<D>;
    Bars<L::kStages>& bar = *(Bars<L::kStages>*)(sm + L::kBar);
    uint64_t *b_s = bar.s, *b_p = bar.p;
    const TileInfo* info = (const TileInfo*)(sm + L::kInfo);
    volatile int* abort_flag = (volatile int*)(sm + L::kMisc + 4);
    Wait wait{abort_flag, status, *abort_flag == 0};
    const uint32_t ts = trow + str * 128, to = trow + kColO + str * 128;
    const int lane = threadIdx.x & 31;
    volatile float ref = kNoRef;  // the reference as a score (in memory: it is looked at once in a while, and in a register the call takes 139 us)
    float m = kFar, l = 0.f;
    bool first = true;
    for (int i = 0; i < tiles; i++, done++) {
        wait(b_s + str, done);
        tc_fence_after();
        if (any) {
            const TileInfo ti = info[(n + i * step) & (kInfos - 1)];
            const int n32 = (ti.blocks + 1) >> 1;
            // Half a tile at a time.  Its weights go to the columns of scores that are taken once the reference is
            // known to do for all of them.
#pragma unroll 1
            for (int h = 0; h < 2; h++) {
                if (2 * h < n32) {
                    uint32_t p[32];
                    float sum;
                    bool moved = false;
                    while (true) {
                        uint32_t x[64];
                        tmem_ld64_raw(ts + h * 64, x);
                        if (ti.part) {
                            const uint32_t k0 = counted(ti, 2 * h, see), k1 = counted(ti, 2 * h + 1, see);
#pragma unroll
                            for (int j = 0; j < 32; j++) {
                                if (!((k0 >> j) & 1)) x[j] = 0xff800000u;  // -inf
                                if (!((k1 >> j) & 1)) x[32 + j] = 0xff800000u;
                            }
                        }
                        if (first) {
                            // (of the run's first scores that there are)
                            float t0 = -INFINITY, t1 = -INFINITY;
#pragma unroll
                            for (int j = 0; j < 64; j += 2) t0 = fmaxf(t0, __uint_as_float(x[j])), t1 = fmaxf(t1, __uint_as_float(x[j + 1]));
                            t0 = fmaxf(kNoRef, fmaxf(t0, t1)), m = near_of(t0, f), ref = t0;
                            first = false;
                        }
                        sum = weigh64(x, f, m, p);
                        if (moved || !__any_sync(0xffffffffu, sum > (h ? 0x1p30f : 0x1p15f))) break;
                        moved = true;
                        // (rare) a row's reference moves up to the largest of its scores from here on, where that one counts more
                        // than 2^9 (2^24), and the weights before and the outputs down with it (this tile's scores came behind
                        // the last one's products)
                        float top = -INFINITY;
                        tmem_st_wait();  // (the first half's weights)
#pragma unroll 1
                        for (int c = 2 * h; c < n32; c++) {
                            const uint32_t k = ti.part ? counted(ti, c, see) : ~0u;
#pragma unroll 1
                            for (int j = 0; j < 32; j += 8) {
                                uint32_t y[8];
                                tmem_ld8(ts + c * 32 + j, y);
#pragma unroll
                                for (int e = 0; e < 8; e++)
                                    if ((k >> (j + e)) & 1) top = fmaxf(top, __uint_as_float(y[e]));
                            }
                        }
                        float far = ref;
                        const float power = m == kFar ? (top - far) * f : fmaf(top, f, -m);
                        const bool up = power > (h ? 24.f : 9.f);
                        const float by = up ? ex2(-power) : 1.f;
                        if (up) ref = far = top, m = near_of(top, f);
                        l *= by;
                        const __nv_bfloat162 by2 = __float2bfloat162_rn(by);
#pragma unroll 1
                        for (int j = 0; j < h * 32; j += 8) {
                            uint32_t y[8];
                            tmem_ld8(ts + j, y);
#pragma unroll
                            for (int e = 0; e < 8; e++) {
                                const __nv_bfloat162 z = __hmul2(*reinterpret_cast<__nv_bfloat162*>(&y[e]), by2);
                                y[e] = *reinterpret_cast<const uint32_t*>(&z);
                            }
                            tmem_st8(ts + j, y);
                        }
#pragma unroll 1
                        for (int j = 0; i > 0 && j < D; j += 8) {
                            uint32_t o[8];
                            tmem_ld8(to + j, o);
#pragma unroll
                            for (int e = 0; e < 8; e++) o[e] = __float_as_uint(__uint_as_float(o[e]) * by);
                            tmem_st8(to + j, o);
                        }
                        take_away(ts + h * 64, m == kFar ? far : 0.f);
                        m = m == kFar ? 0.f : m;
                    }
                    if (moved) m = near_of(ref, f);
                    l += sum;
                    tmem_st16(ts + h * 32, p);
                    tmem_st16(ts + h * 32 + 16, p + 16);
                }
            }
            tmem_st_wait();
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0 && wait.ok) mbar_arrive(b_p + str);
    }
    return make_float2(ref, l);
}

// Tensor maps of keys and values: blocks of 16 rows of the step and of pages, and whole pages.
struct Maps {
    CUtensorMap step[2], block[2], page[2];
};

// What a CTA does.  kBeside: other CTAs of the kernel do other things, and it is known
// (given) where this one begins.
struct Given {
    Prefixes pre;
    Shares shares;
    Start start;
};
template <int D, bool kBeside>
__device__ __forceinline__ void wide_cta(const Kv16Attn& a, const Kv16Sched& s, const Maps& maps, int rows_all, uint8_t* sm, const Given& given)
{
    using L = WideSmem<D>;
    constexpr int kSt = L::kStages;
    Bars<kSt>& bar = *(Bars<kSt>*)(sm + L::kBar);
    uint64_t *b_full = bar.full, *b_empty = bar.empty, *b_s = bar.s, *b_p = bar.p, *b_q = &bar.q,
             *b_o = &bar.o, *b_end = &bar.end;
    TileInfo* info = (TileInfo*)(sm + L::kInfo);
    uint32_t *vis = (uint32_t*)(sm + L::kVis), *odds = (uint32_t*)(sm + L::kOdd);
    uint32_t* tmem_slot = (uint32_t*)(sm + L::kMisc);
    volatile int* abort_flag = (volatile int*)(sm + L::kMisc + 4);
    // (before the queries come)
    Scan* sc = (Scan*)(sm + L::kQ);
    Start* start = (Start*)(sc + 1);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, group = a.group;

    if (warp == 8) tmem_alloc(tmem_slot, 512);
    if (threadIdx.x == 0) {
        for (int i = 0; i < kSt; i++) mbar_init(b_full + i, 1), mbar_init(b_empty + i, 1);
        for (int i = 0; i < 2; i++) mbar_init(b_s + i, 1), mbar_init(b_p + i, 5);
        mbar_init(b_q, 8);
        mbar_init(b_o, 1);
        mbar_init(b_end, 1);
        *abort_flag = 0;
        mbar_fence_init();
    }
    if (threadIdx.x >= 32 && threadIdx.x < 38) prefetch_map(&maps.step[0] + (threadIdx.x - 32));
    if (s.n_seq)
        for (int i = threadIdx.x - 64; i >= 0 && i < a.T; i += kThreads) {
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
    if (!kBeside) {
        pdl_wait();
        pdl_trigger();
    }
    tc_fence_before();
    const Prefixes pre = kBeside ? given.pre : find_starts<WideKind>(a, s, start, sc, (PreShared*)(sm + L::kPre));
    if (kBeside) __syncthreads();
    tc_fence_after();
    const Shares sh = kBeside ? given.shares : sc->shares;
    const Start st = kBeside ? given.start : *start;
    const uint32_t tmem = *tmem_slot;
    // (the swizzle and the products' descriptors count from multiples of 1024)
    const bool placed = (smem_u32(sm) & 1023) == 0, work = st.count > 0 && placed;
    if (!placed && threadIdx.x == 0) kv4_raise(a.status, LA_ERR_CUDA);
    __syncthreads();

    Wait wait{abort_flag, a.status, true};
    const bool& ok = wait.ok;
    int n = 0;     // tiles so far
    int segs = 0;  // runs with tiles so far
    Run<WideKind> run;
    if (work) run.begin(a, s, pre, st, sh);
    if (threadIdx.x == 0 && s.finish && s.items) s.items[blockIdx.x].n = 0;
    if (work && warp < 8) {
        // ------------------------------------------------------------ softmax
        const int q = warp & 3, str = warp >> 2, row = q * 32 + lane;
        const uint32_t trow = tmem + ((uint32_t)(q * 32) << 16), to = trow + kColO + str * 128;
        int done = 0;  // this stream's tiles so far
        do {
            const int nt = run.t1 - run.t0;
            if (run.x.nu && threadIdx.x == 0) run.note(a, s, pre, sh, blockIdx.x);
            if (nt <= 0) {
                // (units, but no keys)
                if (run.x.nu && str == 0)
                    for (int i = 0; i < 2; i++) {
                        float* col = s.slots + ((size_t)blockIdx.x * 2 + run.slot()) * wide_part(D) + i * 128 * (D + 2) + row;
                        col[D * 128] = kNoRef, col[(D + 1) * 128] = 0.f;
                    }
                continue;
            }
            const Entry& x = run.x;
            const int g = run.item / x.mt, r0 = (run.item - g * x.mt) * kWideRows, nrows = min(kWideRows, x.rows - r0);
            const bool pair = nrows > 128;
            const int tiles = pair ? nt : (nt + 1 - str) >> 1;
            const int mine = pair ? str * 128 : 0;  // of the item's rows, the stream's first
            const int gr = x.row0 + r0 + mine + row;
            const bool live_row = mine + row < nrows, any = mine + q * 32 < nrows;
            // ---- queries.  Neighbouring threads take neighbouring 16-byte pieces of a row, all on their way at once.  (In a
            // short loop: unrolled it cost the tiles' loops 10 %, the roles' code shares the instruction caches.  Asking
            // for the next run's while this one's result is written won nothing.)
            if (tiles > 0) {
                constexpr int kPieces = D / 8, kPass = 128 / kPieces;
                const int t = threadIdx.x & 127, pc = t % kPieces, rr = t / kPieces;
                const int first = x.row0 + r0 + mine + rr;
                int si = first / group, sj = first - si * group;
                const int di = kPass / group, dj = kPass - di * group;
                const uint32_t dst = smem_u32(sm) + L::kQ + str * L::kOperand;
#pragma unroll 1
                for (int i = 0; i < 128 / kPass; i++) {
                    const bool there = mine + rr + i * kPass < nrows;
                    const size_t at = there ? (size_t)si * a.q_ld + (size_t)(g * group + sj) * D + 8 * pc : 0;
                    cp16(dst + piece_at(pc, rr + i * kPass), a.q + at, there);
                    si += di, sj += dj;
                    if (sj >= group) sj -= group, si++;
                }
                asm volatile("cp.async.wait_all;" ::: "memory");
                fence_proxy_async();
            }
            __syncwarp();
            if (lane == 0 && ok) mbar_arrive(b_q);
            const int step_row = x.b < 0 ? 0 : ((gr - x.row0) / group < a.T ? (gr - x.row0) / group : a.T - 1);
            const uint32_t* see = vis + 4 * step_row;
            const float2 y = weigh_tiles<D>(sm, trow, str, n + (pair ? 0 : str), pair ? 1 : 2, tiles, done, any, see, a.sl2, a.status);
            float m = y.x, l = y.y;
            wait.ok = wait.ok && *abort_flag == 0;
            done += tiles;
            // ---- the run's result
            wait(b_o, segs);
            tc_fence_after();
            const bool all = run.all();
            const uint32_t* odd = odds + (segs & 7) * 4;
            const bool fix = x.b >= 0 && (odd[0] | odd[1] | odd[2] | odd[3]) != 0;
            float w0 = 1.f, w1 = 0.f;  // of this stream's outputs, and of the other's
            int c0 = 0, c1 = D;
            if (!pair) {
                // both streams' rows are the same: half of the channels each
                float2* ml = (float2*)(sm + L::kQ);  // (the queries are done with)
                ml[str * 128 + row] = make_float2(m, l);
                named_sync(1, 256);
                const float2 other = ml[(str ^ 1) * 128 + row];
                const float top = fmaxf(m, other.x);
                w0 = ex2((m - top) * a.sl2), w1 = ex2((other.x - top) * a.sl2);
                l = l * w0 + other.y * w1, m = top;
                c0 = str * (D / 2), c1 = c0 + D / 2;
            }
            if (any) {
                const bool out = all && s.finish;
                const float inv = 1.f / l;
                float* col = nullptr;
                size_t pitch = 128;
                if (all) col = (x.b < 0 ? s.whole_pre : s.whole) + (size_t)g * (D + 2) * rows_all + gr, pitch = rows_all;
                else col = s.slots + ((size_t)blockIdx.x * 2 + run.slot()) * wide_part(D) + (mine ? 128 * (D + 2) : 0) + row;
                __nv_bfloat16* orow = a.out + ((size_t)(gr / group) * a.H + (size_t)g * group + gr % group) * D;
#pragma unroll 1
                for (int c = c0; c < c1; c += 32) {
                    float o[32];
                    __syncwarp();
                    tmem_ld32(to + c, o);
                    if (!pair) {
                        float u[32];
                        // (a stream without tiles has weight 0, and whatever is in its outputs' place)
                        tmem_ld32(trow + kColO + (str ^ 1) * 128 + c, u);
                        const bool h0 = tiles > 0, h1 = nt > 1 || str == 1;
#pragma unroll
                        for (int j = 0; j < 32; j++) o[j] = (h0 ? o[j] * w0 : 0.f) + (h1 ? u[j] * w1 : 0.f);
                    }
                    if (fix && live_row) {
                        float t[32];  // (in memory for the call; o stays in registers)
#pragma unroll
                        for (int j = 0; j < 32; j++) t[j] = o[j];
                        add_odd_to(a, odd, see, x.b, g * D + c, t);
#pragma unroll
                        for (int j = 0; j < 32; j++) o[j] = t[j];
                    }
                    if (!live_row) continue;
                    if (out) {
#pragma unroll
                        for (int j = 0; j < 32; j += 8)
                            *(uint4*)(orow + c + j) = make_uint4(pack_bf16(o[j] * inv, o[j + 1] * inv), pack_bf16(o[j + 2] * inv, o[j + 3] * inv),
                                                                 pack_bf16(o[j + 4] * inv, o[j + 5] * inv), pack_bf16(o[j + 6] * inv, o[j + 7] * inv));
                    } else {
#pragma unroll
                        for (int j = 0; j < 32; j++) col[(size_t)(c + j) * pitch] = o[j];  // a line per warp
                    }
                }
                if (!out && live_row && (pair || str == 0)) col[(size_t)D * pitch] = m, col[(size_t)(D + 1) * pitch] = l;
            }
            tc_fence_before();
            if (!pair) named_sync(1, 256);  // the other stream's outputs are read, and the queries' place is free
            n += nt;
            segs++;
        } while (run.next(a, s, pre));
    } else if (work && warp == 8) {
        // ----------------------------------------------------------- products
        constexpr uint32_t id_s = idesc_bf16(128, 0, false), id_o = idesc_bf16(128, D, true);
        const uint32_t base = smem_u32(sm);
        const uint64_t dk = desc_sw128_kmajor(base), dv = desc_sw128_mnmajor(base, 128 * 128);
        const uint32_t k_lo = (uint32_t)dk, k_hi = (uint32_t)(dk >> 32), v_lo = (uint32_t)dv, v_hi = (uint32_t)(dv >> 32);
        const bool chosen = elect_one();
        int weighed0 = 0, weighed1 = 0;
        do {
            const int nt = run.t1 - run.t0;
            if (nt <= 0) continue;
            const int g = run.item / run.x.mt, r0 = (run.item - g * run.x.mt) * kWideRows;
            const bool pair = min(kWideRows, run.x.rows - r0) > 128;
            const int jobs = pair ? 2 * nt : nt;  // a tile for a stream: the streams by turns
            auto tile_of = [&](int j) { return n + (pair ? j >> 1 : j); };
            auto scores = [&](int j, int stage, int blocks) {
                const int str = j & 1;
                const bool go = chosen && ok;
                const uint32_t id = id_s | (uint32_t)(2 * blocks) << 17, ka = k_lo + ((L::kRing + stage * L::kOperand) >> 4),
                               qa = k_lo + ((L::kQ + str * L::kOperand) >> 4);
#pragma unroll
                for (int k = 0; k < D / 16; k++) {
                    const uint32_t at = ((k >> 2) * (128 * 128) + (k & 3) * 32) >> 4;
                    mma_ss_if(go, tmem + str * 128, qa + at, ka + at, k_hi, id, k > 0);
                }
                commit_if(go, b_s + str);
                commit_if(go && (!pair || str), b_empty + stage);
            };
            auto blocks_of_tile = [&](int tile) { return info[tile & (kInfos - 1)].blocks; };
            wait(b_q, segs);
            for (int j = 0; j < min(jobs, 2); j++) {
                const int tile = tile_of(j), fill = 2 * tile;
                wait(b_full + fill % kSt, fill / kSt);
                tc_fence_after();
                scores(j, fill % kSt, blocks_of_tile(tile));
            }
#pragma unroll 1
            for (int j = 0; j < jobs; j++) {
                const int str = j & 1, tile = tile_of(j), stage = (2 * tile + 1) % kSt, stage_k = 2 * tile_of(j + 2) % kSt;
                const uint32_t va = v_lo + ((L::kRing + stage * L::kOperand) >> 4), d = tmem + kColO + str * 128, pa = tmem + str * 128;
                wait(b_p + str, str ? weighed1 : weighed0);
                if (str) weighed1++;
                else weighed0++;
                const int blocks = blocks_of_tile(tile);
                int next = blocks_of_tile(tile_of(j + 2));
                tc_fence_after();
                const bool go = chosen && ok;
                auto step16 = [&](int k) { mma_ts_if(go, d, pa + k * 8, va + ((k * 16 * 128) >> 4), v_hi, id_o, j > 1 || k > 0); };
                if (blocks == 8) {
#pragma unroll
                    for (int k = 0; k < 8; k++) step16(k);
                } else {
#pragma unroll 1
                    for (int k = 0; k < blocks; k++) step16(k);
                }
                commit_if(go && (!pair || str), b_empty + stage);
                // (in the place of this tile's weights, behind their products)
                if (j + 2 < jobs) {
                    if (!pair) wait(b_full + stage_k, 2 * tile_of(j + 2) / kSt), next = blocks_of_tile(tile_of(j + 2)), tc_fence_after();
                    scores(j + 2, stage_k, next);
                }
            }
            commit_if(chosen && ok, b_o);
            n += nt;
            segs++;
        } while (run.next(a, s, pre));
        if (!ok && chosen) {
            // let the products that were issued finish before the memory goes
            mma_commit(b_end);
            mbar_drain(b_end, 0);
        }
        __syncwarp();
    } else if (work && (warp == 9 || warp == 11)) {
        // -------------------------------------------------------------- copies
        // A lane for each block and half of the channels; where a page's blocks are in the tile side by side, the
        // first block's lane brings all of them (a warp of lanes with a box of 16 rows each brings 40 GB/s, two
        // warps 56, one with boxes of 64 rows 68).
        // what is read once goes from L2 first: tables, parts and code stay
        const uint64_t once = policy_evict_first(), shared = policy_evict_normal();
        constexpr int kAtoms = L::kAtoms;
        const int v = warp == 11, blk = lane / kAtoms, atom = lane % kAtoms, per_page = 1 << (a.page_log2 - 4);
        do {
            if (run.t1 <= run.t0) continue;
            const Entry& x = run.x;
            const int g = run.item / x.mt, nc = x.nb_cached();
            const uint64_t pol_pre = x.b < 0 && x.mt == 1 ? once : shared, pol_own = x.mt == 1 ? once : shared;
            // block kb's page (its table entry is looked up a tile ahead)
            auto page_of = [&](int kb) {
                if (blk >= 8 || kb >= nc) return 0;
                const bool own = kb >= x.nb_pre;
                const int at = (own ? kb - x.nb_pre : kb) * 16 >> a.page_log2;
                return own ? a.table[(size_t)x.b * a.max_pages + at] : a.ptable[(size_t)x.p * a.pp + at];
            };
            int next = page_of(run.t0 * 8 + blk);
            for (int tile = run.t0; tile < run.t1; tile++, n++) {
                const int kb = tile * 8 + blk, page = next, blocks = min(8, x.nb - tile * 8);
                if (tile + 1 < run.t1) next = page_of(kb + 8);
                const bool mine = blk < blocks, cached = mine && kb < nc, own = kb >= x.nb_pre;
                const bool bad = cached && (unsigned)page >= (unsigned)a.n_pages;
                const int sb = own ? kb - x.nb_pre : kb, segment = own ? nc - x.nb_pre : x.nb_pre;  // of the segment's blocks
                const int tok = sb * 16, live = cached ? min(16, (own ? x.len : x.plen) - tok) : min(16, a.T - (kb - nc) * 16);
                const int in_page = sb & (per_page - 1), p0 = blk - in_page;  // the page's first block, in the tile
                const bool whole = per_page > 1 && cached && p0 >= 0 && p0 + per_page <= 8 && sb - in_page + per_page <= segment;
                const int boxes = __popc(__ballot_sync(0xffffffffu, mine && !bad));
                const int cx = (cached ? 0 : g * D) + atom * 64;
                const int cy = cached ? (int)((((long long)page * a.Hkv + g) << a.page_log2) + (tok & ((1 << a.page_log2) - 1)))
                                      : x.b * a.T + (kb - nc) * 16;
                const int fill = 2 * n + v, stage = fill % kSt;
                // (The parity could be that of the phase two before, were fill - 2 kSt not known to be done with.  Stages are
                // done with in the order of the products, that of their fills but for neighbours (K0 K1 V0 K2 V1 ... where
                // the streams take alternate tiles), and this warp has waited for fill - 2 - kSt, at least 3 fills later.)
                if (fill >= kSt) wait(b_empty + stage, fill / kSt - 1);
                const bool go = __all_sync(0xffffffffu, ok);
                const uint32_t code = !mine || bad ? 0u : cached ? (uint32_t)live : 128u + (kb - nc);
                const uint32_t mask = atom == 0 && blk < 8 ? code << (8 * (blk & 3)) : 0u;
                const uint32_t lo = __reduce_or_sync(0xffffffffu, blk < 4 ? mask : 0u), hi = __reduce_or_sync(0xffffffffu, blk < 4 ? 0u : mask);
                const bool part = __any_sync(0xffffffffu, blk < 8 && code != 16);
                if (lane == 0 && go) {
                    TileInfo* ti = info + v * kInfos + (n & (kInfos - 1));
                    ti->code[0] = lo, ti->code[1] = hi, ti->blocks = blocks, ti->part = part;
                }
                if (bad) kv4_raise(a.status, LA_ERR_ARG);
                if (!go) continue;
                if (lane == 0) mbar_expect_tx(b_full + stage, boxes * 2048);
                __syncwarp();
                if (mine && !bad && (!whole || in_page == 0))
                    tma_load_2d((cached ? whole ? maps.page : maps.block : maps.step) + v, b_full + stage,
                                sm + L::kRing + stage * L::kOperand + atom * (128 * 128) + blk * 2048, cx, cy, own ? pol_own : pol_pre);
                __syncwarp();
            }
        } while (run.next(a, s, pre));
        // no copy may still be on its way when the CTA ends
        // (a stage's last fill: before it the parity would be another's)
        for (int fill = 2 * (n - 1) + v; fill >= 0 && fill >= 2 * n - kSt; fill -= 2) mbar_drain(b_full + fill % kSt, (fill / kSt) & 1);
    } else if (work) {
        // ------------------------------------------------------- values cleared
        // (and one word to the products for all that is to be there beside the weights)
        int said0 = 0, said1 = 0;
        do {
            const int nt = run.t1 - run.t0;
            if (nt <= 0) continue;
            const int g = run.item / run.x.mt, r0 = (run.item - g * run.x.mt) * kWideRows;
            const bool pair = min(kWideRows, run.x.rows - r0) > 128;
            uint32_t* odd = odds + (segs & 7) * 4;
            if (lane < 4) odd[lane] = 0;
            __syncwarp();
            for (int i = 0; i < nt; i++, n++) {
                const int fill = 2 * n + 1, stage = fill % kSt, after = fill + 1;
                // A wait's parity tells a phase from the one before it, not from the one before that.  The stage's last
                // fill were the keys of two tiles ago (or earlier ones): loads end in any order, so these have to be
                // known to be there, by a wait for them (below) or for their scores' weights.
                const bool for0 = pair || !(i & 1), for1 = pair || (i & 1);
                auto last_words = [&](bool w0, bool w1) {
                    if (w0 && said0) wait(b_p, said0 - 1);
                    if (w1 && said1) wait(b_p + 1, said1 - 1);
                };
                if (i == 0) last_words(true, true);
                else if (!pair) last_words(for0, for1);
                wait(b_full + stage, fill / kSt);
                const TileInfo ti = info[kInfos + (n & (kInfos - 1))];
                if (ti.part && ok) {
                    uint8_t* v = sm + L::kRing + stage * L::kOperand;
                    for (int blk = 0; blk < ti.blocks; blk++) {
                        const uint32_t code = ti.code[blk >> 2] >> (8 * (blk & 3)) & 255;
                        const bool step = code & 128;
                        const int j0 = (code & 127) * 16, live = step ? min(16, a.T - j0) : (int)code;
                        const bool look = step && a.T > 1;
                        if (live == 16 && !look) continue;
                        // (a lane's pieces are in rows lane / 8, + 4, ..., of each half of the channels)
                        uint4* at = (uint4*)(v + blk * 2048) + lane;
                        constexpr int kPieces = 4 * L::kAtoms, kAtomStep = 128 * 128 / 16;
                        uint32_t top = 0;  // the largest exponent
                        if (look) {
                            uint4 u[kPieces];
#pragma unroll
                            for (int k = 0; k < kPieces; k++) u[k] = at[(k >> 2) * kAtomStep + (k & 3) * 32];
#pragma unroll
                            for (int k = 0; k < kPieces; k++) {
                                const uint32_t w[4] = {u[k].x, u[k].y, u[k].z, u[k].w};
#pragma unroll
                                for (int c = 0; c < 4; c++) top = max(top, max(w[c] & 0x7f80u, (w[c] >> 16) & 0x7f80u));
                            }
                        }
                        if (__any_sync(0xffffffffu, top == 0x7f80u)) {
                            // (rare)
#pragma unroll 1
                            for (int k = 0; k < kPieces; k++) {
                                uint4* p = at + (k >> 2) * kAtomStep + (k & 3) * 32;
                                const uint4 u = *p;
                                uint32_t w[4] = {u.x, u.y, u.z, u.w};
                                bool found = false;
#pragma unroll
                                for (int c = 0; c < 4; c++) {
                                    const bool b0 = (w[c] & 0x7f80u) == 0x7f80u, b1 = (w[c] & 0x7f800000u) == 0x7f800000u;
                                    if (b0) w[c] &= 0xffff0000u;
                                    if (b1) w[c] &= 0x0000ffffu;
                                    found |= b0 || b1;
                                }
                                const int row = j0 + (lane >> 3) + (k & 3) * 4;
                                if (found) *p = make_uint4(w[0], w[1], w[2], w[3]);
                                if (found && row < a.T) atomicOr(&odd[row >> 5], 1u << (row & 31));
                            }
                        }
                        if (live < 16)
#pragma unroll
                            for (int k = 0; k < kPieces; k++)
                                if ((lane >> 3) + (k & 3) * 4 >= live) at[(k >> 2) * kAtomStep + (k & 3) * 32] = make_uint4(0, 0, 0, 0);
                    }
                    fence_proxy_async();
                }
                // (where both streams use a tile, the next one's keys were asked for two tiles ago; else they may still
                // be on their way, and the products with these values go first)
                if (pair && i + 1 < nt) wait(b_full + after % kSt, after / kSt);
                last_words(for0, for1);  // (not into the phase of the stream's tile before)
                if (for0) said0++;
                if (for1) said1++;
                __syncwarp();
                if (lane == 0 && ok) {
                    if (for0) mbar_arrive(b_p);
                    if (for1) mbar_arrive(b_p + 1);
                }
            }
            segs++;
        } while (run.next(a, s, pre));
    }
    tc_fence_before();
    __syncthreads();
    if (warp == 8) {
        tc_fence_after();
        tmem_dealloc(tmem, 512);
    }
}

template <int D>
__global__ void __launch_bounds__(kThreads, 1)
    k_kv16_wide(const __grid_constant__ Kv16Attn a, const __grid_constant__ Kv16Sched s, const __grid_constant__ Maps maps, int rows_all)
{
    extern __shared__ __align__(1024) uint8_t sm[];
    wide_cta<D, false>(a, s, maps, rows_all, sm, {});
}

// Prefixes by themselves, and their sequences of at most 16 rows a KV head beside them
// on CTAs of their own (as a second kernel these would have to wait for the first one's
// end before they may read what earlier calls wrote).
constexpr int kRowWarps = kThreads / 32;
template <int D>
struct BesideSmem {
    using Rows = RowsSmem<D, kRowWarps>;
    // where the schedules are found: behind the rings of rows_team (in wide_cta's stages, until tiles come)
    static constexpr int kScan = Rows::kScan, kStarts = kScan + 2 * (int)sizeof(Scan), kEnd = (kStarts + kRowWarps * (int)sizeof(Start) + 15) / 16 * 16;
    static constexpr int kPre = WideSmem<D>::kPre > kEnd ? WideSmem<D>::kPre : kEnd;
    static constexpr int kBytes = kPre + (int)sizeof(PreShared);
    static_assert(kBytes <= 227 * 1024, "shared memory");
};

template <int D>
__global__ void __launch_bounds__(kThreads, 1) k_kv16_beside(const __grid_constant__ Kv16Attn a, const __grid_constant__ Kv16Sched sp,
                                                             const __grid_constant__ Kv16Sched ss, const __grid_constant__ Maps maps, int rows_all)
{
    using L = BesideSmem<D>;
    extern __shared__ __align__(1024) uint8_t sm[];
    pdl_wait();
    pdl_trigger();
    Scan* sc = (Scan*)(sm + L::kScan);
    Start* starts = (Start*)(sm + L::kStarts);
    Prefixes pre;
    const int ctas = find_starts_beside<D>(a, sp, ss, starts, sc, (PreShared*)(sm + L::kPre), pre);
    if ((int)blockIdx.x < ctas) wide_cta<D, true>(a, sp, maps, rows_all, sm, Given{pre, sc[0].shares, *starts});
    else rows_team<D, kRowWarps>(a, ss, sm, pre, sc[1].shares, starts[threadIdx.x >> 5]);
}

PFN_cuTensorMapEncodeTiled_v12000 encode_fn()
{
    static const PFN_cuTensorMapEncodeTiled_v12000 fn = [] {
        cudaDriverEntryPointQueryResult q;
        void* p = nullptr;
        const bool ok = cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault, &q) == cudaSuccess &&
                        q == cudaDriverEntryPointSuccess;
        return ok ? (PFN_cuTensorMapEncodeTiled_v12000)p : nullptr;
    }();
    return fn;
}

// A map over rows `ld` elements apart, boxes of 64 channels x `high` rows, 128-byte
// swizzle; rows past the last read as zeros.
bool encode(CUtensorMap* m, const void* base, long long rows, int cols, size_t ld, int high)
{
    const cuuint64_t dims[2] = {(cuuint64_t)cols, (cuuint64_t)rows}, strides[1] = {(cuuint64_t)ld * 2};
    const cuuint32_t box[2] = {64, (cuuint32_t)high}, es[2] = {1, 1};
    return encode_fn()(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, const_cast<void*>(base), dims, strides, box, es, CU_TENSOR_MAP_INTERLEAVE_NONE,
                       CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

}  // namespace

int kv16_wide_teams() { return kSMs; }
int kv16_beside_teams() { return kSMs * kRowWarps; }

bool kv16_wide_init()
{
    auto room = [](auto* kernel, int bytes) { return cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes) == cudaSuccess; };
    return encode_fn() && room(k_kv16_wide<128>, WideSmem<128>::kBytes) && room(k_kv16_wide<64>, WideSmem<64>::kBytes) &&
           room(k_kv16_beside<128>, BesideSmem<128>::kBytes) && room(k_kv16_beside<64>, BesideSmem<64>::kBytes);
}

// beside: the sequences' schedule, where the same kernel takes them.
int launch_kv16_wide(cudaStream_t s, const Kv16Attn& a, const Kv16Sched& w, const Kv16Sched* beside, int D, int rows_all)
{
    Maps m;
    const long long rows = (long long)a.n_pages * a.Hkv << a.page_log2, steps = (long long)a.B * a.T;
    if (rows >= 1LL << 31) return LA_ERR_ARG;  // (more than the card holds)
    const void *pages[2] = {a.kp, a.vp}, *step[2] = {a.ks, a.vs};
    for (int v = 0; v < 2; v++)
        if (!encode(&m.step[v], step[v], steps, a.Hkv * D, v ? a.v_ld : a.k_ld, 16) || !encode(&m.block[v], pages[v], rows, D, D, 16) ||
            !encode(&m.page[v], pages[v], rows, D, D, 1 << a.page_log2))
            return LA_ERR_CUDA;
    const dim3 grid(w.nteams), block(kThreads);
    cudaError_t e;
    if (beside)
        e = D == 128 ? launch_pdl(k_kv16_beside<128>, grid, block, BesideSmem<128>::kBytes, s, a, w, *beside, m, rows_all)
                     : launch_pdl(k_kv16_beside<64>, grid, block, BesideSmem<64>::kBytes, s, a, w, *beside, m, rows_all);
    else
        e = D == 128 ? launch_pdl(k_kv16_wide<128>, grid, block, WideSmem<128>::kBytes, s, a, w, m, rows_all)
                     : launch_pdl(k_kv16_wide<64>, grid, block, WideSmem<64>::kBytes, s, a, w, m, rows_all);
    return e == cudaSuccess ? LA_OK : LA_ERR_CUDA;
}

}  // namespace la
