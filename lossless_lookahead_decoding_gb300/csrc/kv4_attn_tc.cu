// kv4_attn_tc.cu -- the step's masked attention over the paged 4-bit cache for
// many rows per KV head, on tcgen05: lookahead steps, prompt blocks, grouped
// heads with several step rows.
//
// An item is 128 rows (step rows x query heads of one KV head) of a sequence;
// its keys come in tiles of 128: cached ones, then one tile of the step's own
// rows under the mask.  Per tile, in fp16 with fp32 sums:
//   S = Q K^T          Q and K in shared memory, S in tensor memory
//   P = exp2(S f - M)  written over S
//   O += P V           P from tensor memory, V in shared memory
// K and V are unpacked by 8 warps, one key row per two threads: masking two
// codes out of a word leaves fp16 subnormals (c 2^-24 or c 2^-20), and one
// fused multiply-add a pair gives (c - z) s, brought to the tile's own power
// of two: with E the largest scale's, s 2^-E < 2^-8, so a code step has at
// least 11 bits where the scale is within 2^-6 of the tile's largest and loses
// 2^-25 absolute below.  Rounding: q exact (a power of two per row), K and V
// values 2^-11 relative, P 2^-11, the output to bf16; S, the softmax sums and
// O stay in fp32.  The tiles' powers of two go into the exponent of exp2 and,
// for V, into the running reference M, which moves only when a p V unit
// exceeds 2^8.
//
// Tensor bound for full row tiles (128 x 128 x D x 2 products a tile, 1024
// cycles at D = 128), HBM and unpacking bound for few rows.  All roles run at
// once on neighbouring tiles, one CTA per SM: warps 0-7 softmax (a row per
// thread and half of the columns), 8-15 unpack, 16 issues the MMAs, 17 copies
// code blocks ahead.  S, K and V are double buffered, codes triple.
#include <algorithm>
#include <cmath>

#include "kv4_sched.cuh"

namespace la {

namespace {

constexpr int kTcThreads = 576;
constexpr int kTileLog2 = 7, kTile = 128;
constexpr int kRowsTc = 128;
constexpr int kRing = 3;

constexpr uint32_t idesc_f16(int M, int N, bool b_mn)
{
    return idesc_bf16(M, N, b_mn) & ~((1u << 7) | (1u << 10));  // A and B in fp16
}

// D += A B with A (fp16 pairs, K along the columns) in tensor memory.
__device__ __forceinline__ void mma_ts(uint32_t d_tmem, uint32_t a_tmem, uint64_t b, uint32_t idesc, uint32_t acc)
{
    asm volatile(
        "{\n .reg .pred p;\n setp.ne.b32 p, %4, 0;\n tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n}\n" ::"r"(
            d_tmem),
        "r"(a_tmem), "l"(b), "r"(idesc), "r"(acc));
}

// 16 columns of this thread's lane of tensor memory.
__device__ __forceinline__ void tmem_st16(uint32_t taddr, const uint32_t* r)
{
    asm volatile("tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};" ::"r"(
                     taddr),
                 "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]),
                 "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
                 : "memory");
}
__device__ __forceinline__ void tmem_st_wait() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

__device__ __forceinline__ float pow2i(int e)  // 2^e, e in -126 .. 127
{
    return __uint_as_float((uint32_t)(e + 127) << 23);
}

// x 2^e for any e that two such factors reach
__device__ __forceinline__ float scale2(float x, int e) { return x * pow2i(e >> 1) * pow2i(e - (e >> 1)); }

// What the softmax needs to know of a tile; four in turn (a tile's entry is
// written again four tiles later, when its softmax is long done).
struct TileInfo {
    int live, bad;        // keys, and a bit per block of 16 whose page is not in the pool
    int ek, ev;           // powers of two of K and V
    uint32_t odd[4];      // step rows with a NaN or an infinity among their values
};

template <int D>
struct TcSmem {
    static constexpr int kAtoms = D / 64;
    static constexpr int kOperand = kAtoms * 128 * 128;       // [atom][128 rows][128 bytes]
    static constexpr int kQ = 0, kK = kOperand, kV = kK + 2 * kOperand;
    static constexpr int kCodes = kV + 2 * kOperand;
    static constexpr int kStage = 8 * kv4_block_bytes(D);
    static constexpr int kVis = kCodes + kRing * kStage;      // [step row][4]: step rows it sees
    static constexpr int kRowF = kVis + 128 * 16;             // [2 runs] per row: what undoes q's power of two
    static constexpr int kRed = kRowF + 2 * 128 * 4;              // [2 tiles][2 halves][128 rows]
    static constexpr int kInfo = kRed + 4 * 128 * 4;          // TileInfo[4]
    static constexpr int kBar = kInfo + 4 * (int)sizeof(TileInfo);
    static constexpr int kMisc = kBar + 32 * 8;               // ring info, reduction words, start, scan scratch
    static constexpr int kBytes = kMisc + 512 + 1024;         // 1024: to align the base
};

enum {  // barriers
    kFull = 0, kEmpty = 3, kKReady = 6, kVReady = 8, kSDone = 10, kODone = 12, kPReady = 14, kQReady = 16, kOFree = 17, kEnd = 18
};

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

template <int D>
__global__ void __launch_bounds__(kTcThreads, 1) k_kv4_tc(Kv4Attn a)
{
    using L = TcSmem<D>;
    extern __shared__ uint8_t smem_raw[];
    uint8_t* sm = (uint8_t*)(((uintptr_t)smem_raw + 1023) & ~(uintptr_t)1023);
    uint64_t* bar = (uint64_t*)(sm + L::kBar);
    TileInfo* info = (TileInfo*)(sm + L::kInfo);
    uint32_t* vis = (uint32_t*)(sm + L::kVis);
    float* rowf = (float*)(sm + L::kRowF);
    int* ring_info = (int*)(sm + L::kMisc);                // [3]: live | bad << 16
    uint32_t* red_e = (uint32_t*)(sm + L::kMisc + 16);     // [2][8]: largest exponents of the unpacking warps
    uint32_t* tmem_slot = (uint32_t*)(sm + L::kMisc + 80);
    volatile int* abort_flag = (volatile int*)(sm + L::kMisc + 84);
    Start* start = (Start*)(sm + L::kMisc + 96);
    long long* scratch = (long long*)(sm + L::kMisc + 160);  // one per warp
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int group = a.H / a.Hkv;

    if (threadIdx.x == 0) {
        for (int i = 0; i < 3; i++) mbar_init(bar + kFull + i, 1), mbar_init(bar + kEmpty + i, 8);
        for (int i = 0; i < 2; i++) {
            mbar_init(bar + kKReady + i, 8);
            mbar_init(bar + kVReady + i, 8);
            mbar_init(bar + kSDone + i, 1);
            mbar_init(bar + kODone + i, 1);
            mbar_init(bar + kPReady + i, 8);
        }
        mbar_init(bar + kQReady, 8);
        mbar_init(bar + kOFree, 8);
        mbar_init(bar + kEnd, 1);
        *abort_flag = 0;
        mbar_fence_init();
    }
    if (warp == 16) tmem_alloc(tmem_slot, 512);
    for (int i = threadIdx.x; i < a.T; i += kTcThreads) {
        // the step rows that step row i sees (the mask, as bits)
        uint32_t m[4] = {1u, 0u, 0u, 0u};
        auto set = [&](int j) { m[0] |= j < 32 ? 1u << j : 0u, m[1] |= j >= 32 && j < 64 ? 1u << (j - 32) : 0u,
                                m[2] |= j >= 64 && j < 96 ? 1u << (j - 64) : 0u, m[3] |= j >= 96 ? 1u << (j - 96) : 0u; };
        const int nl = a.W * a.n1;
        if (i >= 1 && i <= nl) {
            const int lv = (i - 1) / a.W, c = (i - 1) % a.W;
            for (int j = 1; j <= 1 + c; j++) set(j);
            for (int v = 1; v <= lv; v++) set(1 + v * a.W + c);
        } else if (i > nl) {
            for (int j = i - (i - 1 - nl) % a.n1; j <= i; j++) set(j);
        }
        *(uint4*)(vis + 4 * i) = make_uint4(m[0], m[1], m[2], m[3]);
    }
    pdl_wait();
    pdl_trigger();
    if (blockIdx.x == 0) raise_long(a);
    tc_fence_before();
    find_starts(a, blockIdx.x, 1, start, scratch);
    tc_fence_after();
    const uint32_t tmem = *tmem_slot;
    const Start st = *start;
    MergeRec* rec = (MergeRec*)(a.part + (size_t)a.nteams * 2 * part_floats(kRowsTc, D)) + blockIdx.x;
    if (a.part && threadIdx.x == 0) rec->rest = 0;

    Run run;
    run.left = 0;
    // A wait that gives up ends every later one at once, but no role leaves its
    // loops: the named barriers keep their counts.
    bool ok = true;
    auto wait = [&](int b, int parity) {
        if (ok && !mbar_wait(bar + b, parity, abort_flag)) {
            ok = false;
            *abort_flag = 1;
            kv4_raise(a.status, LA_ERR_TIMEOUT);
        }
    };
    int n = 0;     // tiles so far: n & 1 is the buffer, (n >> 1) & 1 its phase
    int segs = 0;  // runs with tiles so far
    if (st.count > 0 && warp < 8) {
        // ------------------------------------------------------------ softmax
        const int q = warp & 3, half = warp >> 2, row = q * 32 + lane;
        const uint32_t trow = tmem + ((uint32_t)(q * 32) << 16);
        float* red = (float*)(sm + L::kRed);
        run.begin(a, st);
        do {
            const int head = run.item / a.mtiles, mt = run.item - head * a.mtiles;
            const int ntc = (run.len + kTile - 1) / kTile, gr = mt * kRowsTc + row;
            const bool any = mt * kRowsTc + q * 32 < a.rows;  // some row of this warp is there
            float m = kNoRef, l = 0.f;
            for (int tile = run.t0; tile < run.t1; tile++, n++) {
                const int b = n & 1, ph = (n >> 1) & 1;
                wait(kSDone + b, ph);
                tc_fence_after();
                if (any) {
                    const TileInfo* ti = info + (n & 3);
                    const int live = ti->live, bad = ti->bad, iev = ti->ev;
                    const float f = fmaxf(scale2(rowf[(segs & 1) * 128 + row], ti->ek), 1e-37f), ev = (float)iev;
                    const bool step = tile >= ntc;
                    uint2 see = make_uint2(~0u, ~0u);  // the columns of this half that count
                    if (step) {
                        see = *(const uint2*)(vis + 4 * min(gr / group, a.T - 1) + 2 * half);
                    } else if (live < kTile || bad) {
                        const int left = live - half * 64;
                        see.x = left >= 32 ? ~0u : left <= 0 ? 0u : (1u << left) - 1u;
                        see.y = left >= 64 ? ~0u : left <= 32 ? 0u : (1u << (left - 32)) - 1u;
                        const int hb = bad >> (half * 4);
                        see.x &= ~((hb & 1 ? 0xffffu : 0u) | (hb & 2 ? 0xffff0000u : 0u));
                        see.y &= ~((hb & 4 ? 0xffffu : 0u) | (hb & 8 ? 0xffff0000u : 0u));
                    }
                    const bool part = step || live < kTile || bad;
                    // 32 columns at a time, read again after the row's maximum is known
                    float x[32];
                    auto load = [&](int c) {
                        tmem_ld32(trow + b * 128 + half * 64 + c * 32, x);
                        if (part) {
                            const uint32_t s = c ? see.y : see.x;
#pragma unroll
                            for (int j = 0; j < 32; j++)
                                if (!((s >> j) & 1)) x[j] = -INFINITY;
                        }
                    };
                    float t0 = -INFINITY, t1 = -INFINITY;
#pragma unroll
                    for (int c = 0; c < 2; c++) {
                        load(c);
#pragma unroll
                        for (int j = 0; j < 32; j += 4) {
                            t0 = fmaxf(t0, fmaxf(x[j], x[j + 1]));
                            t1 = fmaxf(t1, fmaxf(x[j + 2], x[j + 3]));
                        }
                    }
                    red[(b * 2 + half) * 128 + row] = fmaxf(t0, t1);
                    named_sync(1 + q, 64);
                    const float y = fmaxf(red[b * 2 * 128 + row], red[(b * 2 + 1) * 128 + row]) * f + ev;
                    const bool up = y > m + 8.f;
                    if (__any_sync(0xffffffffu, up)) {
                        // the same rows, and so the same vote, in both halves
                        const float c = up ? ex2(m - y) : 1.f;
                        if (up) m = y;
                        l *= c;
                        if (tile > run.t0) {
                            wait(kODone + (b ^ 1), ((n - 1) >> 1) & 1);
                            tc_fence_after();
#pragma unroll
                            for (int j = 0; j < D / 2; j += 32) {
                                tmem_ld32(trow + 256 + half * (D / 2) + j, x);
#pragma unroll
                                for (int i = 0; i < 32; i++) x[i] *= c;
                                uint32_t y[32];
#pragma unroll
                                for (int i = 0; i < 32; i++) y[i] = __float_as_uint(x[i]);
                                tmem_st16(trow + 256 + half * (D / 2) + j, y);
                                tmem_st16(trow + 256 + half * (D / 2) + j + 16, y + 16);
                            }
                            tmem_st_wait();
                        }
                    }
                    const float c0 = ev - m;
                    float s0 = 0.f, s1 = 0.f;
#pragma unroll
                    for (int c = 0; c < 2; c++) {
                        load(c);
                        uint32_t p[16];
#pragma unroll
                        for (int j = 0; j < 32; j += 2) {
                            const float e0 = ex2(fmaf(x[j], f, c0)), e1 = ex2(fmaf(x[j + 1], f, c0));
                            s0 += e0, s1 += e1;
                            p[j / 2] = pack_f16(e0, e1);
                        }
                        tmem_st16(trow + b * 128 + half * 64 + c * 16, p);
                    }
                    l += scale2(s0 + s1, -iev);
                    tmem_st_wait();
                }
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(bar + kPReady + b);
            }
            // ---- the run's result
            const bool tiles = run.t1 > run.t0, whole = run.u0 == 0 && run.u1 == run.nu;
            if (tiles) {
                const int last = n - 1;
                wait(kODone + (last & 1), (last >> 1) & 1);
                tc_fence_after();
            }
            if (any) {
                red[(2 * (segs & 1) + half) * 128 + row] = l;  // free: its last readers have arrived at kPReady
                named_sync(1 + q, 64);
                const float sum = red[2 * (segs & 1) * 128 + row] + red[(2 * (segs & 1) + 1) * 128 + row];
                named_sync(1 + q, 64);
                float* part = a.part + ((size_t)blockIdx.x * 2 + (run.u0 == 0 ? 1 : 0)) * part_floats(kRowsTc, D);
                const float inv = 1.f / sum;
                const size_t orow = ((size_t)(run.b * (long long)a.T + gr / group) * a.H + head * group + gr % group) * D;
                // the step tile, if it is there, is the last one; its products are done, so its entry is complete
                const uint32_t* odd = info[(n - 1) & 3].odd;
                const bool fix = run.t1 > ntc && (odd[0] | odd[1] | odd[2] | odd[3]) != 0;
#pragma unroll
                for (int j = 0; j < D / 2; j += 32) {
                    float o[32];
                    __syncwarp();
                    if (tiles) {
                        tmem_ld32(trow + 256 + half * (D / 2) + j, o);
                    } else {
#pragma unroll
                        for (int i = 0; i < 32; i++) o[i] = 0.f;
                    }
                    const int c = half * (D / 2) + j;
                    if (fix && gr < a.rows) {
                        // values that are not finite, of the step rows this row sees
                        for (int key = 0; key < a.T; key++) {
                            if (!(((odd[key >> 5] & vis[4 * (gr / group) + (key >> 5)]) >> (key & 31)) & 1)) continue;
                            const __nv_bfloat16* v = a.vs + (size_t)(run.b * (long long)a.T + key) * a.kv_ld + (size_t)head * D + c;
#pragma unroll
                            for (int i = 0; i < 32; i++) {
                                const float x = __bfloat162float(v[i]);
                                if (!(fabsf(x) < INFINITY)) o[i] += x;
                            }
                        }
                    }
                    if (gr < a.rows && whole) {
#pragma unroll
                        for (int i = 0; i < 32; i += 8)
                            *(uint4*)(a.out + orow + c + i) =
                                make_uint4(pack_bf16(o[i] * inv, o[i + 1] * inv), pack_bf16(o[i + 2] * inv, o[i + 3] * inv),
                                           pack_bf16(o[i + 4] * inv, o[i + 5] * inv), pack_bf16(o[i + 6] * inv, o[i + 7] * inv));
                    } else if (gr < a.rows) {
#pragma unroll
                        for (int i = 0; i < 32; i += 4)
                            *(float4*)(part + (size_t)row * D + c + i) = make_float4(o[i], o[i + 1], o[i + 2], o[i + 3]);
                    }
                }
                if (!whole && half == 0 && gr < a.rows) *(float2*)(part + (size_t)kRowsTc * D + 2 * row) = make_float2(m, sum);
            }
            if (run.u0 == 0 && !whole && a.part && threadIdx.x == 0)
                *rec = MergeRec{run.b, run.item, run.nu - run.u1, 0, st.total};
            if (tiles) {
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(bar + kOFree);
                segs++;
            }
        } while (run.next(a));
    } else if (st.count > 0 && warp < 16) {
        // ------------------------------------------------------------- unpack
        const int tid = threadIdx.x - 256, row = tid >> 1, h = tid & 1, uw = warp - 8;
        int fills = 0;  // ring stages taken
        run.begin(a, st);
        do {
            const int head = run.item / a.mtiles, mt = run.item - head * a.mtiles;
            const int ntc = (run.len + kTile - 1) / kTile;
            if (run.t1 <= run.t0) continue;
            // ---- the rows' queries: row by a power of two, channels 32 h + 64 p .. of row `row`
            if (n > 0) wait(kSDone + ((n - 1) & 1), ((n - 1) >> 1) & 1);  // the last tile's S has read the old ones
            {
                const int gr = mt * kRowsTc + row;
                const __nv_bfloat16* src = a.q + (size_t)(run.b * (long long)a.T + gr / group) * a.q_ld +
                                           (size_t)(head * group + gr % group) * D + 32 * h;
                uint4 u[L::kAtoms][4];
                uint32_t top = 0;
#pragma unroll
                for (int p = 0; p < L::kAtoms; p++)
#pragma unroll
                    for (int i = 0; i < 4; i++) {
                        u[p][i] = gr < a.rows ? *(const uint4*)(src + 64 * p + 8 * i) : make_uint4(0, 0, 0, 0);
                        const uint32_t* w = (const uint32_t*)&u[p][i];
#pragma unroll
                        for (int k = 0; k < 4; k++) top = max(top, max((w[k] << 16) & 0x7f800000u, w[k] & 0x7f800000u));
                    }
                top = max(top, __shfl_xor_sync(0xffffffffu, top, 1));
                const int e = min(max((int)(top >> 23), 16), 236);
                const float down = pow2i(11 + 127 - e);  // the largest comes to [2^11, 2^12)
#pragma unroll
                for (int p = 0; p < L::kAtoms; p++)
#pragma unroll
                    for (int i = 0; i < 4; i++) {
                        const uint32_t* w = (const uint32_t*)&u[p][i];
                        uint32_t y[4];
#pragma unroll
                        for (int k = 0; k < 4; k++)
                            y[k] = pack_f16(__uint_as_float(w[k] << 16) * down, __uint_as_float(w[k] & 0xffff0000u) * down);
                        *(uint4*)(sm + L::kQ + p * (128 * 128) + row * 128 + (((4 * h + i) ^ (row & 7)) << 4)) = make_uint4(y[0], y[1], y[2], y[3]);
                    }
                if (h == 0) rowf[(segs & 1) * 128 + row] = pow2i(e - 127 - 11) * a.sl2;
                fence_proxy_async();
                __syncwarp();
                if (lane == 0) mbar_arrive(bar + kQReady);
                segs++;
            }
            for (int tile = run.t0; tile < run.t1; tile++, n++) {
                const int b = n & 1, ph = (n >> 1) & 1;
                uint8_t* kt = sm + L::kK + b * L::kOperand + row * 128;
                uint8_t* vt = sm + L::kV + b * L::kOperand + row * 128;
                TileInfo* ti = info + (n & 3);
                if (tile < ntc) {
                    const int s = fills % kRing;
                    wait(kFull + s, (fills / kRing) & 1);
                    const uint8_t* stage = sm + L::kCodes + s * L::kStage;
                    const int ri = ring_info[s], live = ri & 0xffff, bad = ri >> 16;
                    // the largest scales' exponents of the tile (of keys that count)
                    uint32_t ek = 0, ev = 0;
#pragma unroll
                    for (int i = 0; i < 4; i++) {
                        const int key = lane + 32 * i;
                        if (key < live && !((bad >> (key >> 4)) & 1)) {
                            const uint32_t* par = (const uint32_t*)(stage + (key >> 4) * kv4_block_bytes(D) + 16 * D) + (key & 15);
                            const uint32_t k0 = par[0] >> 23, v0 = par[16] >> 23;
                            ek = max(ek, k0 < 255 ? k0 : 0u);
                            ev = max(ev, v0 < 255 ? v0 : 0u);
                        }
                    }
                    ek = __reduce_max_sync(0xffffffffu, ek), ev = __reduce_max_sync(0xffffffffu, ev);
                    const int Ek = max((int)ek, 20) - 118, Ev = max((int)ev, 20) - 118;  // s 2^-E < 2^-8
                    const uint8_t* blk = stage + (row >> 4) * kv4_block_bytes(D);
                    const uint8_t* crow = blk + (row & 15) * 32 + h * 16;
                    const bool here = row < live && !((bad >> (row >> 4)) & 1);
                    auto factors = [&](uint32_t par, int E, __half2& lo, __half2& hi, __half2& off) {
                        const float sc = here ? scale2(__uint_as_float(par & 0xffff0000u), -E) : 0.f;
                        lo = __float2half2_rn(sc * 0x1p24f);
                        hi = __float2half2_rn(sc * 0x1p20f);
                        off = __float2half2_rn(-(float)(par & 15u) * sc);
                    };
                    const uint32_t* par = (const uint32_t*)(blk + 16 * D) + (row & 15);
                    __half2 lo, hi, off;
                    factors(par[0], Ek, lo, hi, off);
                    if (n >= 2) wait(kSDone + b, ph ^ 1);  // S of tile n - 2 has read this K
#pragma unroll
                    for (int p = 0; p < L::kAtoms; p++) {
                        const uint4 w = *(const uint4*)(crow + p * 512);
                        const uint32_t* u = (const uint32_t*)&w;
#pragma unroll
                        for (int i = 0; i < 4; i++)
                            *(uint4*)(kt + p * (128 * 128) + (((4 * h + i) ^ (row & 7)) << 4)) = unpack8(u[i], lo, hi, off);
                    }
                    if (tid == 0) ti->live = live, ti->bad = bad, ti->ek = Ek, ti->ev = Ev;
                    fence_proxy_async();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(bar + kKReady + b);
                    factors(par[16], Ev, lo, hi, off);
                    if (n >= 2) wait(kODone + b, ph ^ 1);  // O of tile n - 2 has read this V
#pragma unroll
                    for (int p = 0; p < L::kAtoms; p++) {
                        const uint4 w = *(const uint4*)(crow + 8 * D + p * 512);
                        const uint32_t* u = (const uint32_t*)&w;
#pragma unroll
                        for (int i = 0; i < 4; i++)
                            *(uint4*)(vt + p * (128 * 128) + (((4 * h + i) ^ (row & 7)) << 4)) = unpack8(u[i], lo, hi, off);
                    }
                    fence_proxy_async();
                    __syncwarp();
                    if (lane == 0) {
                        mbar_arrive(bar + kVReady + b);
                        mbar_arrive(bar + kEmpty + s);
                    }
                    fills++;
                } else {
                    // the step's own rows: bf16 to fp16 by the tile's largest finite exponent
                    const bool here = row < a.T;
                    const size_t at = (size_t)(run.b * (long long)a.T + row) * a.kv_ld + (size_t)head * D + 32 * h;
                    uint32_t e[2] = {0, 0};
#pragma unroll
                    for (int kv = 0; kv < 2; kv++) {
                        const __nv_bfloat16* src = (kv ? a.vs : a.ks) + at;
#pragma unroll
                        for (int p = 0; p < L::kAtoms; p++)
#pragma unroll
                            for (int i = 0; i < 4; i++) {
                                const uint4 u = here ? *(const uint4*)(src + 64 * p + 8 * i) : make_uint4(0, 0, 0, 0);
                                const uint32_t* w = (const uint32_t*)&u;
#pragma unroll
                                for (int k = 0; k < 4; k++) {
                                    const uint32_t x0 = (w[k] >> 7) & 255u, x1 = (w[k] >> 23) & 255u;
                                    e[kv] = max(e[kv], max(x0 < 255 ? x0 : 0u, x1 < 255 ? x1 : 0u));
                                }
                            }
                        e[kv] = __reduce_max_sync(0xffffffffu, e[kv]);
                        if (lane == 0) red_e[kv * 8 + uw] = e[kv];
                    }
                    if (tid < 4) ti->odd[tid] = 0;
                    named_sync(5, 256);
#pragma unroll
                    for (int kv = 0; kv < 2; kv++)
#pragma unroll
                        for (int i = 0; i < 8; i++) e[kv] = max(e[kv], red_e[kv * 8 + i]);
                    named_sync(5, 256);  // red_e may be written again
                    const int E[2] = {max((int)e[0], 28) - 135, max((int)e[1], 28) - 135};  // the largest comes to [2^8, 2^9)
                    if (tid == 0) ti->live = kTile, ti->bad = 0, ti->ek = E[0], ti->ev = E[1];
#pragma unroll
                    for (int kv = 0; kv < 2; kv++) {
                        if (n >= 2) wait((kv ? kODone : kSDone) + b, ph ^ 1);
                        const __nv_bfloat16* src = (kv ? a.vs : a.ks) + at;
                        const float f = pow2i(-E[kv]);
                        bool odd = false;
#pragma unroll
                        for (int p = 0; p < L::kAtoms; p++)
#pragma unroll
                            for (int i = 0; i < 4; i++) {
                                const uint4 u = here ? *(const uint4*)(src + 64 * p + 8 * i) : make_uint4(0, 0, 0, 0);
                                const uint32_t* w = (const uint32_t*)&u;
                                uint32_t y[4];
#pragma unroll
                                for (int k = 0; k < 4; k++) {
                                    float x0 = __uint_as_float(w[k] << 16), x1 = __uint_as_float(w[k] & 0xffff0000u);
                                    if (kv) {
                                        // zero times these is NaN: the product runs without them (TileInfo::odd)
                                        if (!(fabsf(x0) < INFINITY)) odd = true, x0 = 0.f;
                                        if (!(fabsf(x1) < INFINITY)) odd = true, x1 = 0.f;
                                    }
                                    y[k] = pack_f16(x0 * f, x1 * f);
                                }
                                *(uint4*)((kv ? vt : kt) + p * (128 * 128) + (((4 * h + i) ^ (row & 7)) << 4)) =
                                    make_uint4(y[0], y[1], y[2], y[3]);
                            }
                        if (odd) atomicOr(&ti->odd[row >> 5], 1u << (row & 31));
                        fence_proxy_async();
                        __syncwarp();
                        if (lane == 0) mbar_arrive(bar + (kv ? kVReady : kKReady) + b);
                    }
                }
            }
        } while (run.next(a));
    } else if (st.count > 0 && warp == 16) {
        // ---------------------------------------------------------------- MMA
        if (lane == 0) {
            constexpr uint32_t id_s = idesc_f16(128, kTile, false), id_o = idesc_f16(128, D, true);
            auto scores = [&](bool first) {
                const int b = n & 1;
                wait(kKReady + b, (n >> 1) & 1);
                if (first) wait(kQReady, segs & 1);
                if (!ok) return;
                tc_fence_after();
#pragma unroll
                for (int k = 0; k < D / 16; k++) {
                    const uint32_t qa = smem_u32(sm + L::kQ + (k >> 2) * (128 * 128)) + (k & 3) * 32;
                    const uint32_t ka = smem_u32(sm + L::kK + b * L::kOperand + (k >> 2) * (128 * 128)) + (k & 3) * 32;
                    mma_bf16(tmem + b * 128, desc_sw128_kmajor(qa), desc_sw128_kmajor(ka), id_s, k > 0);
                }
                mma_commit(bar + kSDone + b);
            };
            auto outputs = [&](int i, bool first) {  // tile i
                const int b = i & 1, ph = (i >> 1) & 1;
                wait(kPReady + b, ph);
                wait(kVReady + b, ph);
                if (first && segs > 0) wait(kOFree, (segs - 1) & 1);
                if (!ok) return;
                tc_fence_after();
#pragma unroll
                for (int k = 0; k < kTile / 16; k++) {
                    const uint32_t va = smem_u32(sm + L::kV + b * L::kOperand) + k * 16 * 128;
                    mma_ts(tmem + 256, tmem + b * 128 + (k >> 2) * 64 + (k & 3) * 8, desc_sw128_mnmajor(va, 128 * 128), id_o,
                           !first || k > 0);
                }
                mma_commit(bar + kODone + b);
            };
            run.begin(a, st);
            do {
                if (run.t1 <= run.t0) continue;
                scores(true);
                for (int tile = run.t0; tile < run.t1; tile++) {
                    const int i = n++;
                    if (tile + 1 < run.t1) scores(false);  // of the next tile, while this one's softmax runs
                    outputs(i, tile == run.t0);
                }
                segs++;
            } while (run.next(a));
            if (!ok) {
                // let the products that were issued finish before the memory goes
                mma_commit(bar + kEnd);
                mbar_drain(bar + kEnd, 0);
            }
        }
        __syncwarp();
    } else if (st.count > 0) {
        // -------------------------------------------------------------- copies
        const uint64_t pol = policy_evict_first();
        int fills = 0;
        run.begin(a, st);
        do {
            const int head = run.item / a.mtiles, ntc = (run.len + kTile - 1) / kTile;
            for (int tile = run.t0; tile < min(run.t1, ntc); tile++) {
                const int s = fills % kRing, blk = tile * 8 + lane, live = min(run.len - tile * kTile, kTile);
                const bool mine = lane < 8 && lane * 16 < live;
                const int page = mine ? __ldg(a.table + (size_t)run.b * a.max_pages + (blk >> a.blk_log2)) : 0;
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
        } while (run.next(a));
        // no copy may still be on its way when the CTA ends
        for (int i = 1; i <= kRing && i <= fills; i++) mbar_drain(bar + kFull + (fills - i) % kRing, ((fills - i) / kRing) & 1);
    }
    __syncwarp();
    tc_fence_before();
    __syncthreads();
    if (warp == 16) {
        tc_fence_after();
        tmem_dealloc(tmem, 512);
    }
}

struct TcPlan {
    int nteams, mtiles;
    bool merge;
    size_t bytes;
};

constexpr int kTcExtra = 2;

TcPlan tc_plan(const la_kv4_desc& c, const la_kv4_attn& a)
{
    TcPlan p;
    const int T = 1 + (a.W + a.G) * (a.N - 1), rows = T * (a.n_heads / c.n_kv_heads);
    p.mtiles = ceil_div(rows, kRowsTc);
    const long long items = (long long)a.batch * c.n_kv_heads * p.mtiles;
    const int room = c.max_pages * c.page, max_len = a.max_len > 0 && a.max_len < room ? a.max_len : room;
    const long long units = items * (kTcExtra + (max_len + kTile - 1) / kTile + 1);
    p.nteams = (int)std::max(1LL, std::min((long long)kSMs, std::max(items, units / (kTcExtra + 2))));
    p.merge = !(a.batch == 1 && items % p.nteams == 0);
    p.bytes = p.merge ? (size_t)p.nteams * (2 * part_floats(kRowsTc, c.head_dim) * 4 + sizeof(MergeRec)) : 0;
    return p;
}

}  // namespace

size_t kv4_tc_bytes(const la_kv4_desc& c, const la_kv4_attn& a) { return tc_plan(c, a).bytes; }

bool kv4_tc_init()
{
    return cudaFuncSetAttribute(k_kv4_tc<128>, cudaFuncAttributeMaxDynamicSharedMemorySize, TcSmem<128>::kBytes) == cudaSuccess &&
           cudaFuncSetAttribute(k_kv4_tc<64>, cudaFuncAttributeMaxDynamicSharedMemorySize, TcSmem<64>::kBytes) == cudaSuccess;
}

int launch_kv4_tc(cudaStream_t s, const la_kv4_desc& c, const la_kv4_attn& a, Kv4Attn k)
{
    const TcPlan p = tc_plan(c, a);
    k.mtiles = p.mtiles, k.nteams = p.nteams, k.extra = kTcExtra;
    k.tile_log2 = kTileLog2, k.step_tiles = 1;
    k.part = p.merge ? (float*)a.workspace : nullptr;
    cudaError_t e = c.head_dim == 128
                        ? launch_pdl(k_kv4_tc<128>, dim3(p.nteams), dim3(kTcThreads), TcSmem<128>::kBytes, s, k)
                        : launch_pdl(k_kv4_tc<64>, dim3(p.nteams), dim3(kTcThreads), TcSmem<64>::kBytes, s, k);
    if (e == cudaSuccess && p.merge) e = launch_kv4_merge(s, k, c.head_dim, kRowsTc);
    return e == cudaSuccess ? LA_OK : LA_ERR_CUDA;
}

}  // namespace la
