// kv16_rows.cuh -- the step's masked attention over the paged bf16 cache for at
// most 16 rows per KV head: single tokens, small lookahead steps, few heads.  A
// kernel of its own (kv16_rows.cu), or some CTAs of the kernel that takes the
// prefixes of such sequences (kv16_wide.cu).
//
// A warp is a team: it streams its run of 16-key blocks through a ring of its
// own in shared memory and waits for no other.  m16n8k16 has the rows as its
// 16-row side and 8 keys (S = Q K^T) or 8 channels (O += P V) as the other, so
// P goes from one product's accumulators to the other's operand as it stands.
// cp.async fills the ring 16 bytes a lane, so that a block's missing keys are
// not read but filled with zeros (whatever a page holds there), and in a
// swizzle that keeps ldmatrix free of bank conflicts.  Feeding runs ahead of
// the products by the ring's stages, over the ends of items.
//
// P = exp2((S - M) f) in bf16, S, M, the sums and O in fp32.  The reference M is
// the row's largest score of the run's first block and moves, to the largest so
// far, only when a row's P of a block sum to more than 2^15: a vote per block, no
// reduction.
//
// HBM bound: 4 D bytes a key and KV head, 32 products a block.  By itself a CTA of 8
// teams a SM (243 registers: queries and outputs stay in them): 128 single tokens of
// 32 heads over 31 to 256 keys (300 MB) 58 us, 5.2 TB/s; 64 of 8 KV heads over 2 to 9 K
// 220 us, 6.5 TB/s (with 12 teams 60 and 235).  Two stages of 8 KB a team: with three
// the former, behind 1000 shared keys, took 78 us, not 71.  Beside prefixes 12 teams a
// SM, of the 168 registers that k_kv16_wide leaves a thread: the same behind 1000
// shared keys 64.5 us in all (with 8 of its 12 warps as teams 72.7).
#pragma once
#include "kv16_sched.cuh"

namespace la {
namespace {

template <int D, int kWarps>
struct RowsSmem {
    static constexpr int kSide = 16 * D * 2;               // a block's keys, or its values
    static constexpr int kStages = D == 128 ? 2 : 4;
    static constexpr int kRing = kWarps * kStages * 2 * kSide;
    static constexpr int kInfo = kRing;                    // of each stage: keys | step << 8
    static constexpr int kMisc = kInfo + kWarps * kStages * 4;
    static constexpr int kScan = (kMisc + 7) / 8 * 8, kStarts = kScan + (int)sizeof(Scan), kPre = kStarts + kWarps * (int)sizeof(Start);
    static constexpr int kBytes = kPre + (int)sizeof(PreShared);
    static_assert(kBytes <= 227 * 1024, "shared memory");
    static __device__ __forceinline__ Scan* scan(uint8_t* sm) { return (Scan*)(sm + kScan); }
    static __device__ __forceinline__ Start* starts(uint8_t* sm) { return (Start*)(sm + kStarts); }
    static __device__ __forceinline__ PreShared* pre(uint8_t* sm) { return (PreShared*)(sm + kPre); }
};

__device__ __forceinline__ void mma(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1)
{
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
                 : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
                 : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
__device__ __forceinline__ void ldsm4(uint32_t (&r)[4], uint32_t addr)
{
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(addr)
                 : "memory");
}
__device__ __forceinline__ void ldsm4_t(uint32_t (&r)[4], uint32_t addr)
{
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(addr)
                 : "memory");
}
// 16 bytes, or zeros (then nothing is read)
__device__ __forceinline__ void cp16(uint32_t dst, const void* src, bool there, uint64_t pol)
{
    asm volatile("cp.async.cg.shared.global.L2::cache_hint [%0], [%1], 16, %2, %3;" ::"r"(dst), "l"(src), "r"(there ? 16 : 0), "l"(pol) : "memory");
}
__device__ __forceinline__ void cp_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_wait()
{
    asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}
__device__ __forceinline__ void prefetch_l1(const void* p) { asm volatile("prefetch.global.L1 [%0];" ::"l"(p)); }

// of a bf16 pair (weights are summed as rounded: what one loses is then lost above and below)
__device__ __forceinline__ float sum_of(uint32_t u) { return __uint_as_float(u << 16) + __uint_as_float(u & 0xffff0000u); }

__device__ __forceinline__ bool odd(float x) { return !(fabsf(x) < INFINITY); }

// What a warp does, its run known; sm is the CTA's shared memory.
template <int D, int kWarps>
__device__ __forceinline__ void rows_team(const Kv16Attn& a, const Kv16Sched& s, uint8_t* sm, const Prefixes& pre, const Shares& sh, const Start& st)
{
    using L = RowsSmem<D, kWarps>;
    constexpr int kPieces = D / 8, kRowsPass = 32 / kPieces;  // 16-byte pieces of a row; rows of a warp's copy instruction
    constexpr int kSteps = D / 16;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, gid = lane >> 2, tig = lane & 3, team = st.team;
    if (st.count <= 0) return;
    const uint32_t ring = smem_u32(sm) + warp * (L::kStages * 2 * L::kSide);
    int* info = (int*)(sm + L::kInfo) + warp * L::kStages;

    // ---- feeding
    Run<RowsKind> f;
    f.begin(a, s, pre, st, sh);
    Run<RowsKind> c = f;
    bool feeding = true;
    const int pc = lane % kPieces, r0 = lane / kPieces;
    // what is read once goes from L2 first: tables, parts and code stay
    const uint64_t once = policy_evict_first(), shared = policy_evict_normal();
    int fk = f.t0, stage_in = 0, window = -1, page_of = 0;
    auto start_feed = [&]() {
        fk = f.t0;
        if (lane < a.R && f.t1 > f.t0) {
            const int gr = f.x.row0 + lane;
            const __nv_bfloat16* src = a.q + (size_t)(gr / a.group) * a.q_ld + (size_t)(f.item * a.group + gr % a.group) * D;
            prefetch_l1(src);
            if (D == 128) prefetch_l1(src + 64);
        }
    };
    start_feed();
    auto feed = [&]() {
        while (feeding && fk >= f.t1) {
            const int e = f.e;
            feeding = f.next(a, s, pre);
            if (!feeding) break;
            if (f.e != e) window = -1;
            start_feed();
        }
        if (feeding) {
            const int nc = f.x.nb_cached(), g = f.item;
            const __nv_bfloat16 *k, *v;
            int live;
            uint64_t pol = once;
            size_t k_row = D, v_row = D;
            if (fk < nc) {
                // the pages of 32 table entries at a time, one a lane
                const bool own = fk >= f.x.nb_pre;
                pol = own ? once : shared;
                const int tok = (own ? fk - f.x.nb_pre : fk) * 16, n = own ? f.x.len : f.x.plen, at = tok >> a.page_log2;
                const int w = (at >> 5) * 2 + own;
                if (w != window) {
                    window = w;
                    const int* row = own ? a.table + (size_t)f.x.b * a.max_pages : a.ptable + (size_t)f.x.p * a.pp;
                    const int i = (at & ~31) + lane;
                    page_of = (long long)i << a.page_log2 < n ? row[i] : 0;
                }
                const int page = __shfl_sync(0xffffffffu, page_of, at & 31);
                const bool bad = (unsigned)page >= (unsigned)a.n_pages;
                if (bad && lane == 0) kv4_raise(a.status, LA_ERR_ARG);
                live = bad ? 0 : min(16, n - tok);
                const size_t row = (((size_t)(bad ? 0 : page) * a.Hkv + g) << a.page_log2) + (tok & ((1 << a.page_log2) - 1));
                k = a.kp + row * D, v = a.vp + row * D;
                if (lane == 0) info[stage_in] = live;
            } else {
                live = a.T;
                const size_t row = (size_t)f.x.b * a.T;
                k = a.ks + row * a.k_ld + (size_t)g * D, v = a.vs + row * a.v_ld + (size_t)g * D;
                k_row = a.k_ld, v_row = a.v_ld;
                if (lane == 0) info[stage_in] = live | 256;
            }
            const uint32_t dst = ring + stage_in * (2 * L::kSide) + r0 * (D * 2);
            const char *k8 = (const char*)(k + r0 * k_row + pc * 8), *v8 = (const char*)(v + r0 * v_row + pc * 8);
            const size_t k_step = k_row * (2 * kRowsPass), v_step = v_row * (2 * kRowsPass);
#pragma unroll
            for (int i = 0; i < 16 / kRowsPass; i++) {
                const bool there = r0 + i * kRowsPass < live;
                const uint32_t at = dst + i * (kRowsPass * D * 2) + ((pc ^ ((r0 + i * kRowsPass) & 7)) << 4);
                cp16(at, there ? k8 + i * k_step : (const char*)a.kp, there, pol);
                cp16(at + L::kSide, there ? v8 + i * v_step : (const char*)a.kp, there, pol);
            }
            fk++;
        }
        cp_commit();
        if (++stage_in == L::kStages) stage_in = 0;
    };
#pragma unroll 1
    for (int i = 0; i < L::kStages; i++) feed();

    // ---- this lane's rows, and the step rows they see (the same in every item)
    const int ra = gid, rb = gid + 8;
    const bool two = a.R > 8;
    uint32_t see_a = 0, see_b = 0;
    for (int j = 0; j < a.T; j++) {
        see_a |= (kv4_sees(min(ra / a.group, a.T - 1), j, a.W, a.n1) ? 1u : 0u) << j;
        see_b |= (kv4_sees(min(rb / a.group, a.T - 1), j, a.W, a.n1) ? 1u : 0u) << j;
    }
    // fragment addresses within a stage
    const int krow = (lane & 7) + (lane >= 16 ? 8 : 0), kpc = (lane >> 3) & 1;
    const int vrow = (lane & 7) + (lane & 8), vpc = lane >> 4;
    const uint32_t k_at = krow * (D * 2), v_at = L::kSide + vrow * (D * 2);
    int stage = 0;
    do {
        if (c.t1 <= c.t0) {
            // (units, but no keys)
            if (c.x.nu && lane == 0) c.note(a, s, pre, sh, team);
            if (c.x.nu && lane < a.R)
                *(float2*)(s.slots + ((size_t)team * 2 + c.slot()) * rows_part(D, a.R) + (size_t)a.R * D + 2 * lane) = make_float2(kNoRef, 0.f);
            continue;
        }
        const int g = c.item;
        uint32_t q[kSteps][4];
        {
            auto row_of = [&](int r) {
                const int gr = c.x.row0 + r;
                return a.q + (size_t)(gr / a.group) * a.q_ld + (size_t)(g * a.group + gr % a.group) * D + 2 * tig;
            };
            const __nv_bfloat16 *qa = row_of(min(ra, a.R - 1)), *qb = row_of(min(rb, a.R - 1));
            const bool ha = ra < a.R, hb = rb < a.R;
#pragma unroll
            for (int k = 0; k < kSteps; k++) {
                q[k][0] = ha ? *(const uint32_t*)(qa + 16 * k) : 0u;
                q[k][2] = ha ? *(const uint32_t*)(qa + 16 * k + 8) : 0u;
                q[k][1] = hb ? *(const uint32_t*)(qb + 16 * k) : 0u;
                q[k][3] = hb ? *(const uint32_t*)(qb + 16 * k + 8) : 0u;
            }
        }
        float o[D / 8][4];
#pragma unroll
        for (int i = 0; i < D / 8; i++)
#pragma unroll
            for (int j = 0; j < 4; j++) o[i][j] = 0.f;
        float ma = kNoRef, mb = kNoRef, la = 0.f, lb = 0.f;
#pragma unroll 1
        for (int t = c.t0; t < c.t1; t++) {
            cp_wait<L::kStages - 1>();
            __syncwarp();
            const int what = info[stage], live = what & 255;
            const bool step = what >= 256;
            const uint32_t base = ring + stage * (2 * L::kSide);
            bool found = false;
            if (step && a.T > 1) {
                // values that are not finite reach only the rows that see them: not through the product
                uint8_t* side = sm + warp * (L::kStages * 2 * L::kSide) + stage * (2 * L::kSide) + L::kSide;
                for (int i = lane; i < L::kSide / 16; i += 32) {
                    uint4 u = *(uint4*)(side + i * 16);
                    uint32_t w[4] = {u.x, u.y, u.z, u.w};
                    bool here = false;
#pragma unroll
                    for (int j = 0; j < 4; j++) {
                        const bool lo = (w[j] & 0x7f80u) == 0x7f80u, hi = (w[j] & 0x7f800000u) == 0x7f800000u;
                        if (lo) w[j] &= 0xffff0000u;
                        if (hi) w[j] &= 0x0000ffffu;
                        here |= lo || hi;
                    }
                    if (here) *(uint4*)(side + i * 16) = make_uint4(w[0], w[1], w[2], w[3]);
                    found |= here;
                }
                found = __any_sync(0xffffffffu, found);
                __syncwarp();
            }
            // S: keys 0-7 and 8-15, even and odd steps apart for shorter chains
            float x[2][4], y[2][4];
#pragma unroll
            for (int i = 0; i < 2; i++)
#pragma unroll
                for (int j = 0; j < 4; j++) x[i][j] = y[i][j] = 0.f;
#pragma unroll
            for (int k = 0; k < kSteps; k += 2) {
                uint32_t r[4], u[4];
                ldsm4(r, base + k_at + (((2 * k + kpc) ^ (krow & 7)) << 4));
                ldsm4(u, base + k_at + (((2 * k + 2 + kpc) ^ (krow & 7)) << 4));
                mma(x[0], q[k], r[0], r[1]);
                mma(x[1], q[k], r[2], r[3]);
                mma(y[0], q[k + 1], u[0], u[1]);
                mma(y[1], q[k + 1], u[2], u[3]);
            }
#pragma unroll
            for (int i = 0; i < 2; i++)
#pragma unroll
                for (int j = 0; j < 4; j++) x[i][j] += y[i][j];
            if (live < 16 || step) {
                const uint32_t all = (1u << live) - 1u, see[2] = {step ? see_a : all, step ? see_b : all};
#pragma unroll
                for (int i = 0; i < 2; i++)
#pragma unroll
                    for (int j = 0; j < 4; j++)
                        if (!((see[j >> 1] >> (8 * i + 2 * tig + (j & 1))) & 1)) x[i][j] = -INFINITY;
            }
            uint32_t p[4] = {0, 0, 0, 0};
            float sa, sb = 0.f;
            bool look = t == c.t0;
            while (true) {
                if (look) {
                    float ya = fmaxf(fmaxf(x[0][0], x[0][1]), fmaxf(x[1][0], x[1][1]));
                    float yb = fmaxf(fmaxf(x[0][2], x[0][3]), fmaxf(x[1][2], x[1][3]));
                    ya = fmaxf(ya, __shfl_xor_sync(0xffffffffu, ya, 1)), yb = fmaxf(yb, __shfl_xor_sync(0xffffffffu, yb, 1));
                    ya = fmaxf(ya, __shfl_xor_sync(0xffffffffu, ya, 2)), yb = fmaxf(yb, __shfl_xor_sync(0xffffffffu, yb, 2));
                    const float na = fmaxf(ma, ya), nb = fmaxf(mb, yb);
                    const float fa = ex2((ma - na) * a.sl2), fb = ex2((mb - nb) * a.sl2);
                    ma = na, mb = nb, la *= fa, lb *= fb;
#pragma unroll
                    for (int i = 0; i < D / 8; i++) o[i][0] *= fa, o[i][1] *= fa, o[i][2] *= fb, o[i][3] *= fb;
                }
                const float e0 = ex2((x[0][0] - ma) * a.sl2), e1 = ex2((x[0][1] - ma) * a.sl2),
                            e2 = ex2((x[1][0] - ma) * a.sl2), e3 = ex2((x[1][1] - ma) * a.sl2);
                p[0] = pack_bf16(e0, e1), p[2] = pack_bf16(e2, e3);
                sa = sum_of(p[0]) + sum_of(p[2]);
                if (two) {
                    const float g0 = ex2((x[0][2] - mb) * a.sl2), g1 = ex2((x[0][3] - mb) * a.sl2),
                                g2 = ex2((x[1][2] - mb) * a.sl2), g3 = ex2((x[1][3] - mb) * a.sl2);
                    p[1] = pack_bf16(g0, g1), p[3] = pack_bf16(g2, g3);
                    sb = sum_of(p[1]) + sum_of(p[3]);
                }
                if (look || !__any_sync(0xffffffffu, sa > 32768.f || sb > 32768.f)) break;
                look = true;
            }
            la += sa, lb += sb;
#pragma unroll
            for (int n = 0; n < D / 16; n++) {
                uint32_t r[4];
                ldsm4_t(r, base + v_at + (((2 * n + vpc) ^ (vrow & 7)) << 4));
                mma(o[2 * n], p, r[0], r[1]);
                mma(o[2 * n + 1], p, r[2], r[3]);
            }
            if (found) {
#pragma unroll 1
                for (int j = 0; j < a.T; j++) {
                    const __nv_bfloat16* v = a.vs + ((size_t)c.x.b * a.T + j) * a.v_ld + (size_t)g * D + 2 * tig;
                    const bool za = (see_a >> j) & 1, zb = (see_b >> j) & 1;
#pragma unroll
                    for (int i = 0; i < D / 8; i++) {
                        const float v0 = __bfloat162float(v[8 * i]), v1 = __bfloat162float(v[8 * i + 1]);
                        if (odd(v0)) o[i][0] += za ? v0 : 0.f, o[i][2] += zb ? v0 : 0.f;
                        if (odd(v1)) o[i][1] += za ? v1 : 0.f, o[i][3] += zb ? v1 : 0.f;
                    }
                }
            }
            if (++stage == L::kStages) stage = 0;
            __syncwarp();
            feed();
        }
        // ---- the run's result
        la += __shfl_xor_sync(0xffffffffu, la, 1), lb += __shfl_xor_sync(0xffffffffu, lb, 1);
        la += __shfl_xor_sync(0xffffffffu, la, 2), lb += __shfl_xor_sync(0xffffffffu, lb, 2);
        const bool all = c.all();
        if (lane == 0) c.note(a, s, pre, sh, team);
#pragma unroll
        for (int half = 0; half < 2; half++) {
            const int r = half ? rb : ra;
            const float m = half ? mb : ma, l = half ? lb : la;
            if (r >= a.R) continue;
            if (all && s.finish) {
                const float inv = 1.f / l;
                const int gr = c.x.row0 + r;
                __nv_bfloat16* dst = a.out + ((size_t)(gr / a.group) * a.H + (size_t)g * a.group + gr % a.group) * D + 2 * tig;
#pragma unroll
                for (int i = 0; i < D / 8; i++)
                    *(uint32_t*)(dst + 8 * i) = pack_bf16(o[i][2 * half] * inv, o[i][2 * half + 1] * inv);
            } else {
                // by row: [rows][D], then [rows][M, sum]
                const size_t rows = all ? (size_t)a.B * a.R * a.Hkv : a.R;
                const size_t at = all ? (size_t)g * a.B * a.R + c.x.row0 + r : r;
                float* part = all ? s.whole : s.slots + ((size_t)team * 2 + c.slot()) * rows_part(D, a.R);
                float* dst = part + at * D + 2 * tig;
#pragma unroll
                for (int i = 0; i < D / 8; i++) *(float2*)(dst + 8 * i) = make_float2(o[i][2 * half], o[i][2 * half + 1]);
                if (tig == 0) *(float2*)(part + rows * D + 2 * at) = make_float2(m, l);
            }
        }
    } while (c.next(a, s, pre));
    cp_wait<0>();
}

}  // namespace
}  // namespace la
