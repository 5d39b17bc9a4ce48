// kv4_sched.cuh -- how the attention kernels over the 4-bit cache share their
// work: items (sequence, KV head, row tile) are laid end to end in units of a
// tile and cut into equal runs, one per team; and small helpers of both.
#pragma once
#include <cuda_fp16.h>

#include "kv4.cuh"

namespace la {
namespace {

using namespace ptx;

constexpr int kSMs = 152;
constexpr float kNoRef = -3e38f;  // below every score: exp2(-inf - kNoRef) = 0
constexpr uint32_t kLo = 0x000f000fu, kHi = 0x00f000f0u;  // a pair of codes as fp16: c 2^-24, c 2^-20

__device__ __forceinline__ void bulk_load(void* dst, const void* src, uint32_t bytes, uint64_t* bar, uint64_t pol)
{
    asm volatile(
        "cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes.L2::cache_hint [%0], [%1], %2, [%3], %4;" ::"r"(
            smem_u32(dst)),
        "l"(src), "r"(bytes), "r"(smem_u32(bar)), "l"(pol)
        : "memory");
}

__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi)
{
    __nv_bfloat162 v = __floats2bfloat162_rn(lo, hi);
    return *reinterpret_cast<uint32_t*>(&v);
}

__device__ __forceinline__ uint32_t pack_f16(float lo, float hi)
{
    __half2 v = __floats2half2_rn(lo, hi);
    return *reinterpret_cast<uint32_t*>(&v);
}

__device__ __forceinline__ uint32_t cluster_rank()
{
    uint32_t r;
    asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
    return r;
}
__device__ __forceinline__ uint32_t cluster_size()
{
    uint32_t r;
    asm volatile("mov.u32 %0, %%cluster_nctarank;" : "=r"(r));
    return r;
}
__device__ __forceinline__ void cluster_sync()
{
    asm volatile("barrier.cluster.arrive.aligned;\n barrier.cluster.wait.aligned;" ::: "memory");
}
// the address of p in the shared memory of CTA `rank` of the cluster
__device__ __forceinline__ uint32_t peer(const void* p, uint32_t rank)
{
    uint32_t a;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(a) : "r"(smem_u32(p)), "r"(rank));
    return a;
}
__device__ __forceinline__ float2 ld_peer2(uint32_t addr)
{
    float2 v;
    asm volatile("ld.shared::cluster.v2.f32 {%0, %1}, [%2];" : "=f"(v.x), "=f"(v.y) : "r"(addr) : "memory");
    return v;
}
__device__ __forceinline__ float4 ld_peer4(uint32_t addr)
{
    float4 v;
    asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];" : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w) : "r"(addr) : "memory");
    return v;
}

// `items` clusters of `size` CTAs, as launch_pdl otherwise.
inline cudaError_t launch_cluster(void (*kern)(Kv4Attn), unsigned items, unsigned size, int threads, size_t smem, cudaStream_t s,
                                  const Kv4Attn& k)
{
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(items * size);
    cfg.blockDim = dim3(threads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = s;
    cudaLaunchAttribute at[2];
    at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[0].val.programmaticStreamSerializationAllowed = 1;
    at[1].id = cudaLaunchAttributeClusterDimension;
    at[1].val.clusterDim.x = size, at[1].val.clusterDim.y = 1, at[1].val.clusterDim.z = 1;
    cfg.attrs = at;
    cfg.numAttrs = 2;
    return cudaLaunchKernelEx(&cfg, kern, k);
}

// ------------------------------------------------------------ the schedule ---

__device__ __forceinline__ int seq_len(const Kv4Attn& a, int b)
{
    const int len = a.lens[b];
    return len > a.max_len ? -1 : len;  // too long: raised by raise_long(), left alone everywhere
}

// An item's work in units of a tile: `extra` units for its queries and its
// result, its cached tiles, its step rows' tile.
__device__ __forceinline__ int item_units(const Kv4Attn& a, int len)
{
    return len < 0 ? 0 : a.extra + ((len + (1 << a.tile_log2) - 1) >> a.tile_log2) + 1;
}

// Sequences whose length is over its bound (one CTA calls it).
__device__ __forceinline__ void raise_long(const Kv4Attn& a)
{
    for (int b = threadIdx.x; b < a.B; b += blockDim.x)
        if (a.lens[b] > a.max_len) kv4_raise(a.status, LA_ERR_ARG);
}

// The equal runs: team t begins at unit q t + min(t, r) of all items' units
// (q, r: their number divided by the teams').
struct Shares {
    long long q;
    int r, pad;
    __device__ __forceinline__ long long at(int t) const { return q * t + min(t, r); }
};

__device__ __noinline__ long long div_long(long long a, int b) { return a / b; }

__device__ __forceinline__ Shares shares_of(long long total, int teams)
{
    // (a 64-bit division takes half a microsecond)
    if (total < (1LL << 31)) {
        const uint32_t q = (uint32_t)total / (uint32_t)teams;
        return Shares{q, (int)((uint32_t)total - q * (uint32_t)teams), 0};
    }
    const long long q = div_long(total, teams);
    return Shares{q, (int)(total - q * teams), 0};
}

struct Start {
    int b;
    long long off, count;  // offset in the units of sequence b's items; units of the team
    Shares sh;
};

// Where each of the CTA's teams begins: teams t0 .. t0 + n - 1 of a.nteams
// take equal runs of all items' units in (sequence, item) order.
__device__ void find_starts(const Kv4Attn& a, int t0, int n, Start* starts, long long* scratch)
{
    const int items = a.Hkv * a.mtiles, per = ceil_div(a.B, (int)blockDim.x), b0 = threadIdx.x * per;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, nw = blockDim.x >> 5;
    long long mine = 0;
    for (int b = b0; b < min(b0 + per, a.B); b++) mine += (long long)items * item_units(a, seq_len(a, b));
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
        const Shares sh = shares_of(total, a.nteams);
        for (int i = 0; i < n; i++) {
            const long long u0 = sh.at(t0 + i), u1 = t0 + i < a.nteams ? sh.at(t0 + i + 1) : u0;
            if (u0 >= u1 || u0 < before || u0 >= before + mine) continue;
            long long at = before;
            for (int b = b0; b < min(b0 + per, a.B); b++) {
                const long long c = (long long)items * item_units(a, seq_len(a, b));
                if (u0 < at + c) {
                    starts[i] = Start{b, u0 - at, u1 - u0, sh};
                    break;
                }
                at += c;
            }
        }
    }
    __syncthreads();
}

// The run of units of one item that a team works on, and its tiles t0 .. t1 - 1.
struct Run {
    int b, item, len, nu, u0, u1, t0, t1;
    long long left;
    __device__ __forceinline__ void cut(const Kv4Attn& a, int from)
    {
        u0 = from;
        u1 = (int)min((long long)nu, u0 + left);
        left -= u1 - u0;
        t0 = max(u0 - a.extra, 0);
        t1 = max(u1 - a.extra, 0);
    }
    __device__ __forceinline__ void begin(const Kv4Attn& a, const Start& s)
    {
        left = s.count;
        b = s.b;
        len = seq_len(a, b);
        nu = item_units(a, len);
        item = s.off < (1LL << 31) ? (int)((uint32_t)s.off / (uint32_t)nu) : (int)div_long(s.off, nu);
        cut(a, (int)(s.off - (long long)item * nu));
    }
    __device__ __forceinline__ bool next(const Kv4Attn& a)
    {
        if (left <= 0) return false;
        if (++item == a.Hkv * a.mtiles) {
            item = 0;
            do {
                if (++b >= a.B) return false;  // only if the lengths change under the call
                len = seq_len(a, b);
                nu = item_units(a, len);
            } while (nu == 0);
        }
        cut(a, 0);
        return true;
    }
};

// Items that several teams hold, one record per team, filled by the team that
// holds the item's first tile.
struct MergeRec {
    int b, item, rest, pad;  // rest: the item's units that other teams hold (0: none begins here)
    Shares sh;
};

// A part: R rows of D outputs, each row's M and sum. R = 8: [R][D], [R][2];
// R = 128 (a thread per row): [D][R], [2][R].
__host__ __device__ constexpr size_t part_floats(int R, int D) { return (size_t)R * (D + 2); }

}  // namespace

// Joins the parts of split items (kv4_attn.cu); R: rows of an item's tile.
cudaError_t launch_kv4_merge(cudaStream_t s, const Kv4Attn& k, int D, int R);

// The kernel for many rows per KV head (kv4_attn_tc.cu).
size_t kv4_tc_bytes(const la_kv4_desc& c, const la_kv4_attn& a);
bool kv4_tc_init();
int launch_kv4_tc(cudaStream_t s, const la_kv4_desc& c, const la_kv4_attn& a, Kv4Attn k);

}  // namespace la
