// kv16_rows.cu -- the attention of at most 16 rows per KV head (kv16_rows.cuh) as
// a kernel of its own: a CTA of 8 teams a SM.
#include "kv16_rows.cuh"

namespace la {
namespace {

constexpr int kWarps = 8;

template <int D>
__global__ void __launch_bounds__(kWarps * 32, 1) k_kv16_rows(const __grid_constant__ Kv16Attn a, const __grid_constant__ Kv16Sched s)
{
    using L = RowsSmem<D, kWarps>;
    extern __shared__ __align__(16) uint8_t sm[];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    pdl_wait();
    pdl_trigger();
    const Prefixes pre = find_starts<RowsKind>(a, s, L::starts(sm), L::scan(sm), L::pre(sm));
    const Shares sh = L::scan(sm)->shares;
    const Start st = L::starts(sm)[warp];
    if (s.finish && s.items && lane == 0) {
        const int id = blockIdx.x * kWarps + warp;  // (every entry is written by one warp)
        if (id >= sh.nteams && id < s.nteams) s.items[id].n = 0;
        if (st.count > 0) s.items[st.team].n = 0;
    }
    rows_team<D, kWarps>(a, s, sm, pre, sh, st);
}

}  // namespace

int kv16_rows_teams() { return kSMs * kWarps; }

bool kv16_rows_init()
{
    return cudaFuncSetAttribute(k_kv16_rows<128>, cudaFuncAttributeMaxDynamicSharedMemorySize, RowsSmem<128, kWarps>::kBytes) == cudaSuccess &&
           cudaFuncSetAttribute(k_kv16_rows<64>, cudaFuncAttributeMaxDynamicSharedMemorySize, RowsSmem<64, kWarps>::kBytes) == cudaSuccess;
}

cudaError_t launch_kv16_rows(cudaStream_t s, const Kv16Attn& a, const Kv16Sched& w, int D)
{
    const dim3 grid((w.nteams + kWarps - 1) / kWarps), block(kWarps * 32);
    return D == 128 ? launch_pdl(k_kv16_rows<128>, grid, block, RowsSmem<128, kWarps>::kBytes, s, a, w)
                    : launch_pdl(k_kv16_rows<64>, grid, block, RowsSmem<64, kWarps>::kBytes, s, a, w);
}

}  // namespace la
