// kv4.cuh -- the paged 4-bit KV cache: its format, and what its kernels share.
//
// A key or value vector of one token and KV head (D channels) is held as 4-bit
// codes c with a bf16 scale s and a zero point z in 0..15 and stands for
// (c - z) s.  Sixteen tokens of one head are one block of 16 D + 128 bytes,
// contiguous, so that any tile of 16 keys is one bulk copy whatever the page
// size is:
//   K codes  [D / 64 panels][16 tokens][32 bytes]
//   V codes  the same
//   K parameters [16 words], V parameters [16 words]
// A panel row holds 64 channels as 8 words; word w holds channels 8w..8w+7,
// channel 2i at bits 4i and channel 2i + 1 at bits 16 + 4i: one shift and one
// mask give two neighbouring channels in the two halves of a register.
// Rows of 32 bytes (and not of D / 2) keep the warp's shared-memory reads of
// both the K and the V fragments free of bank conflicts (see kv4_key).
// A parameter word is the scale's bf16 bits above the bf16 bits of 128 + z
// (0x4300 | z): a code is turned into bf16 by writing it into the mantissa of
// 128, and subtracting 128 + z is then exact.
#pragma once
#include "../../include/lookahead.h"
#include "common.cuh"
#include "ptx.cuh"

namespace la {

constexpr int kKv4Block = 16;  // tokens per block

__host__ __device__ constexpr int kv4_block_bytes(int D) { return 16 * D + 128; }

// Device status word: the first error stays until the caller clears it.
__device__ __forceinline__ void kv4_raise(int* status, int code)
{
    if (status) atomicCAS(status, 0, code);
}

// Bytes from the page array's start to the block of (page, head, block of the page).
__host__ __device__ __forceinline__ size_t kv4_block_at(int page, int head, int blk, int n_kv_heads, int blk_log2, int D)
{
    return ((((size_t)page * n_kv_heads + head) << blk_log2) + blk) * kv4_block_bytes(D);
}

// packed pairs of fp32: one instruction for two
__device__ __forceinline__ uint64_t pair(float a, float b)
{
    uint64_t r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a), "f"(b));
    return r;
}
__device__ __forceinline__ void unpair(uint64_t x, float& a, float& b) { asm("mov.b64 {%0, %1}, %2;" : "=f"(a), "=f"(b) : "l"(x)); }
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c)
{
    uint64_t r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
    return r;
}
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b)
{
    uint64_t r;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}

// Whether step row j is visible to step row i (the combined 2D-window +
// verification mask): every row sees row 0; lookahead row (l, c) sees level 0
// up to column c and column c up to level l; verification row (g, i) sees its
// own candidate up to i.
__host__ __device__ __forceinline__ bool kv4_sees(int i, int j, int W, int n1)
{
    if (j == 0) return true;
    if (j > i) return false;
    const int nl = W * n1;
    if (i <= nl) {
        const int c = (i - 1) % W, cj = (j - 1) % W;
        return cj == c || (j <= W && cj < c);
    }
    return j > nl && (i - 1 - nl) / n1 == (j - 1 - nl) / n1;
}

struct Kv4Attn {
    const uint8_t* pages;
    const __nv_bfloat16 *q, *ks, *vs;
    __nv_bfloat16* out;
    const int *lens, *table;
    int* status;
    float* part;             // partial outputs, maxima and sums of split items
    int B, H, Hkv, T, W, n1; // n1 = N - 1
    int q_ld, kv_ld;
    int n_pages, max_pages, max_len, blk_log2;
    int rows, mtiles;        // rows of one KV head (T x heads per KV head), row tiles
    int tile_log2;           // keys of a tile (the step's rows are one tile)
    int nteams, extra;       // teams that share the items; tiles an item counts for beyond its own
    float sl2;               // log2(e) / sqrt(D)
};

// Host helpers of both caches' entry points.
inline int log2_of(int x)
{
    int l = 0;
    while ((1 << l) < x) l++;
    return l;
}

inline bool aligned(const void* p, int to) { return ((uintptr_t)p & (uintptr_t)(to - 1)) == 0; }

// every address one of an int (a misaligned access would end the context)
template <typename... P>
bool ints_aligned(const P*... p)
{
    return (aligned(p, 4) && ...);
}

// kv4_cache.cu
int launch_kv4_plan(cudaStream_t s, const la_kv4_desc& c, const int* lens, const int* n_new, int B, const int* free_pages,
                    const int* n_free, int* table, int* slots, int n_slots, int stride, int* new_lens, int* left);
int launch_kv4_release(cudaStream_t s, const la_kv4_desc& c, const int* done, int B, int* lens, const int* table,
                       int* free_pages, int* n_free);
int launch_kv4_append(cudaStream_t s, const la_kv4_desc& c, const void* k, const void* v, int dtype, int ld, int n_rows,
                      const int* rows, const int* slots, int n);
int launch_kv4_read(cudaStream_t s, const la_kv4_desc& c, const int* slots, int n, void* k, void* v, int dtype, int ld);

// kv4_attn.cu
size_t kv4_attn_bytes(const la_kv4_desc& c, const la_kv4_attn& a);
int launch_kv4_attn(cudaStream_t s, const la_kv4_desc& c, const la_kv4_attn& a);

}  // namespace la
