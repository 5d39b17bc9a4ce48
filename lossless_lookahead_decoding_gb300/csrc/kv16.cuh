// kv16.cuh -- the paged bf16 KV cache: what its kernels and entry points share.
// Pages are plain arrays, [n_pages][KV heads][page][D] of keys and of values:
// the rows of a page and head are contiguous, so any 16 tokens of them are one
// box of a tensor map.
#pragma once
#include "kv4.cuh"

namespace la {

struct Kv16Attn {
    const __nv_bfloat16 *q, *ks, *vs;
    __nv_bfloat16* out;
    const int *lens, *table;
    const int *plens, *ptable, *pfirst;
    int* status;
    const __nv_bfloat16 *kp, *vp;
    int B, H, Hkv, T, W, n1;  // n1 = N - 1
    int q_ld, k_ld, v_ld;
    int n_pages, max_pages, max_len, page_log2;
    int nP, pp, max_plen;     // prefixes, entries of a row of ptable, longest prefix
    float sl2;                // log2(e) / sqrt(D)
};

bool kv16_desc_ok(const la_kv16_desc* c);   // shapes
bool kv16_pool_ok(const la_kv16_desc* c);   // and pointers

// kv16_attn.cu
size_t kv16_attn_bytes(const la_kv16_desc& c, const la_kv16_attn& a);
int launch_kv16_attn(cudaStream_t s, const la_kv16_desc& c, const la_kv16_attn& a);

}  // namespace la
