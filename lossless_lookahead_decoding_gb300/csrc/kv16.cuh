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
    int group, R;             // query heads of a KV head; its rows of one sequence, T x group
    int q_ld, k_ld, v_ld;
    int n_pages, max_pages, max_len, page_log2;
    int nP, pp, max_plen;     // prefixes, entries of a row of ptable, longest prefix
    int concat;               // a sequence's keys begin with its prefix's (else prefixes are entries of their own)
    float sl2;                // log2(e) / sqrt(D)
};

// Of a schedule, once it is known (on the device, for the merge).
struct Kv16Shares {
    long long q;              // team t begins at unit q t + min(t, r)
    int r, nteams, whole, pad;  // whole: a unit is a whole item; nteams 0: nothing to do
};

// How one kernel's teams share its entries (prefixes, then sequences), and
// where what they do not finish goes.
struct Kv16Sched {
    int n_pre, n_seq;         // entries
    int row_tile;             // rows of an item
    int blk_log2;             // blocks of 16 keys in a tile
    int wide;                 // with more rows than these an entry's tiles count twice
    int extra;                // units an item counts for beyond its tiles
    int nteams, min_run, slack;
    int finish;               // whole items go to the output (else to `whole`)
    int first;                // the call's first kernel
    Kv16Shares* shares;
    long long* base;          // [entries]: units before each
    float* slots;             // [nteams][2]: parts of split items
    float *whole, *whole_pre; // by row: results of sequences' and of prefixes' whole items
};

bool kv16_desc_ok(const la_kv16_desc* c);   // shapes
bool kv16_pool_ok(const la_kv16_desc* c);   // and pointers

// kv16_attn.cu
size_t kv16_attn_bytes(const la_kv16_desc& c, const la_kv16_attn& a);
int launch_kv16_attn(cudaStream_t s, const la_kv16_desc& c, const la_kv16_attn& a);

}  // namespace la
