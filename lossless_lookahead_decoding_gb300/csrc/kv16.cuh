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

// An item whose parts are to be joined, left by the team that begins it.
struct alignas(16) Kv16Item {
    int t0, n;        // the teams that have a part, one after the other (n 0: none)
    int row, rows;    // its first row (among all sequences' rows of its KV head), and how many
    int g;            // KV head
    int pre_row;      // first row of the sequence's prefix (-1: none)
    int pad[2];
};

// What the two kinds of teams work in: rows of an item; blocks of 16 keys in a tile;
// with more rows than these (0: never) an entry's tiles count twice; units an item
// counts for beyond its tiles; units worth a team; units that whole items are worth.
// Measured around these (in a graph, us): slack 0 for 0 to 30, 4 steps of 121 rows 29.7
// for 21.3 and 6 blocks of 100 rows 45.2 for 42.2; slack 0 of RowsKind, two short chats
// 12.5 for 7.75, 48, 128 single tokens behind 1000 83.7 for 65.5 and 32 behind 32 767
// 72.8 for 55.0.  extra halved and doubled, min_run 2 and 16 (24): all within 4 %.
struct WideKind {
    static constexpr int row_tile = 256, blk_log2 = 3, twice = 128, extra = 4, min_run = 6, slack = 12;
};
struct RowsKind {
    static constexpr int row_tile = 16, blk_log2 = 0, twice = 0, extra = 2, min_run = 8, slack = 16;  // (one item holds all rows)
};

// How one kind of teams share its entries (prefixes, then sequences), and
// where what they do not finish goes.
struct Kv16Sched {
    int n_pre, n_seq;         // entries
    int nteams, per_cta;      // teams; of a CTA
    int direct;               // team t has item t: all items are sequences', and there is a team for each
    int finish;               // whole items go to the output (else to `whole`)
    Kv16Item* items;          // finish: [nteams]; else [KV heads][rows]: of prefixes, then of sequences
    int* bad;                 // prefix_first is out of order, or there is too much to do: nothing is done
    float* slots;             // [nteams][2]: parts of split items
    float *whole, *whole_pre; // by row: results of sequences' and of prefixes' whole items
};

bool kv16_desc_ok(const la_kv16_desc* c);   // shapes
bool kv16_pool_ok(const la_kv16_desc* c);   // and pointers

// kv16_attn.cu
size_t kv16_attn_bytes(const la_kv16_desc& c, const la_kv16_attn& a);
int launch_kv16_attn(cudaStream_t s, const la_kv16_desc& c, const la_kv16_attn& a);

}  // namespace la
