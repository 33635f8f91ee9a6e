// gqa_prefill.h -- arguments and work plan of the prompt attention kernels
// (gqa_prefill, gqa_prefill_paged), dense and paged alike.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <stdint.h>

#include "gqa_params.h"

namespace gqa {

// Where the keys lie.
enum PrefillSource {
    kPreDense,  // packed tensors, by TMA
    kPrePages,  // bf16 pool whose pages are whole swizzle atoms (8 tokens), by TMA
    kPreCopy,   // bf16 pool of any page size, through registers
    kPreFp8,    // 8-bit and 4-bit pools, converted on the way into shared memory
    kPreInt8,
    kPreInt4,
};

constexpr int kPreKeys = 128;   // keys of a step
constexpr int kPreTile = 128;   // query rows of a tile; an item has one or two
constexpr int kPreMinSplit = 6; // steps that a part of a divided item has at least, as planned
constexpr int kPreSnap = 3;     // ... and as cut: nearer to an item's end, the cut moves there

// A piece of work is steps [s0, s1) of an item: up to 2 * tok_tile consecutive tokens of one sequence, for one block of
// query heads of one KV head (the item's rows), over the keys that its last row sees.
struct PrefillItem {
    int q_row;   // first token's row of q
    int n_tok;
    int req;
    int steps;   // of kPreKeys keys
    int limit0;  // keys that the first token sees, before clamping into [0, L]; each further one sees one more
    int L;       // keys of the sequence
    int k_row;   // first key's row of k and v (dense)
    int cost;
};

struct PrefillPlan {
    int n_items;
    int rounds;     // whole items: worker w takes, in round r, number r * W + w, or r * W + W - 1 - w in odd rounds
    int total;      // items x head blocks
    int n_joins;    // items with partial results
};

struct PrefillArgs {
    const __nv_bfloat16 *q;
    long long q_stride;
    __nv_bfloat16 *out;
    float *lse;
    const int32_t *cu_q;  // [B + 1] or null: per_q rows each
    int per_q;
    // dense keys
    const __nv_bfloat16 *k;
    const __nv_bfloat16 *v;
    long long k_stride, v_stride;
    const int32_t *cu_k;  // [B + 1] or null: per_k keys each
    int per_k;
    int Tk;
    // paged keys
    const uint8_t *k_pool;
    const uint8_t *v_pool;
    const __half *params;
    const int32_t *page_table;
    const int32_t *seq_lens;
    int page_size, pages_per_req, num_pages;
    unsigned page_mul;  // t / page_size = t * page_mul >> page_shift
    int page_shift;
    int box_rows;  // tokens of a TMA box
    const float *k_scales;
    const float *v_scales;
    int n_scales;
    float v_scale;

    int Tq, B, Hq, Hkv, G;
    int g_tile;    // query heads of a tile: rows are tok_tile tokens x g_tile heads
    int tok_tile;
    int head_blocks;  // Hkv x blocks of g_tile heads of a KV head
    int causal;
    float alpha;  // scale * log2(e), times the host K scale

    // the plan, in the workspace
    int workers;
    int may_split;
    int direct;  // no plan: CTA i has item i, whole
    int max_items;
    PrefillPlan *plan;
    PrefillItem *items;      // [max_items], longest first
    // where the planning CTA's shared memory does not hold them
    PrefillItem *unsorted;   // [max_items]
    int *tile_prefix;        // [B + 1]
    long long *cost_prefix;  // [max_items + 1]
    int4 *joins;             // [workers]: of a divided item its number, the worker with its beginning and the one with its end
    int2 *cuts;              // [workers + 1]: where a worker's share of the divided part begins (number, step)
    float *o_part;           // [2 workers][2 * kPreTile][Dv]
    float *lse_part;         // [2 workers][2 * kPreTile], log2 domain

    unsigned long long wait_limit_ns;
    int fault_mode;  // test hook: 1 = the first tile of K is never loaded
    unsigned *err;   // device error word
};

}  // namespace gqa
