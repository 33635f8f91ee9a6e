// gqa_prefill.h -- arguments of the prompt attention kernels (gqa_prefill,
// gqa_prefill_paged), dense and paged alike.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <stdint.h>

#include "gqa_params.h"

namespace gqa {

// Where the keys lie: packed dense tensors, or one of the paged cache's types.
enum { kPreDense = -1 };  // else a gqa_kv_dtype

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
    const float *k_scales;
    const float *v_scales;
    int n_scales;
    float v_scale;

    int Tq, B, Hq, Hkv, G;
    int causal;
    float alpha;  // scale * log2(e), times the host K scale
    unsigned long long wait_limit_ns;
    int fault_mode;  // test hook: 1 = the first tile of K is never loaded
    unsigned *err;   // device error word
};

}  // namespace gqa
