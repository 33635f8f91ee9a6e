// gqa_paged_int4.cu -- paged decode over whole requests from a 4-bit cache.
//
// First form: one CTA per query row and head, its warps striding over the
// tokens with an online softmax each, merged in shared memory.
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <cmath>

#include "gqa_common.cuh"
#include "gqa_host.h"

namespace gqa {
namespace {

struct Int4Args {
    const __nv_bfloat16 *q;
    const uint8_t *k_pool, *v_pool;
    const __half *params;
    const int32_t *page_table, *seq_lens;
    __nv_bfloat16 *out;
    float *lse;
    int B, Sq, Hq, Hkv, page_size, pages_per_req, num_pages;
    float alpha;  // scale * log2(e)
    unsigned *err;
};

template <int D>
__global__ void __launch_bounds__(128) gqa_paged_int4_kernel(const Int4Args a) {
    constexpr int E = D / 32;  // elements per lane
    __shared__ float sm_m[4], sm_l[4], sm_o[4][D];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int h = blockIdx.x % a.Hq, i = blockIdx.x / a.Hq, b = blockIdx.y;
    const int g = h / (a.Hq / a.Hkv);
    pdl_wait_primary();
    const int cap = a.pages_per_req * a.page_size;
    const int len0 = __ldg(a.seq_lens + b);
    const int len = min(max(len0, 0), cap);
    bool bad = len != len0;
    const size_t row = (size_t(b) * a.Sq + i) * a.Hq + h;
    float q[E], o[E], m = -INFINITY, l = 0.f;
#pragma unroll
    for (int e = 0; e < E; ++e) q[e] = __bfloat162float(a.q[row * D + lane * E + e]), o[e] = 0.f;
    const int n = len - a.Sq + i + 1;  // visible tokens
    for (int t = warp; t < n; t += 4) {
        const int page = __ldg(a.page_table + size_t(b) * a.pages_per_req + t / a.page_size);
        if (page < 0 || page >= a.num_pages) {
            bad = true;
            continue;
        }
        const size_t head_row = (size_t(page) * a.page_size + t % a.page_size) * a.Hkv + g;
        float kz[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) kz[j] = __half2float(a.params[head_row * 4 + j]);
        float s = 0.f, v[E];
#pragma unroll
        for (int e = 0; e < E; ++e) {
            const int d = lane * E + e;
            const uint8_t kc = a.k_pool[head_row * (D / 2) + d / 2], vc = a.v_pool[head_row * (D / 2) + d / 2];
            s += q[e] * (float((kc >> (4 * (d & 1))) & 15) * kz[0] + kz[1]);
            v[e] = float((vc >> (4 * (d & 1))) & 15) * kz[2] + kz[3];
        }
#pragma unroll
        for (int off = 16; off > 0; off >>= 1) s += __shfl_xor_sync(0xffffffffu, s, off);
        s *= a.alpha;
        const float mn = fmaxf(m, s);
        const float corr = exp2f(m - mn), p = exp2f(s - mn);
        l = l * corr + p;
#pragma unroll
        for (int e = 0; e < E; ++e) o[e] = o[e] * corr + p * v[e];
        m = mn;
    }
    if (lane == 0) sm_m[warp] = m, sm_l[warp] = l;
#pragma unroll
    for (int e = 0; e < E; ++e) sm_o[warp][lane * E + e] = o[e];
    if (bad) flag_error(a.err, kErrIndex);
    __syncthreads();
    float M = -INFINITY, L = 0.f;
    for (int w = 0; w < 4; ++w) M = fmaxf(M, sm_m[w]);
    float f[4];
    for (int w = 0; w < 4; ++w) {
        f[w] = sm_l[w] == 0.f ? 0.f : exp2f(sm_m[w] - M);
        L += f[w] * sm_l[w];
    }
    if (threadIdx.x < D) {
        float x = 0.f;
        for (int w = 0; w < 4; ++w) x += f[w] * sm_o[w][threadIdx.x];
        a.out[row * D + threadIdx.x] = __float2bfloat16(L == 0.f ? 0.f : x / L);
    }
    if (a.lse != nullptr && threadIdx.x == 0)
        a.lse[(size_t(b) * a.Hq + h) * a.Sq + i] = L == 0.f ? -INFINITY : (M + log2f(L)) * 0.69314718055994530942f;
}

constexpr int kInt4MaxRows = 128;  // query rows per KV head

gqa_status check_int4(int B, int Sq, int Hq, int Hkv, int D, int page_size, int pages_per_req, int num_pages) {
    gqa_status st = host_check_pages(B, Hkv, D, page_size, pages_per_req, num_pages);
    if (st != GQA_OK) return st;
    if (Sq < 1 || Hq < 1 || Hq % Hkv != 0) return GQA_ERR_INVALID_ARG;
    if ((long long)(Hq / Hkv) * Sq > kInt4MaxRows) return GQA_ERR_UNSUPPORTED;
    return GQA_OK;
}

}  // namespace
}  // namespace gqa

using namespace gqa;

extern "C" gqa_status gqa_decode_paged_int4(const void *q, const void *k_pool, const void *v_pool,
                                            const void *kv_params, const int32_t *page_table,
                                            const int32_t *seq_lens, void *out, float *lse, int B, int Sq, int Hq,
                                            int Hkv, int D, int page_size, int pages_per_req, int num_pages,
                                            float scale, int num_splits, void *workspace, size_t workspace_bytes,
                                            gqa_stream_t stream) {
    gqa_status st = check_int4(B, Sq, Hq, Hkv, D, page_size, pages_per_req, num_pages);
    if (st != GQA_OK) return st;
    if (num_splits < 0) return GQA_ERR_INVALID_ARG;
    if (q == nullptr || k_pool == nullptr || v_pool == nullptr || kv_params == nullptr || page_table == nullptr ||
        seq_lens == nullptr || out == nullptr)
        return GQA_ERR_INVALID_ARG;
    if (!host_aligned(q, 16) || !host_aligned(k_pool, 16) || !host_aligned(v_pool, 16) || !host_aligned(out, 16) ||
        !host_aligned(kv_params, 16) || !host_aligned(lse, 4) || !host_aligned(page_table, 4) ||
        !host_aligned(seq_lens, 4))
        return GQA_ERR_ALIGNMENT;
    int dev = 0;
    if (!host_current_device(&dev)) return GQA_ERR_CUDA;
    Int4Args a = {};
    a.q = static_cast<const __nv_bfloat16 *>(q);
    a.k_pool = static_cast<const uint8_t *>(k_pool);
    a.v_pool = static_cast<const uint8_t *>(v_pool);
    a.params = static_cast<const __half *>(kv_params);
    a.page_table = page_table;
    a.seq_lens = seq_lens;
    a.out = static_cast<__nv_bfloat16 *>(out);
    a.lse = lse;
    a.B = B;
    a.Sq = Sq;
    a.Hq = Hq;
    a.Hkv = Hkv;
    a.page_size = page_size;
    a.pages_per_req = pages_per_req;
    a.num_pages = num_pages;
    a.alpha = host_resolve_scale(scale, D) * 1.4426950408889634f;
    a.err = host_error_word(dev);
    cudaStream_t cs = reinterpret_cast<cudaStream_t>(stream);
    const dim3 grid(unsigned(Sq * Hq), unsigned(B));
    if (D == 64)
        gqa_paged_int4_kernel<64><<<grid, 128, 0, cs>>>(a);
    else
        gqa_paged_int4_kernel<128><<<grid, 128, 0, cs>>>(a);
    if (cudaGetLastError() != cudaSuccess) return GQA_ERR_CUDA;
    (void)workspace;
    (void)workspace_bytes;
    return GQA_OK;
}

extern "C" int gqa_decode_paged_int4_num_splits(int B, int Sq, int Hq, int Hkv, int D, int page_size,
                                                int pages_per_req) {
    const gqa_status st = check_int4(B, Sq, Hq, Hkv, D, page_size, pages_per_req, 1);
    return st == GQA_OK ? 1 : -int(st);
}

extern "C" size_t gqa_decode_paged_int4_workspace_bytes(int B, int Sq, int Hq, int Hkv, int D, int page_size,
                                                        int pages_per_req, int num_splits) {
    return 0;
}
