// gqa_merge.cu -- attentions over parts of the keys made one by their LSEs.
//
//   w_p = exp(lse_p - max),  out = sum_p w_p out_p / sum_p w_p,  lse = max + ln sum_p w_p
//
// A thread takes 16 bytes (8 elements) of one row: all parts' pieces and the row's LSEs are loaded before any is used,
// the weights are worked out by every thread of the row (n exponentials, far less than the loads cost).  Bound by HBM: two
// parts of 16K tokens, 64 heads of 128, 128 us = 6.4 TB/s, 94 % of the measured copy rate.
#include "gqa_common.cuh"
#include "gqa_host.h"

namespace gqa {
namespace {

struct MergeArgs {
    const __nv_bfloat16 *outs[GQA_MERGE_MAX_PARTS];
    const float *lses[GQA_MERGE_MAX_PARTS];
    __nv_bfloat16 *out;
    float *lse;
    long long rows;
    int D8;  // pieces of a row
};

constexpr int kMergeThreads = 256;

template <int N>
__global__ void __launch_bounds__(kMergeThreads) gqa_merge_kernel(const MergeArgs a) {
    const int per = kMergeThreads / a.D8;  // whole rows of a CTA
    const int r = threadIdx.x / a.D8, piece = threadIdx.x % a.D8;
    const long long row = (long long)blockIdx.x * per + r;
    const bool there = r < per && row < a.rows;
    uint4 x[N];
    float s[N];
    if (there) {
#pragma unroll
        for (int p = 0; p < N; ++p) {
            s[p] = a.lses[p][row];
            x[p] = *reinterpret_cast<const uint4 *>(a.outs[p] + (row * a.D8 + piece) * 8);
        }
    }
    __syncthreads();  // lse may be one of the parts': every thread of the row has read it
    if (!there) return;
    float top = -INFINITY;
#pragma unroll
    for (int p = 0; p < N; ++p) top = fmaxf(top, s[p]);
    const float ref = top == -INFINITY ? 0.f : top;
    float w[N], total = 0.f;
#pragma unroll
    for (int p = 0; p < N; ++p) {
        w[p] = expf(s[p] - ref);
        total += w[p];
    }
    const float inv = 1.f / total;
    float o[8] = {};
#pragma unroll
    for (int p = 0; p < N; ++p) {
        if (s[p] == -INFINITY) continue;  // no share, whatever the part's row holds
        const float share = w[p] * inv;
        const __nv_bfloat162 *e = reinterpret_cast<const __nv_bfloat162 *>(&x[p]);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const float2 f = __bfloat1622float2(e[i]);
            o[2 * i] = fmaf(share, f.x, o[2 * i]);
            o[2 * i + 1] = fmaf(share, f.y, o[2 * i + 1]);
        }
    }
    uint4 y;
    y.x = pack_bf16x2(o[0], o[1]);
    y.y = pack_bf16x2(o[2], o[3]);
    y.z = pack_bf16x2(o[4], o[5]);
    y.w = pack_bf16x2(o[6], o[7]);
    *reinterpret_cast<uint4 *>(a.out + (row * a.D8 + piece) * 8) = y;
    if (a.lse != nullptr && piece == 0) a.lse[row] = total == 0.f ? -INFINITY : ref + logf(total);
}

template <int N>
void launch_merge(int n, const MergeArgs &a, cudaStream_t stream) {
    if constexpr (N > 0) {
        if (n != N) return launch_merge<N - 1>(n, a, stream);
        const int per = kMergeThreads / a.D8;
        gqa_merge_kernel<N><<<unsigned((a.rows + per - 1) / per), kMergeThreads, 0, stream>>>(a);
    }
}

}  // namespace
}  // namespace gqa

using namespace gqa;

extern "C" gqa_status gqa_merge(const void *const *outs, const float *const *lses, int n, void *out, float *lse,
                                long long rows, int D, gqa_stream_t stream) {
    if (outs == nullptr || lses == nullptr || n < 1 || n > GQA_MERGE_MAX_PARTS || rows < 0 || D < 1)
        return GQA_ERR_INVALID_ARG;
    if (D % 8 != 0 || D > 256 || rows >= (1LL << 31)) return GQA_ERR_UNSUPPORTED;
    if (rows == 0) return GQA_OK;
    MergeArgs a = {};
    for (int p = 0; p < n; ++p) {
        if (outs[p] == nullptr || lses[p] == nullptr) return GQA_ERR_INVALID_ARG;
        if (!host_aligned(outs[p], 16) || !host_aligned(lses[p], 4)) return GQA_ERR_ALIGNMENT;
        a.outs[p] = static_cast<const __nv_bfloat16 *>(outs[p]);
        a.lses[p] = lses[p];
    }
    if (out == nullptr) return GQA_ERR_INVALID_ARG;
    if (!host_aligned(out, 16) || !host_aligned(lse, 4)) return GQA_ERR_ALIGNMENT;
    int dev = 0;
    if (!host_current_device(&dev)) return GQA_ERR_CUDA;
    a.out = static_cast<__nv_bfloat16 *>(out);
    a.lse = lse;
    a.rows = rows;
    a.D8 = D / 8;
    launch_merge<GQA_MERGE_MAX_PARTS>(n, a, reinterpret_cast<cudaStream_t>(stream));
    if (cudaGetLastError() != cudaSuccess) return GQA_ERR_CUDA;
    return GQA_OK;
}
