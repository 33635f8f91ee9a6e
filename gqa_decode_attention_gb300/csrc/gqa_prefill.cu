// gqa_prefill.cu -- attention over packed prompts and of new tokens over the
// paged cache: kernel, and the C entry points.
#include <cmath>

#include "gqa_common.cuh"
#include "gqa_host.h"
#include "gqa_prefill.h"

namespace gqa {
namespace {

// First and one past the last row of sequence b, clamped into [0, total].
__device__ __forceinline__ void prefill_range(const int32_t *cu, int per, int b, int total, unsigned *err, int *from,
                                              int *to) {
    if (cu == nullptr) {
        *from = b * per, *to = (b + 1) * per;
        return;
    }
    const int f = cu[b], t = cu[b + 1];
    *from = min(max(f, 0), total);
    *to = min(max(t, *from), total);
    if (*from != f || *to != t) flag_error(err, kErrIndex);
}

template <int N>
__device__ __forceinline__ void load_bf16(float (&x)[N], const __nv_bfloat16 *p) {
#pragma unroll
    for (int i = 0; i < N; i += 2) {
        const float2 f = __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162 *>(p + i));
        x[i] = f.x, x[i + 1] = f.y;
    }
}

// Elements d .. d + N - 1 of key `row` (of a pool) and KV head g.
template <int KVT, int D, int N>
__device__ __forceinline__ void load_codes(float (&x)[N], const uint8_t *pool, const __half *params, int which,
                                           long long row, int Hkv, int g, int d) {
    const long long head = row * Hkv + g;
    if constexpr (KVT == GQA_KV_BF16) {
        load_bf16(x, reinterpret_cast<const __nv_bfloat16 *>(pool) + head * D + d);
    } else if constexpr (KVT == GQA_KV_INT4) {
        const float scale = __half2float(params[head * 4 + 2 * which]);
        const float zero = __half2float(params[head * 4 + 2 * which + 1]);
#pragma unroll
        for (int i = 0; i < N; i += 2) {
            const int c = pool[head * (D / 2) + (d + i) / 2];
            x[i] = float(c & 15) * scale + zero, x[i + 1] = float(c >> 4) * scale + zero;
        }
    } else {
#pragma unroll
        for (int i = 0; i < N; ++i) {
            const uint8_t c = pool[head * D + d + i];
            if constexpr (KVT == GQA_KV_INT8) {
                x[i] = float(int8_t(c));
            } else {
                const uint32_t h = e4m3x2_to_f16x2(c);
                x[i] = __half2float(*reinterpret_cast<const __half *>(&h));
            }
        }
    }
}

// One warp a (query row, head): the keys one after the other, the head size over the lanes.
template <int KVT, int D, int DV>
__global__ void __launch_bounds__(128) gqa_prefill_kernel(const PrefillArgs a) {
    const int lane = threadIdx.x & 31;
    const long long unit = (long long)blockIdx.x * 4 + (threadIdx.x >> 5);
    if (unit >= (long long)a.Tq * a.Hq) return;
    const int t = int(unit / a.Hq), h = int(unit % a.Hq), g = h / a.G;
    int from = 0, to = 0, b = 0;
    if (a.cu_q == nullptr) {
        b = t / a.per_q;
        prefill_range(nullptr, a.per_q, b, a.Tq, a.err, &from, &to);
    } else {
        b = a.B;
        for (int x = a.B - 1; x >= 0; --x) {
            int f, e;
            prefill_range(a.cu_q, 0, x, a.Tq, a.err, &f, &e);
            if (t >= f && t < e) b = x, from = f, to = e;
        }
        if (b == a.B) return;
    }
    int kf = 0, kt = 0;
    if constexpr (KVT == kPreDense) {
        prefill_range(a.cu_k, a.per_k, b, a.Tk, a.err, &kf, &kt);
    } else {
        const int cap = a.pages_per_req * a.page_size;
        kt = min(max(a.seq_lens[b], 0), cap);
        if (kt != a.seq_lens[b]) flag_error(a.err, kErrIndex);
    }
    const int L = kt - kf;
    const int seen = a.causal ? min(max(L - (to - from) + (t - from) + 1, 0), L) : L;
    constexpr int N = D / 32, NV = DV / 32;
    float q[N], o[NV] = {}, m = -INFINITY, l = 0.f;
    load_bf16(q, a.q + t * a.q_stride + h * D + lane * N);
    float alpha = a.alpha, vs = a.v_scale;
    if (a.k_scales != nullptr) {
        alpha *= a.k_scales[a.n_scales > 1 ? g : 0];
        vs = a.v_scales[a.n_scales > 1 ? g : 0];
    }
    for (int j = 0; j < seen; ++j) {
        float k[N] = {}, v[NV] = {};
        if constexpr (KVT == kPreDense) {
            load_bf16(k, a.k + (long long)(kf + j) * a.k_stride + g * D + lane * N);
            load_bf16(v, a.v + (long long)(kf + j) * a.v_stride + g * DV + lane * NV);
        } else {
            const int page = a.page_table[(long long)b * a.pages_per_req + j / a.page_size];
            if (page < 0 || page >= a.num_pages) {
                flag_error(a.err, kErrIndex);
            } else {
                const long long row = (long long)page * a.page_size + j % a.page_size;
                load_codes<KVT, D>(k, a.k_pool, a.params, 0, row, a.Hkv, g, lane * N);
                load_codes<KVT, D>(v, a.v_pool, a.params, 1, row, a.Hkv, g, lane * NV);
            }
        }
        float s = 0.f;
#pragma unroll
        for (int i = 0; i < N; ++i) s += q[i] * k[i];
#pragma unroll
        for (int x = 16; x > 0; x >>= 1) s += __shfl_xor_sync(0xffffffffu, s, x);
        s *= alpha;
        const float m2 = fmaxf(m, s);
        const float use = m2 == -INFINITY ? 0.f : m2;
        const float f = exp2f(m - use), p = exp2f(s - use);
        m = m2;
        l = l * f + p;
#pragma unroll
        for (int i = 0; i < NV; ++i) o[i] = o[i] * f + p * v[i];
    }
    const float inv = l == 0.f ? 0.f : vs / l;
    __nv_bfloat16 *dst = a.out + (long long)unit * DV + lane * NV;
#pragma unroll
    for (int i = 0; i < NV; ++i) dst[i] = __float2bfloat16(l == 0.f ? 0.f : o[i] * inv);
    if (a.lse != nullptr && lane == 0) a.lse[unit] = l == 0.f ? -INFINITY : (m + log2f(l)) * 0.69314718055994530942f;
}

template <int KVT, int D, int DV>
gqa_status launch_prefill(const PrefillArgs &a, cudaStream_t stream) {
    const long long units = (long long)a.Tq * a.Hq;
    gqa_prefill_kernel<KVT, D, DV><<<unsigned((units + 3) / 4), 128, 0, stream>>>(a);
    if (cudaGetLastError() != cudaSuccess) return GQA_ERR_CUDA;
    return GQA_OK;
}

// What both entry points check alike.
gqa_status check_prefill(int Tq, int B, int Hq, int Hkv, int Dqk, int Dv) {
    if (Tq < 0 || B < 1 || Hkv < 1 || Hq < 1 || Hq % Hkv != 0) return GQA_ERR_INVALID_ARG;
    if (!((Dqk == 64 && Dv == 64) || (Dqk == 128 && Dv == 128) || (Dqk == 192 && Dv == 128))) return GQA_ERR_UNSUPPORTED;
    if (B > 65535 || Hq / Hkv > 4096 || (long long)Tq * Hq >= (1LL << 31)) return GQA_ERR_UNSUPPORTED;
    return GQA_OK;
}

}  // namespace
}  // namespace gqa

using namespace gqa;

extern "C" size_t gqa_prefill_workspace_bytes(int Tq, int B, int Hq, int Hkv, int Dqk, int Dv) {
    (void)Tq, (void)B, (void)Hq, (void)Hkv, (void)Dqk, (void)Dv;
    return 0;
}

extern "C" size_t gqa_prefill_paged_workspace_bytes(int T, int B, int Hq, int Hkv, int D) {
    return gqa_prefill_workspace_bytes(T, B, Hq, Hkv, D, D);
}

extern "C" gqa_status gqa_prefill(const void *q, long long q_stride, const void *k, long long k_stride, const void *v,
                                  long long v_stride, const int32_t *cu_q, const int32_t *cu_k, void *out, float *lse,
                                  int Tq, int Tk, int B, int Hq, int Hkv, int Dqk, int Dv, int causal, float scale,
                                  void *workspace, size_t workspace_bytes, gqa_stream_t stream) {
    gqa_status st = check_prefill(Tq, B, Hq, Hkv, Dqk, Dv);
    if (st != GQA_OK) return st;
    if (Tk < 0 || (cu_q == nullptr && Tq % B != 0) || (cu_q == nullptr && cu_k == nullptr && Tk % B != 0))
        return GQA_ERR_INVALID_ARG;
    if (Tq > 0 && (q == nullptr || out == nullptr || (Tk > 0 && (k == nullptr || v == nullptr)))) return GQA_ERR_INVALID_ARG;
    if (q_stride < (long long)Hq * Dqk || k_stride < (long long)Hkv * Dqk || v_stride < (long long)Hkv * Dv)
        return GQA_ERR_INVALID_ARG;
    if (q_stride % 8 != 0 || k_stride % 8 != 0 || v_stride % 8 != 0 || !host_aligned(q, 16) || !host_aligned(k, 16) ||
        !host_aligned(v, 16) || !host_aligned(out, 16) || !host_aligned(lse, 4) || !host_aligned(cu_q, 4) ||
        !host_aligned(cu_k, 4))
        return GQA_ERR_ALIGNMENT;
    if (Tq == 0) return GQA_OK;
    int dev = 0;
    if (!host_current_device(&dev)) return GQA_ERR_CUDA;
    PrefillArgs a = {};
    a.q = static_cast<const __nv_bfloat16 *>(q);
    a.k = static_cast<const __nv_bfloat16 *>(k);
    a.v = static_cast<const __nv_bfloat16 *>(v);
    a.q_stride = q_stride, a.k_stride = k_stride, a.v_stride = v_stride;
    a.cu_q = cu_q;
    a.cu_k = cu_k != nullptr ? cu_k : cu_q;
    a.per_q = Tq / B, a.per_k = Tk / B;
    a.Tk = Tk;
    a.out = static_cast<__nv_bfloat16 *>(out);
    a.lse = lse;
    a.v_scale = 1.f;
    a.Tq = Tq, a.B = B, a.Hq = Hq, a.Hkv = Hkv, a.G = Hq / Hkv;
    a.causal = causal != 0;
    a.alpha = host_resolve_scale(scale, Dqk) * 1.4426950408889634f;
    a.wait_limit_ns = host_wait_limit_ns();
    a.fault_mode = host_fault_mode();
    a.err = host_error_word(dev);
    cudaStream_t cs = reinterpret_cast<cudaStream_t>(stream);
    if (Dqk == 64) return launch_prefill<kPreDense, 64, 64>(a, cs);
    if (Dqk == 128) return launch_prefill<kPreDense, 128, 128>(a, cs);
    return launch_prefill<kPreDense, 192, 128>(a, cs);
}

extern "C" gqa_status gqa_prefill_paged(const void *q, long long q_stride, int kv_dtype, const void *k_pool,
                                        const void *v_pool, const void *kv_params, float k_scale, float v_scale,
                                        const float *k_scales, const float *v_scales, int n_scales,
                                        const int32_t *page_table, const int32_t *seq_lens, const int32_t *cu_tokens,
                                        void *out, float *lse, int T, int B, int Hq, int Hkv, int D, int page_size,
                                        int pages_per_req, int num_pages, int causal, float scale, void *workspace,
                                        size_t workspace_bytes, gqa_stream_t stream) {
    gqa_status st = host_check_pages(B, Hkv, D, page_size, pages_per_req, num_pages);
    if (st != GQA_OK) return st;
    st = check_prefill(T, B, Hq, Hkv, D, D);
    if (st != GQA_OK) return st;
    if ((long long)pages_per_req * page_size > (1LL << 31) - 256) return GQA_ERR_UNSUPPORTED;  // key indexes step past the end
    st = host_check_cache(kv_dtype, kv_params, k_scale, v_scale, k_scales, v_scales, n_scales, Hkv);
    if (st != GQA_OK) return st;
    if (cu_tokens == nullptr && T % B != 0) return GQA_ERR_INVALID_ARG;
    if (k_pool == nullptr || v_pool == nullptr || page_table == nullptr || seq_lens == nullptr ||
        (T > 0 && (q == nullptr || out == nullptr)) || q_stride < (long long)Hq * D)
        return GQA_ERR_INVALID_ARG;
    if (q_stride % 8 != 0 || !host_aligned(q, 16) || !host_aligned(out, 16) || !host_aligned(k_pool, 16) ||
        !host_aligned(v_pool, 16) || !host_aligned(lse, 4) || !host_aligned(page_table, 4) ||
        !host_aligned(seq_lens, 4) || !host_aligned(cu_tokens, 4))
        return GQA_ERR_ALIGNMENT;
    if (T == 0) return GQA_OK;
    int dev = 0;
    if (!host_current_device(&dev)) return GQA_ERR_CUDA;
    PrefillArgs a = {};
    a.q = static_cast<const __nv_bfloat16 *>(q);
    a.q_stride = q_stride;
    a.cu_q = cu_tokens;
    a.per_q = T / B;
    a.out = static_cast<__nv_bfloat16 *>(out);
    a.lse = lse;
    a.k_pool = static_cast<const uint8_t *>(k_pool);
    a.v_pool = static_cast<const uint8_t *>(v_pool);
    a.params = static_cast<const __half *>(kv_params);
    a.page_table = page_table;
    a.seq_lens = seq_lens;
    a.page_size = page_size, a.pages_per_req = pages_per_req, a.num_pages = num_pages;
    const bool kv8 = kv_dtype == GQA_KV_FP8_E4M3FN || kv_dtype == GQA_KV_INT8;
    const bool host_scales = kv8 && k_scales == nullptr;
    a.k_scales = kv8 ? k_scales : nullptr;
    a.v_scales = kv8 ? v_scales : nullptr;
    a.n_scales = n_scales;
    a.v_scale = host_scales ? v_scale : 1.f;
    a.Tq = T, a.B = B, a.Hq = Hq, a.Hkv = Hkv, a.G = Hq / Hkv;
    a.causal = causal != 0;
    a.alpha = host_resolve_scale(scale, D) * 1.4426950408889634f * (host_scales ? k_scale : 1.f);
    a.wait_limit_ns = host_wait_limit_ns();
    a.fault_mode = host_fault_mode();
    a.err = host_error_word(dev);
    cudaStream_t cs = reinterpret_cast<cudaStream_t>(stream);
#define GQA_PREFILL_KVT(KVT) \
    (D == 64 ? launch_prefill<KVT, 64, 64>(a, cs) : launch_prefill<KVT, 128, 128>(a, cs))
    switch (kv_dtype) {
        case GQA_KV_BF16: return GQA_PREFILL_KVT(GQA_KV_BF16);
        case GQA_KV_FP8_E4M3FN: return GQA_PREFILL_KVT(GQA_KV_FP8_E4M3FN);
        case GQA_KV_INT8: return GQA_PREFILL_KVT(GQA_KV_INT8);
        default: return GQA_PREFILL_KVT(GQA_KV_INT4);
    }
#undef GQA_PREFILL_KVT
}
