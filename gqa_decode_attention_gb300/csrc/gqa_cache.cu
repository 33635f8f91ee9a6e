// gqa_cache.cu -- writing a paged K/V cache (gqa_paged_append) and reading it
// back dense (gqa_paged_gather).
//
// Both are streams: every element is read once and written once with a few
// operations in between, so HBM bounds a prompt and the launch bounds a decode
// step.  What matters is that the loads do not wait for the index work (the
// request of a token, its position, its page), and that each thread moves
// 16-byte pieces.
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <cmath>

#include "gqa_common.cuh"
#include "gqa_host.h"

namespace gqa {
namespace {

struct AppendArgs {
    const __nv_bfloat16 *q, *k, *v;  // [T, heads, D], token strides below
    long long q_stride, k_stride, v_stride;
    __nv_bfloat16 *q_out;  // [T, Hq, D]
    uint8_t *k_pool, *v_pool;
    __half *params;  // 4-bit pools: [num_pages, page_size, Hkv, 4]
    float k_inv, v_inv;  // 8-bit pools: 1 / scale, used when k_scales is null
    const float *k_scales, *v_scales;
    int n_scales;
    const int32_t *page_table, *seq_lens;
    const int32_t *cu_tokens;  // [B + 1] or null: T / B tokens a request
    const float *cos_sin;      // [max_pos, rot_dim]
    int rot_dim, max_pos, interleaved;
    int T, B, Hq, Hkv, page_size, pages_per_req, num_pages;
    unsigned *err;
};

struct GatherArgs {
    const uint8_t *k_pool, *v_pool;
    const __half *params;
    float k_scale, v_scale;
    const float *k_scales, *v_scales;
    int n_scales;
    const int32_t *page_table, *seq_lens, *starts;
    __nv_bfloat16 *k_out, *v_out;  // [B, rows, Hkv, D]
    int B, rows, Hkv, page_size, pages_per_req, num_pages;
    unsigned *err;
};

__device__ __forceinline__ void unpack8(const uint4 &w, float (&x)[8]) {
    const uint32_t r[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        x[2 * i] = __uint_as_float(r[i] << 16);
        x[2 * i + 1] = __uint_as_float(r[i] & 0xffff0000u);
    }
}

__device__ __forceinline__ uint4 pack8(const float (&x)[8]) {
    return make_uint4(pack_bf16x2(x[0], x[1]), pack_bf16x2(x[2], x[3]), pack_bf16x2(x[4], x[5]),
                      pack_bf16x2(x[6], x[7]));
}

// Two fp32 values as E4M3FN codes (low byte: lo), rounded to nearest even,
// values past +-448 saturated, NaN kept.
__device__ __forceinline__ uint32_t e4m3x2_from_f32(float lo, float hi) {
    uint16_t r;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
    return r;
}

// Symmetric int8 code of x * inv: nearest even, clamped to +-127, NaN as 0.
__device__ __forceinline__ uint32_t int8_code(float x, float inv) {
    float y = rintf(__fmul_rn(x, inv));
    y = y == y ? fminf(fmaxf(y, -127.f), 127.f) : 0.f;
    return uint32_t(int(y)) & 0xffu;
}

constexpr float kF16Max = 65504.f;

// A finite value within the range of fp16 (a 4-bit row's scale and zero are
// fp16): NaN counts as 0, larger values as +-65504.
__device__ __forceinline__ float int4_input(float x) { return x == x ? fminf(fmaxf(x, -kF16Max), kF16Max) : 0.f; }

// ------------------------------------------------------------------ append
//
// One item: 16 elements of a token's head (two 16-byte pieces), which hold
// whole rotation pairs: slot s of a head takes the pieces at 8 s and
// rot / 2 + 8 s (pairs i, i + rot / 2), or the 16 neighbours at 16 s
// (neighbouring pairs, and the elements past rot_dim).  Items of a token run
// over its q, k and v heads; a CTA of 128 threads holds 128 U of them, U a
// thread.  The threads of one head are neighbours in a warp, which is where a
// 4-bit row's minimum and maximum are reduced.  The slot is the same for all
// of a thread's items, so it loads its cosines and sines once.
//
// All U items are loaded before the token's request, position and page are
// looked up, so their latency overlaps that chain of dependent loads.
//
// The rotation is rounded after every product and sum (no fused multiply-add):
// the codes of an 8-bit or 4-bit cache then do not depend on how a compiler
// contracts the expression, and a plain fp32 computation of the same formula
// gives the same bytes.
constexpr int kAppendThreads = 128;

template <int D, int KVT, int U>
__global__ void __launch_bounds__(kAppendThreads) gqa_paged_append_kernel(const AppendArgs a) {
    constexpr int SLOTS = D / 16;
    const int t = blockIdx.x;
    const int lane = threadIdx.x & 31;
    const int items = (a.Hq + 2 * a.Hkv) * SLOTS;
    const int item0 = blockIdx.y * (kAppendThreads * U) + threadIdx.x;
    const int s = threadIdx.x % SLOTS;
    const bool rotated = 16 * s < a.rot_dim;
    const bool halves = rotated && !a.interleaved;
    const int off_a = halves ? 8 * s : 16 * s;
    const int off_b = halves ? a.rot_dim / 2 + 8 * s : 16 * s + 8;

    pdl_wait_primary();  // inputs may be written by the previous kernel in the stream

    uint4 wa[U], wb[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
        const int item = item0 + u * kAppendThreads;
        const int h = item / SLOTS;
        const __nv_bfloat16 *src = h < a.Hq           ? a.q + (long long)t * a.q_stride + h * D
                                   : h < a.Hq + a.Hkv ? a.k + (long long)t * a.k_stride + (h - a.Hq) * D
                                                      : a.v + (long long)t * a.v_stride + (h - a.Hq - a.Hkv) * D;
        wa[u] = wb[u] = make_uint4(0, 0, 0, 0);
        if (item < items) {
            wa[u] = *reinterpret_cast<const uint4 *>(src + off_a);
            wb[u] = *reinterpret_cast<const uint4 *>(src + off_b);
        }
    }

    // the token's request: the number of requests that end at or before it
    int b, first, count;
    if (a.cu_tokens == nullptr) {
        count = a.T / a.B;
        b = t / count;
        first = b * count;
    } else {
        int lo = 0, n = a.B;
        while (n > 0) {
            const int step = (n + 31) / 32;
            const int p = (lane + 1) * step - 1;
            const bool past = p < n && __ldg(a.cu_tokens + lo + p + 1) <= t;
            const int c = __popc(__ballot_sync(0xffffffffu, past));
            lo += c * step;
            n = min(step - 1, n - c * step);
        }
        b = lo;
        if (b >= a.B) return;  // a row behind the last request
        first = __ldg(a.cu_tokens + b);
        count = __ldg(a.cu_tokens + b + 1) - first;
    }
    const int cap = a.pages_per_req * a.page_size;
    const int len = __ldg(a.seq_lens + b);
    const long long pos_ll = (long long)len - count + (t - first);
    if (t < first || pos_ll < 0 || pos_ll >= cap || (a.rot_dim > 0 && pos_ll >= a.max_pos)) {
        if (threadIdx.x == 0) flag_error(a.err, kErrIndex);
        return;
    }
    const int pos = int(pos_ll);
    const int page = __ldg(a.page_table + (long long)b * a.pages_per_req + pos / a.page_size);
    float cs[8], sn[8];
    if (rotated) {
        const float4 *row = reinterpret_cast<const float4 *>(a.cos_sin + (long long)pos * a.rot_dim + 8 * s);
        const float4 *row2 = reinterpret_cast<const float4 *>(a.cos_sin + (long long)pos * a.rot_dim + a.rot_dim / 2 + 8 * s);
        const float4 c0 = __ldg(row), c1 = __ldg(row + 1), s0 = __ldg(row2), s1 = __ldg(row2 + 1);
        cs[0] = c0.x, cs[1] = c0.y, cs[2] = c0.z, cs[3] = c0.w, cs[4] = c1.x, cs[5] = c1.y, cs[6] = c1.z, cs[7] = c1.w;
        sn[0] = s0.x, sn[1] = s0.y, sn[2] = s0.z, sn[3] = s0.w, sn[4] = s1.x, sn[5] = s1.y, sn[6] = s1.z, sn[7] = s1.w;
    }
    const bool page_ok = page >= 0 && page < a.num_pages;
    if (!page_ok && threadIdx.x == 0) flag_error(a.err, kErrIndex);
    const long long row = page_ok ? (long long)page * a.page_size + pos % a.page_size : 0;

#pragma unroll
    for (int u = 0; u < U; ++u) {
        const int item = item0 + u * kAppendThreads;
        const int h = item / SLOTS;
        const bool is_q = h < a.Hq;
        const bool is_v = h >= a.Hq + a.Hkv;
        const int g = is_v ? h - a.Hq - a.Hkv : h - a.Hq;  // KV head
        const bool store_kv = item < items && !is_q && page_ok;
        float x[8], y[8];
        unpack8(wa[u], x);
        unpack8(wb[u], y);
        if (rotated && !is_v) {
            if (a.interleaved) {
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const float x0 = x[2 * i], x1 = x[2 * i + 1], y0 = y[2 * i], y1 = y[2 * i + 1];
                    x[2 * i] = __fsub_rn(__fmul_rn(x0, cs[i]), __fmul_rn(x1, sn[i]));
                    x[2 * i + 1] = __fadd_rn(__fmul_rn(x1, cs[i]), __fmul_rn(x0, sn[i]));
                    y[2 * i] = __fsub_rn(__fmul_rn(y0, cs[i + 4]), __fmul_rn(y1, sn[i + 4]));
                    y[2 * i + 1] = __fadd_rn(__fmul_rn(y1, cs[i + 4]), __fmul_rn(y0, sn[i + 4]));
                }
            } else {
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    const float x0 = x[i], y0 = y[i];
                    x[i] = __fsub_rn(__fmul_rn(x0, cs[i]), __fmul_rn(y0, sn[i]));
                    y[i] = __fadd_rn(__fmul_rn(y0, cs[i]), __fmul_rn(x0, sn[i]));
                }
            }
        }
        if (is_q) {
            __nv_bfloat16 *dst = a.q_out + ((long long)t * a.Hq + h) * D;
            *reinterpret_cast<uint4 *>(dst + off_a) = pack8(x);
            *reinterpret_cast<uint4 *>(dst + off_b) = pack8(y);
        }
        uint8_t *pool = is_v ? a.v_pool : a.k_pool;
        const long long head_row = row * a.Hkv + g;
        if constexpr (KVT == GQA_KV_BF16) {
            if (store_kv) {
                __nv_bfloat16 *dst = reinterpret_cast<__nv_bfloat16 *>(pool) + head_row * D;
                *reinterpret_cast<uint4 *>(dst + off_a) = pack8(x);
                *reinterpret_cast<uint4 *>(dst + off_b) = pack8(y);
            }
        } else if constexpr (KVT == GQA_KV_INT4) {
            // the row's range over the D / 16 threads of the head (every lane
            // takes part: a warp can hold q heads beside k heads)
            float mn = INFINITY, mx = -INFINITY;
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                x[i] = int4_input(x[i]);
                y[i] = int4_input(y[i]);
                mn = fminf(mn, fminf(x[i], y[i]));
                mx = fmaxf(mx, fmaxf(x[i], y[i]));
            }
#pragma unroll
            for (int o = 1; o < SLOTS; o *= 2) {
                mn = fminf(mn, __shfl_xor_sync(0xffffffffu, mn, o));
                mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, o));
            }
            const __half zero_h = __float2half_rn(mn);
            const float zero = __half2float(zero_h);
            const __half step_h = __float2half_rn(fmaxf(__fmul_rn(__fsub_rn(mx, zero), 1.f / 15.f), 0.f));
            const float step = __half2float(step_h);
            const float inv = step > 0.f ? __fdiv_rn(1.f, step) : 0.f;
            uint32_t ca = 0, cb = 0;
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const float ux = fminf(fmaxf(rintf(__fmul_rn(__fsub_rn(x[i], zero), inv)), 0.f), 15.f);
                const float uy = fminf(fmaxf(rintf(__fmul_rn(__fsub_rn(y[i], zero), inv)), 0.f), 15.f);
                ca |= uint32_t(ux) << (4 * i);
                cb |= uint32_t(uy) << (4 * i);
            }
            if (store_kv) {
                uint8_t *dst = pool + head_row * (D / 2);
                *reinterpret_cast<uint32_t *>(dst + off_a / 2) = ca;
                *reinterpret_cast<uint32_t *>(dst + off_b / 2) = cb;
                if (s == 0)
                    *reinterpret_cast<__half2 *>(a.params + head_row * 4 + (is_v ? 2 : 0)) = __halves2half2(step_h, zero_h);
            }
        } else if (store_kv) {
            const float *scales = is_v ? a.v_scales : a.k_scales;
            const float inv = scales != nullptr ? __fdiv_rn(1.f, __ldg(scales + (a.n_scales > 1 ? g : 0)))
                                                : (is_v ? a.v_inv : a.k_inv);
            uint32_t c[4];
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const float *p = j < 2 ? x + 4 * j : y + 4 * (j - 2);
                if constexpr (KVT == GQA_KV_FP8_E4M3FN)
                    c[j] = e4m3x2_from_f32(__fmul_rn(p[0], inv), __fmul_rn(p[1], inv)) |
                           e4m3x2_from_f32(__fmul_rn(p[2], inv), __fmul_rn(p[3], inv)) << 16;
                else
                    c[j] = int8_code(p[0], inv) | int8_code(p[1], inv) << 8 | int8_code(p[2], inv) << 16 |
                           int8_code(p[3], inv) << 24;
            }
            uint8_t *dst = pool + head_row * D;
            *reinterpret_cast<uint2 *>(dst + off_a) = make_uint2(c[0], c[1]);
            *reinterpret_cast<uint2 *>(dst + off_b) = make_uint2(c[2], c[3]);
        }
    }
}

// Launches with the programmatic-dependent-launch attribute: the CTAs may be
// scheduled while the previous kernel drains and wait for it before reading.
template <class Args>
cudaError_t launch_pdl(void (*kern)(Args), const Args &a, dim3 grid, int threads, cudaStream_t stream) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = dim3(threads);
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kern, a);
}

template <int D, int KVT>
cudaError_t launch_append(const AppendArgs &a, cudaStream_t stream) {
    constexpr int U = 4;
    const int items = (a.Hq + 2 * a.Hkv) * (D / 16);
    const int per = kAppendThreads * U;
    return launch_pdl(gqa_paged_append_kernel<D, KVT, U>, a, dim3(unsigned(a.T), unsigned((items + per - 1) / per)),
                      kAppendThreads, stream);
}

// ------------------------------------------------------------------ gather
//
// A unit is 8 elements of K and the same 8 of V: one 16-byte store each.  The
// units of a request are contiguous in the output, so a CTA takes a run of
// them, neighbouring threads write neighbouring pieces, and a thread has the
// loads of all its units in flight before it converts the first.
constexpr int kGatherThreads = 256;
constexpr int kGatherUnits = 4;

template <int KVT>
__device__ __forceinline__ uint4 gather_load(const uint8_t *pool, long long elem) {
    if constexpr (KVT == GQA_KV_BF16) return __ldg(reinterpret_cast<const uint4 *>(pool + elem * 2));
    if constexpr (KVT == GQA_KV_INT4) return make_uint4(__ldg(reinterpret_cast<const unsigned int *>(pool + elem / 2)), 0, 0, 0);
    const uint2 x = __ldg(reinterpret_cast<const uint2 *>(pool + elem));
    return make_uint4(x.x, x.y, 0, 0);
}

// value = code * scale + zero in fp32 (the product is exact for 4-bit codes
// and fp16 scales; 8-bit values round once here and once to bf16)
template <int KVT>
__device__ __forceinline__ uint4 gather_value(const uint4 &w, float scale, float zero) {
    if constexpr (KVT == GQA_KV_BF16) return w;
    float x[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        if constexpr (KVT == GQA_KV_INT4) {
            x[i] = __fadd_rn(__fmul_rn(float((w.x >> (4 * i)) & 15u), scale), zero);
        } else {
            const uint32_t word = i < 4 ? w.x : w.y;
            if constexpr (KVT == GQA_KV_INT8) {
                x[i] = __fmul_rn(float(int8_t(word >> (8 * (i & 3)))), scale);
            } else if ((i & 1) == 0) {
                const uint32_t h2 = e4m3x2_to_f16x2(uint16_t(word >> (8 * (i & 3))));
                const float2 f = __half22float2(*reinterpret_cast<const __half2 *>(&h2));
                x[i] = __fmul_rn(f.x, scale);
                x[i + 1] = __fmul_rn(f.y, scale);
            }
        }
    }
    return pack8(x);
}

template <int D, int KVT>
__global__ void __launch_bounds__(kGatherThreads) gqa_paged_gather_dense_kernel(const GatherArgs a) {
    const int b = blockIdx.y;
    const int upt = a.Hkv * (D / 8);  // units of a token
    pdl_wait_primary();
    const int cap = a.pages_per_req * a.page_size;
    const int len0 = __ldg(a.seq_lens + b), start0 = a.starts != nullptr ? __ldg(a.starts + b) : 0;
    const int len = min(max(len0, 0), cap), start = max(start0, 0);
    const int n = min(len - start, a.rows);
    if (threadIdx.x == 0 && blockIdx.x == 0 && (len != len0 || start != start0)) flag_error(a.err, kErrIndex);
    const long long unit0 = (long long)blockIdx.x * (kGatherThreads * kGatherUnits);
    if (n <= 0 || unit0 >= (long long)n * upt) return;
    const int tok0 = int(unit0 / upt);
    const int rem0 = int(unit0 - (long long)tok0 * upt);

    uint4 kw[kGatherUnits], vw[kGatherUnits];
    float ks[kGatherUnits], kz[kGatherUnits], vs[kGatherUnits], vz[kGatherUnits];
    bool there[kGatherUnits];
    bool bad = false;
#pragma unroll
    for (int i = 0; i < kGatherUnits; ++i) {
        const unsigned r = unsigned(rem0) + threadIdx.x + i * kGatherThreads;
        const int j = tok0 + int(r / unsigned(upt));  // output row
        const int u = int(r % unsigned(upt));
        there[i] = j < n;
        kw[i] = vw[i] = make_uint4(0, 0, 0, 0);
        ks[i] = kz[i] = vs[i] = vz[i] = 0.f;
        if (!there[i]) continue;
        const int pos = start + j;
        const int page = __ldg(a.page_table + (long long)b * a.pages_per_req + pos / a.page_size);
        if (page < 0 || page >= a.num_pages) {
            bad = true;  // the row reads as zeros
            continue;
        }
        const long long head_row = ((long long)page * a.page_size + pos % a.page_size) * a.Hkv + u / (D / 8);
        const long long elem = head_row * D + 8 * (u % (D / 8));
        kw[i] = gather_load<KVT>(a.k_pool, elem);
        vw[i] = gather_load<KVT>(a.v_pool, elem);
        if constexpr (KVT == GQA_KV_INT4) {
            const uint2 p = __ldg(reinterpret_cast<const uint2 *>(a.params + head_row * 4));
            const float2 pk = __half22float2(*reinterpret_cast<const __half2 *>(&p.x));
            const float2 pv = __half22float2(*reinterpret_cast<const __half2 *>(&p.y));
            ks[i] = pk.x, kz[i] = pk.y, vs[i] = pv.x, vz[i] = pv.y;
        } else if constexpr (KVT != GQA_KV_BF16) {
            const int si = a.n_scales > 1 ? u / (D / 8) : 0;
            ks[i] = a.k_scales != nullptr ? __ldg(a.k_scales + si) : a.k_scale;
            vs[i] = a.v_scales != nullptr ? __ldg(a.v_scales + si) : a.v_scale;
        }
    }
    if (bad) flag_error(a.err, kErrIndex);
#pragma unroll
    for (int i = 0; i < kGatherUnits; ++i) {
        if (!there[i]) continue;
        const long long o = ((long long)b * a.rows * upt + unit0 + threadIdx.x + i * kGatherThreads) * 8;
        *reinterpret_cast<uint4 *>(a.k_out + o) = gather_value<KVT>(kw[i], ks[i], kz[i]);
        *reinterpret_cast<uint4 *>(a.v_out + o) = gather_value<KVT>(vw[i], vs[i], vz[i]);
    }
}

template <int D, int KVT>
cudaError_t launch_gather(const GatherArgs &a, cudaStream_t stream) {
    const long long units = (long long)a.rows * a.Hkv * (D / 8);
    const long long per = kGatherThreads * kGatherUnits;
    return launch_pdl(gqa_paged_gather_dense_kernel<D, KVT>, a, dim3(unsigned((units + per - 1) / per), unsigned(a.B)),
                      kGatherThreads, stream);
}

// Checks shared by both entry points: pool type, scales, parameters.
gqa_status check_cache(int kv_dtype, const void *params, float k_scale, float v_scale, const float *k_scales,
                       const float *v_scales, int n_scales, int Hkv) {
    if (kv_dtype < GQA_KV_BF16 || kv_dtype > GQA_KV_INT4) return GQA_ERR_INVALID_ARG;
    if ((kv_dtype == GQA_KV_INT4) != (params != nullptr)) return GQA_ERR_INVALID_ARG;
    const bool kv8 = kv_dtype == GQA_KV_FP8_E4M3FN || kv_dtype == GQA_KV_INT8;
    if (k_scales != nullptr || v_scales != nullptr) {
        if (!kv8 || k_scales == nullptr || v_scales == nullptr || (n_scales != 1 && n_scales != Hkv))
            return GQA_ERR_INVALID_ARG;
        if (!host_aligned(k_scales, 4) || !host_aligned(v_scales, 4)) return GQA_ERR_ALIGNMENT;
    } else if (kv8 && (!std::isfinite(k_scale) || !std::isfinite(v_scale))) {
        return GQA_ERR_INVALID_ARG;
    }
    return host_aligned(params, 8) ? GQA_OK : GQA_ERR_ALIGNMENT;
}

}  // namespace
}  // namespace gqa

using namespace gqa;

#define GQA_CACHE_DISPATCH(FN)                                                                    \
    (kv_dtype == GQA_KV_BF16         ? (D == 64 ? FN<64, GQA_KV_BF16>(a, cs) : FN<128, GQA_KV_BF16>(a, cs))   \
     : kv_dtype == GQA_KV_FP8_E4M3FN ? (D == 64 ? FN<64, GQA_KV_FP8_E4M3FN>(a, cs)                            \
                                                : FN<128, GQA_KV_FP8_E4M3FN>(a, cs))                          \
     : kv_dtype == GQA_KV_INT8       ? (D == 64 ? FN<64, GQA_KV_INT8>(a, cs) : FN<128, GQA_KV_INT8>(a, cs))   \
                                     : (D == 64 ? FN<64, GQA_KV_INT4>(a, cs) : FN<128, GQA_KV_INT4>(a, cs)))

extern "C" gqa_status gqa_paged_append(const void *q, long long q_stride, void *q_out, const void *k,
                                       long long k_stride, const void *v, long long v_stride, int kv_dtype,
                                       void *k_pool, void *v_pool, void *kv_params, float k_scale, float v_scale,
                                       const float *k_scales, const float *v_scales, int n_scales,
                                       const int32_t *page_table, const int32_t *seq_lens,
                                       const int32_t *cu_tokens, const float *cos_sin, int rot_dim, int max_pos,
                                       int interleaved, int T, int B, int Hq, int Hkv, int D, int page_size,
                                       int pages_per_req, int num_pages, gqa_stream_t stream) {
    gqa_status st = host_check_pages(B, Hkv, D, page_size, pages_per_req, num_pages);
    if (st != GQA_OK) return st;
    const bool has_q = q != nullptr || q_out != nullptr;
    if (T < 0 || (has_q && (Hq < 1 || q == nullptr || q_out == nullptr))) return GQA_ERR_INVALID_ARG;
    if (cu_tokens == nullptr && T % B != 0) return GQA_ERR_INVALID_ARG;
    if (rot_dim < 0 || rot_dim > D || rot_dim % 16 != 0) return GQA_ERR_INVALID_ARG;
    if (rot_dim > 0 && (cos_sin == nullptr || max_pos < 1)) return GQA_ERR_INVALID_ARG;
    st = check_cache(kv_dtype, kv_params, k_scale, v_scale, k_scales, v_scales, n_scales, Hkv);
    if (st != GQA_OK) return st;
    const bool kv8 = kv_dtype == GQA_KV_FP8_E4M3FN || kv_dtype == GQA_KV_INT8;
    if (kv8 && k_scales == nullptr && (!(k_scale > 0.f) || !(v_scale > 0.f))) return GQA_ERR_INVALID_ARG;
    if (k_pool == nullptr || v_pool == nullptr || page_table == nullptr || seq_lens == nullptr ||
        (T > 0 && (k == nullptr || v == nullptr)))
        return GQA_ERR_INVALID_ARG;
    const long long heads_max = 1 << 20;
    if (Hkv > heads_max || (has_q && Hq > heads_max)) return GQA_ERR_UNSUPPORTED;
    if (k_stride < (long long)Hkv * D || v_stride < (long long)Hkv * D || (has_q && q_stride < (long long)Hq * D))
        return GQA_ERR_INVALID_ARG;
    if (k_stride % 8 != 0 || v_stride % 8 != 0 || (has_q && q_stride % 8 != 0)) return GQA_ERR_ALIGNMENT;
    if (!host_aligned(q, 16) || !host_aligned(q_out, 16) || !host_aligned(k, 16) || !host_aligned(v, 16) ||
        !host_aligned(k_pool, 16) || !host_aligned(v_pool, 16) || !host_aligned(cos_sin, 16) ||
        !host_aligned(page_table, 4) || !host_aligned(seq_lens, 4) || !host_aligned(cu_tokens, 4))
        return GQA_ERR_ALIGNMENT;
    if (T == 0) return GQA_OK;
    int dev = 0;
    if (!host_current_device(&dev)) return GQA_ERR_CUDA;
    AppendArgs a = {};
    a.q = static_cast<const __nv_bfloat16 *>(q);
    a.k = static_cast<const __nv_bfloat16 *>(k);
    a.v = static_cast<const __nv_bfloat16 *>(v);
    a.q_stride = q_stride;
    a.k_stride = k_stride;
    a.v_stride = v_stride;
    a.q_out = static_cast<__nv_bfloat16 *>(q_out);
    a.k_pool = static_cast<uint8_t *>(k_pool);
    a.v_pool = static_cast<uint8_t *>(v_pool);
    a.params = static_cast<__half *>(kv_params);
    a.k_inv = 1.0f / k_scale;
    a.v_inv = 1.0f / v_scale;
    a.k_scales = k_scales;
    a.v_scales = v_scales;
    a.n_scales = n_scales;
    a.page_table = page_table;
    a.seq_lens = seq_lens;
    a.cu_tokens = cu_tokens;
    a.cos_sin = cos_sin;
    a.rot_dim = rot_dim;
    a.max_pos = max_pos;
    a.interleaved = interleaved != 0;
    a.T = T;
    a.B = B;
    a.Hq = has_q ? Hq : 0;
    a.Hkv = Hkv;
    a.page_size = page_size;
    a.pages_per_req = pages_per_req;
    a.num_pages = num_pages;
    a.err = host_error_word(dev);
    cudaStream_t cs = reinterpret_cast<cudaStream_t>(stream);
    if (GQA_CACHE_DISPATCH(launch_append) != cudaSuccess) {
        cudaGetLastError();
        return GQA_ERR_CUDA;
    }
    return GQA_OK;
}

extern "C" gqa_status gqa_paged_gather(int kv_dtype, const void *k_pool, const void *v_pool, const void *kv_params,
                                       float k_scale, float v_scale, const float *k_scales, const float *v_scales,
                                       int n_scales, const int32_t *page_table, const int32_t *seq_lens,
                                       const int32_t *starts, void *k_out, void *v_out, int B, int rows, int Hkv,
                                       int D, int page_size, int pages_per_req, int num_pages, gqa_stream_t stream) {
    gqa_status st = host_check_pages(B, Hkv, D, page_size, pages_per_req, num_pages);
    if (st != GQA_OK) return st;
    if (rows < 0) return GQA_ERR_INVALID_ARG;
    st = check_cache(kv_dtype, kv_params, k_scale, v_scale, k_scales, v_scales, n_scales, Hkv);
    if (st != GQA_OK) return st;
    if (k_pool == nullptr || v_pool == nullptr || page_table == nullptr || seq_lens == nullptr ||
        (rows > 0 && (k_out == nullptr || v_out == nullptr)))
        return GQA_ERR_INVALID_ARG;
    if (Hkv > (1 << 20) || (long long)rows * Hkv * (D / 8) >= (1LL << 40)) return GQA_ERR_UNSUPPORTED;
    if (!host_aligned(k_pool, 16) || !host_aligned(v_pool, 16) || !host_aligned(k_out, 16) ||
        !host_aligned(v_out, 16) || !host_aligned(page_table, 4) || !host_aligned(seq_lens, 4) ||
        !host_aligned(starts, 4))
        return GQA_ERR_ALIGNMENT;
    if (rows == 0) return GQA_OK;
    int dev = 0;
    if (!host_current_device(&dev)) return GQA_ERR_CUDA;
    GatherArgs a = {};
    a.k_pool = static_cast<const uint8_t *>(k_pool);
    a.v_pool = static_cast<const uint8_t *>(v_pool);
    a.params = static_cast<const __half *>(kv_params);
    a.k_scale = k_scale;
    a.v_scale = v_scale;
    a.k_scales = k_scales;
    a.v_scales = v_scales;
    a.n_scales = n_scales;
    a.page_table = page_table;
    a.seq_lens = seq_lens;
    a.starts = starts;
    a.k_out = static_cast<__nv_bfloat16 *>(k_out);
    a.v_out = static_cast<__nv_bfloat16 *>(v_out);
    a.B = B;
    a.rows = rows;
    a.Hkv = Hkv;
    a.page_size = page_size;
    a.pages_per_req = pages_per_req;
    a.num_pages = num_pages;
    a.err = host_error_word(dev);
    cudaStream_t cs = reinterpret_cast<cudaStream_t>(stream);
    if (GQA_CACHE_DISPATCH(launch_gather) != cudaSuccess) {
        cudaGetLastError();
        return GQA_ERR_CUDA;
    }
    return GQA_OK;
}
