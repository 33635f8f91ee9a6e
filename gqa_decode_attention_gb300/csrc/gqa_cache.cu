// gqa_cache.cu -- writing a paged K/V cache (gqa_paged_append) and reading it
// back dense (gqa_paged_gather).
//
// Both are streams: every element is read once and written once with a few
// operations in between, so HBM bounds a prompt and the launch bounds a decode
// step.  What matters is that the loads do not wait for the index work (the
// request of a token, its position, its page), and that each thread moves
// 16-byte pieces.  Measured on GB300: 37K prompt tokens of 64/8 heads of 128
// into an FP8 cache 226 us, 96 % of the copy peak; one decode step of 32 such
// requests 3.3 us; 103K tokens of 8 heads of 128 gathered from a 4-bit cache
// 110 us -- four fifths of its bytes are writes, and a plain fill of the same
// size takes 109 to 113 us.
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
    int lanes, heads_per_cta;  // heads of a token side by side in a CTA, and all that it walks over
    int tokens;                // of a CTA
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
    int tokens;  // of a warp
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

// Conversions between small integers and fp32 go through the mantissa (the
// sum with 2^23, or 1.5 * 2^23 for signed values, rounds to the nearest even
// integer and holds it in its low bits): the conversion instructions run at a
// quarter of that rate.
constexpr float kMagic = 8388608.f, kMagicSigned = 12582912.f;

// Symmetric int8 code of x * inv: nearest even, clamped to +-127, NaN as 0.
__device__ __forceinline__ uint32_t int8_code(float x, float inv) {
    const float y = __fmul_rn(x, inv);
    const float c = y == y ? fminf(fmaxf(y, -127.f), 127.f) : 0.f;
    return __float_as_uint(c + kMagicSigned) & 0xffu;
}

// Code in 0..15 of (x - zero) * inv, nearest even.
__device__ __forceinline__ uint32_t int4_code(float x, float zero, float inv) {
    const float y = fminf(fmaxf(__fmul_rn(__fsub_rn(x, zero), inv), 0.f), 15.f);
    return __float_as_uint(y + kMagic) & 15u;
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
// (neighbouring pairs, and the elements past rot_dim).  A CTA holds a run of
// tokens; `lanes` heads of a token lie side by side (the slots of a head on
// neighbouring threads, which is where a 4-bit row's minimum and maximum are
// reduced), and a thread walks over the token's heads in steps of `lanes`: its
// slot and token stay, so it loads its cosines and sines once a token.
//
// A token's request, position and page are a chain of dependent loads, some
// microseconds long.  So a CTA looks up all of its tokens at once, a warp a
// token, with the first heads' loads already in flight, and holds several
// groups of tokens when there are enough for that (one group a CTA ran 24
// heads of 64, 20K tokens, at 2 TB/s).
//
// The rotation is rounded after every product and sum (no fused multiply-add):
// the codes of an 8-bit or 4-bit cache then do not depend on how a compiler
// contracts the expression, and a plain fp32 computation of the same formula
// gives the same bytes.
constexpr int kAppendThreads = 256;
constexpr int kAppendBatch = 3;  // heads a thread has in flight
constexpr int kAppendTokens = 128;  // most tokens of a CTA

struct AppendToken {
    long long row;  // pool row; -1: no place for K and V; -2: skipped whole
    int pos;
};

// The request that holds row t: the number of requests, from `lo` on, that end
// at or before it.  Called by a whole warp with the same arguments.
__device__ __forceinline__ int request_of(const int32_t *cu, int lo, int B, int t) {
    const int lane = threadIdx.x & 31;
    int n = B - lo;
    while (n > 0) {
        const int step = (n + 31) / 32;
        const int p = (lane + 1) * step - 1;
        const bool past = p < n && __ldg(cu + lo + p + 1) <= t;
        const int c = __popc(__ballot_sync(0xffffffffu, past));
        lo += c * step;
        n = min(step - 1, n - c * step);
    }
    return lo;
}

template <int D, int KVT>
__global__ void __launch_bounds__(kAppendThreads, 3) gqa_paged_append_kernel(const AppendArgs a) {
    constexpr int SLOTS = D / 16;
    __shared__ AppendToken tokens[kAppendTokens];
    const int per_token = SLOTS * a.lanes;  // threads
    const int side = kAppendThreads / per_token;  // tokens side by side
    const int t0 = blockIdx.x * a.tokens, n_tok = min(a.tokens, a.T - t0);
    const int mine = threadIdx.x / per_token;
    const int s = threadIdx.x % SLOTS;
    const int heads = a.Hq + 2 * a.Hkv;
    const int h_first = blockIdx.y * a.heads_per_cta + threadIdx.x % per_token / SLOTS;
    const int h_end = min(heads, (int(blockIdx.y) + 1) * a.heads_per_cta);
    const bool rotated = 16 * s < a.rot_dim;
    const bool halves = rotated && !a.interleaved;
    const int off_a = halves ? 8 * s : 16 * s;
    const int off_b = halves ? a.rot_dim / 2 + 8 * s : 16 * s + 8;

    pdl_wait_primary();  // inputs may be written by the previous kernel in the stream

    uint4 wa[kAppendBatch], wb[kAppendBatch];
    auto load = [&](int t, int h0) {
#pragma unroll
        for (int u = 0; u < kAppendBatch; ++u) {
            const int h = h0 + u * a.lanes;
            const __nv_bfloat16 *src = h < a.Hq           ? a.q + (long long)t * a.q_stride + h * D
                                       : h < a.Hq + a.Hkv ? a.k + (long long)t * a.k_stride + (h - a.Hq) * D
                                                          : a.v + (long long)t * a.v_stride + (h - a.Hq - a.Hkv) * D;
            wa[u] = wb[u] = make_uint4(0, 0, 0, 0);
            if (h < h_end && t < t0 + n_tok) {
                wa[u] = *reinterpret_cast<const uint4 *>(src + off_a);
                wb[u] = *reinterpret_cast<const uint4 *>(src + off_b);
            }
        }
    };
    load(t0 + mine, h_first);

    const int warp = threadIdx.x >> 5;
    for (int i = warp, b = 0; i < n_tok; i += kAppendThreads / 32) {
        const int t = t0 + i;
        int start, count;
        if (a.cu_tokens == nullptr) {
            count = a.T / a.B;
            b = t / count;
            start = b * count;
        } else {
            b = request_of(a.cu_tokens, b, a.B, t);
            start = b < a.B ? __ldg(a.cu_tokens + b) : 0;
            count = b < a.B ? __ldg(a.cu_tokens + b + 1) - start : 0;
        }
        if ((threadIdx.x & 31) != 0) continue;
        AppendToken tok = {-2, 0};
        bool bad = false;
        if (b < a.B) {  // else a row behind the last request
            const long long pos = (long long)__ldg(a.seq_lens + b) - count + (t - start);
            bad = t < start || pos < 0 || pos >= a.pages_per_req * a.page_size || (a.rot_dim > 0 && pos >= a.max_pos);
            if (!bad) {
                tok.pos = int(pos);
                const int page = __ldg(a.page_table + (long long)b * a.pages_per_req + tok.pos / a.page_size);
                bad = page < 0 || page >= a.num_pages;
                tok.row = bad ? -1 : (long long)page * a.page_size + tok.pos % a.page_size;
            }
        }
        tokens[i] = tok;
        if (bad && blockIdx.y == 0) flag_error(a.err, kErrIndex);
    }
    __syncthreads();

    for (int base = 0; base < n_tok; base += side) {
        const int t = t0 + base + mine;
        const AppendToken tok = base + mine < n_tok ? tokens[base + mine] : AppendToken{-2, 0};
        const bool there = tok.row >= -1;
        if (base > 0) load(t, h_first);
        float cs[8], sn[8];
        if (rotated && there) {
            const float4 *row = reinterpret_cast<const float4 *>(a.cos_sin + (long long)tok.pos * a.rot_dim + 8 * s);
            const float4 *row2 = reinterpret_cast<const float4 *>(a.cos_sin + (long long)tok.pos * a.rot_dim + a.rot_dim / 2 + 8 * s);
            const float4 c0 = __ldg(row), c1 = __ldg(row + 1), s0 = __ldg(row2), s1 = __ldg(row2 + 1);
            cs[0] = c0.x, cs[1] = c0.y, cs[2] = c0.z, cs[3] = c0.w, cs[4] = c1.x, cs[5] = c1.y, cs[6] = c1.z, cs[7] = c1.w;
            sn[0] = s0.x, sn[1] = s0.y, sn[2] = s0.z, sn[3] = s0.w, sn[4] = s1.x, sn[5] = s1.y, sn[6] = s1.z, sn[7] = s1.w;
        } else {
#pragma unroll
            for (int i = 0; i < 8; ++i) cs[i] = 1.f, sn[i] = 0.f;
        }

        // every thread makes the same number of rounds: 4-bit rows are reduced by shuffles
        const int rounds = (a.heads_per_cta + a.lanes * kAppendBatch - 1) / (a.lanes * kAppendBatch);
        for (int round = 0; round < rounds; ++round) {
            const int h0 = h_first + round * kAppendBatch * a.lanes;
            if (round > 0) load(t, h0);
#pragma unroll
            for (int u = 0; u < kAppendBatch; ++u) {
                const int h = h0 + u * a.lanes;
                const bool is_q = h < a.Hq;
                const bool is_v = h >= a.Hq + a.Hkv;
                const int g = is_v ? h - a.Hq - a.Hkv : h - a.Hq;  // KV head
                const bool valid = h < h_end && there;
                const bool store_kv = valid && !is_q && tok.row >= 0;
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
                if (is_q && valid) {
                    __nv_bfloat16 *dst = a.q_out + ((long long)t * a.Hq + h) * D;
                    *reinterpret_cast<uint4 *>(dst + off_a) = pack8(x);
                    *reinterpret_cast<uint4 *>(dst + off_b) = pack8(y);
                }
                uint8_t *pool = is_v ? a.v_pool : a.k_pool;
                const long long head_row = tok.row * a.Hkv + g;
                if constexpr (KVT == GQA_KV_BF16) {
                    if (store_kv) {
                        __nv_bfloat16 *dst = reinterpret_cast<__nv_bfloat16 *>(pool) + head_row * D;
                        *reinterpret_cast<uint4 *>(dst + off_a) = pack8(x);
                        *reinterpret_cast<uint4 *>(dst + off_b) = pack8(y);
                    }
                } else if constexpr (KVT == GQA_KV_INT4) {
                    if (!__any_sync(0xffffffffu, store_kv)) continue;
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
                        ca |= int4_code(x[i], zero, inv) << (4 * i);
                        cb |= int4_code(y[i], zero, inv) << (4 * i);
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

// With enough tokens a CTA walks over all heads of its tokens, with the number
// of heads side by side (a power of two up to 16: 65K tokens of 80 heads of 128
// took 227 us with 16, 237 with 32) that leaves the fewest places of a batch
// empty, and of those the fewest batches; with few tokens (a decode step) the
// heads are spread over the grid, one head a thread.
template <int D, int KVT>
cudaError_t launch_append(AppendArgs a, cudaStream_t stream) {
    constexpr int SLOTS = D / 16;
    const int heads = a.Hq + 2 * a.Hkv;
    int lanes = 1;
    long best = -1;
    for (int n = 1; n <= 16; n *= 2) {
        const long batches = (heads + n * kAppendBatch - 1) / (n * kAppendBatch);
        const long cost = 16 * batches * kAppendBatch * n + batches * heads;
        if (best < 0 || cost < best) best = cost, lanes = n;
    }
    a.lanes = lanes;
    a.heads_per_cta = heads;
    const int side = kAppendThreads / (SLOTS * lanes);
    const long groups = (long(a.T) + side - 1) / side;
    if (groups < 304) a.heads_per_cta = lanes;  // fewer than two CTAs an SM
    // several groups of tokens a CTA where that leaves 16 CTAs an SM
    long per = groups / (16 * 152);
    if (per > kAppendTokens / side) per = kAppendTokens / side;
    a.tokens = side * int(per < 1 ? 1 : per);
    const long ctas = (long(a.T) + a.tokens - 1) / a.tokens;
    return launch_pdl(gqa_paged_append_kernel<D, KVT>, a,
                      dim3(unsigned(ctas), unsigned((heads + a.heads_per_cta - 1) / a.heads_per_cta)), kAppendThreads, stream);
}

// ------------------------------------------------------------------ gather
//
// A warp takes a run of at most 32 tokens of one request; each lane looks up
// one token's pool row.  A unit is 16 elements of a token's K and the same 16 of
// V; neighbouring lanes take neighbouring units, so they read and write
// neighbouring pieces, and a lane has the loads of a batch of units in flight
// before it converts the first.
constexpr int kGatherThreads = 256;
constexpr int kGatherUnits = 2;  // of a lane in flight (4 at four CTAs an SM: 116 us where these take 111)

// Codes of 16 elements: 32 bytes of bf16, 16 of 8-bit codes, 8 of 4-bit codes.
template <int KVT>
struct GatherCodes {
    uint32_t w[KVT == GQA_KV_BF16 ? 8 : KVT == GQA_KV_INT4 ? 2 : 4];
};

template <int KVT>
__device__ __forceinline__ void gather_load(GatherCodes<KVT> &c, const uint8_t *pool, long long elem) {
    if constexpr (KVT == GQA_KV_INT4) {
        const uint2 x = __ldg(reinterpret_cast<const uint2 *>(pool + elem / 2));
        c.w[0] = x.x, c.w[1] = x.y;
    } else {
#pragma unroll
        for (int i = 0; i < (KVT == GQA_KV_BF16 ? 2 : 1); ++i) {
            const uint4 x = __ldg(reinterpret_cast<const uint4 *>(pool + elem * (KVT == GQA_KV_BF16 ? 2 : 1)) + i);
            c.w[4 * i] = x.x, c.w[4 * i + 1] = x.y, c.w[4 * i + 2] = x.z, c.w[4 * i + 3] = x.w;
        }
    }
}

// value = code * scale + zero in fp32 (the product is exact for 4-bit codes
// and fp16 scales; 8-bit values round once here and once to bf16); elements
// 8 half .. 8 half + 7
template <int KVT>
__device__ __forceinline__ uint4 gather_value(const GatherCodes<KVT> &c, int half, float scale, float zero) {
    if constexpr (KVT == GQA_KV_BF16) {
        return make_uint4(c.w[4 * half], c.w[4 * half + 1], c.w[4 * half + 2], c.w[4 * half + 3]);
    } else {
        float x[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            if constexpr (KVT == GQA_KV_INT4) {
                x[i] = fmaf(__uint_as_float((c.w[half] >> (4 * i) & 15u) | 0x4b000000u) - kMagic, scale, zero);
            } else {
                const uint32_t word = c.w[2 * half + i / 4];
                if constexpr (KVT == GQA_KV_INT8) {
                    const uint32_t byte = (word >> (8 * (i & 3)) & 0xffu) ^ 0x80u;  // code + 128
                    x[i] = __fmul_rn(__uint_as_float(byte | 0x4b000000u) - (kMagic + 128.f), scale);
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
}

template <int D, int KVT>
__global__ void __launch_bounds__(kGatherThreads, 5) gqa_paged_gather_dense_kernel(const GatherArgs a) {
    constexpr int SLOTS = D / 16, U = kGatherUnits;
    const int b = blockIdx.y, lane = threadIdx.x & 31;
    pdl_wait_primary();
    const int cap = a.pages_per_req * a.page_size;
    const int len0 = __ldg(a.seq_lens + b), start0 = a.starts != nullptr ? __ldg(a.starts + b) : 0;
    const int len = min(max(len0, 0), cap), start = max(start0, 0);
    const int n = min(len - start, a.rows);
    if (threadIdx.x == 0 && blockIdx.x == 0 && (len != len0 || start != start0)) flag_error(a.err, kErrIndex);
    // the warp's first output row
    const long long j_first = ((long long)blockIdx.x * (kGatherThreads / 32) + (threadIdx.x >> 5)) * a.tokens;
    if (j_first >= n) return;
    const int j0 = int(j_first), run = min(a.tokens, n - j0);
    int row_l = -1;  // pool row of token `lane` of the run, -1 where the page is out of range
    if (lane < run) {
        const int pos = start + j0 + lane;
        const int page = __ldg(a.page_table + (long long)b * a.pages_per_req + pos / a.page_size);
        if (page >= 0 && page < a.num_pages)
            row_l = page * a.page_size + pos % a.page_size;  // num_pages * page_size < 2^31
        else
            flag_error(a.err, kErrIndex);
    }
    const unsigned upt = unsigned(a.Hkv) * SLOTS;  // units of a token
    const unsigned units = unsigned(run) * upt;
    for (unsigned u0 = 0; u0 < units; u0 += 32 * U) {
        GatherCodes<KVT> k[U], v[U];
        float ks[U], kz[U], vs[U], vz[U];
#pragma unroll
        for (int i = 0; i < U; ++i) {
            const unsigned x = u0 + i * 32 + lane;
            const unsigned j = x / upt, u = x - j * upt;  // token of the run, unit of the token
            const int r = __shfl_sync(0xffffffffu, row_l, j & 31);
            const long long row = x < units ? r : -1;
            k[i] = v[i] = {};  // a row without a page reads as zeros
            ks[i] = kz[i] = vs[i] = vz[i] = 0.f;
            if (row < 0) continue;
            const long long head_row = row * a.Hkv + u / SLOTS;
            const long long elem = head_row * D + 16 * (u % SLOTS);
            gather_load<KVT>(k[i], a.k_pool, elem);
            gather_load<KVT>(v[i], a.v_pool, elem);
            if constexpr (KVT == GQA_KV_INT4) {
                const uint2 p = __ldg(reinterpret_cast<const uint2 *>(a.params + head_row * 4));
                const float2 pk = __half22float2(*reinterpret_cast<const __half2 *>(&p.x));
                const float2 pv = __half22float2(*reinterpret_cast<const __half2 *>(&p.y));
                ks[i] = pk.x, kz[i] = pk.y, vs[i] = pv.x, vz[i] = pv.y;
            } else if constexpr (KVT != GQA_KV_BF16) {
                const int si = a.n_scales > 1 ? int(u / SLOTS) : 0;
                ks[i] = a.k_scales != nullptr ? __ldg(a.k_scales + si) : a.k_scale;
                vs[i] = a.v_scales != nullptr ? __ldg(a.v_scales + si) : a.v_scale;
            }
        }
#pragma unroll
        for (int i = 0; i < U; ++i) {
            const unsigned x = u0 + i * 32 + lane;
            if (x >= units) continue;
            const long long o = (((long long)b * a.rows + j0) * upt + x) * 16;
#pragma unroll
            for (int half = 0; half < 2; ++half) {
                *reinterpret_cast<uint4 *>(a.k_out + o + 8 * half) = gather_value<KVT>(k[i], half, ks[i], kz[i]);
                *reinterpret_cast<uint4 *>(a.v_out + o + 8 * half) = gather_value<KVT>(v[i], half, vs[i], vz[i]);
            }
        }
    }
}

template <int D, int KVT>
cudaError_t launch_gather(GatherArgs a, cudaStream_t stream) {
    // Tokens of a warp: one batch of its lanes' units, fewer while that leaves
    // less than 32 warps an SM.  (Runs of 32 tokens of 8 heads of 128, 2048 units
    // a warp, took 145 us where runs of 2 took 110: a CTA should write one short
    // piece of the output at a time.)
    const long long all = (long long)a.rows * a.B / (32 * 152);
    const int most = 32 * kGatherUnits / (a.Hkv * (D / 16));
    a.tokens = most > 32 ? 32 : most < 1 ? 1 : most;
    if (all < a.tokens) a.tokens = all < 1 ? 1 : int(all);
    const int per = a.tokens * (kGatherThreads / 32);
    return launch_pdl(gqa_paged_gather_dense_kernel<D, KVT>, a,
                      dim3(unsigned((a.rows + per - 1) / per), unsigned(a.B)), kGatherThreads, stream);
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
    st = host_check_cache(kv_dtype, kv_params, k_scale, v_scale, k_scales, v_scales, n_scales, Hkv);
    if (st != GQA_OK) return st;
    const bool kv8 = kv_dtype == GQA_KV_FP8_E4M3FN || kv_dtype == GQA_KV_INT8;
    if (kv8 && k_scales == nullptr && (!(k_scale > 0.f) || !(v_scale > 0.f))) return GQA_ERR_INVALID_ARG;
    if (k_pool == nullptr || v_pool == nullptr || page_table == nullptr || seq_lens == nullptr ||
        (T > 0 && (k == nullptr || v == nullptr)))
        return GQA_ERR_INVALID_ARG;
    if (Hkv > (1 << 18) || (has_q && Hq > (1 << 18)) || T > (1 << 30)) return GQA_ERR_UNSUPPORTED;
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
    st = host_check_cache(kv_dtype, kv_params, k_scale, v_scale, k_scales, v_scales, n_scales, Hkv);
    if (st != GQA_OK) return st;
    if (k_pool == nullptr || v_pool == nullptr || page_table == nullptr || seq_lens == nullptr ||
        (rows > 0 && (k_out == nullptr || v_out == nullptr)))
        return GQA_ERR_INVALID_ARG;
    if (Hkv > (1 << 20) || rows > (1 << 30)) return GQA_ERR_UNSUPPORTED;
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
