// gqa_paged_int4.cuh -- paged decode over whole requests from a 4-bit cache
// (sm_103a): the main kernel and the merge of partial results.
//
// Mathematics.  With codes u in 0..15 and a token's own scale and zero,
// K^_t = u_t ks_t + kz_t and V^_t = v_t vs_t + vz_t, a row's scores and output are
//   s_t = scale (ks_t sum_d q_d u_td + kz_t sum_d q_d)
//   O_d = (sum_t p_t vs_t (v_td - 8) + sum_t p_t (vz_t + 8 vs_t)) / sum_t p_t,  p_t = e^(s_t).
// So the tensor cores multiply plain codes: q.u, and (p vs).v, whose sums start
// at -8 sum p vs; scale and zero of K enter the scores, those of V the weights
// and one extra sum a row.
//
// What bounds it.  A token costs 2 (D/2 + 4) bytes per KV head, a quarter of a
// bf16 cache, so the walk must turn codes into operands at four times the
// pace per byte.  The operand's cost is the kernel's budget:
//  - A 4-bit code masked out of its 16-bit half is the fp16 subnormal u 2^-24
//    (or 16 u 2^-24 for the second code of the half): an MMA operand of two
//    codes is one AND of the stored word, with no conversion, bias or
//    subtraction, and the factors (2^24, 2^20) come off once, in q for K and in
//    the epilogue for V.
//  - q's order along D and the output's order are free, so K's operands take
//    the codes in the order in which they lie in the word.  V's operands pair
//    two tokens of one element: a byte permute merges two tokens' halves, then
//    the same masks apply.
//  - The running maximum is a lazy reference: the row's maximum is only
//    reduced over the warp (and O rescaled) when some weight would pass 2^15,
//    which after the first steps of a walk is rare; a step otherwise costs one vote.
//
// What is rounded.  q (bf16) is exact in fp16 after a power of two that is
// taken from the row's largest element, down to 2^-27 of that.  The codes are
// exact.  p vs is rounded to fp16, half a step of which is 2^-11, an eighth of
// the bf16 output's.  That rounding counts by what a weight is multiplied with:
// the code's distance from the middle, which is of the size of V's spread
// (against the code itself, three times that, the output's error against 64
// bits was 1.7e-3 to 1.79e-3 where its own rounding is 1.64e-3 to 1.67e-3).
// Everything that is summed is summed in fp32.
//
// Layout.  As in the other paged kernels a CTA takes a block of KV heads and a
// worker's share of all requests' steps (here of 32 tokens).  One CTA fills an
// SM: 16 consumer warps for 8 query rows each, or 8 for 16 rows, one per head
// (and per group of rows), and four producer warps with few registers, one for
// each of up to four rings of shared-memory stages, or in turns on fewer; a ring
// is a worker.  (Of the ways tried on 32 requests of 16K to 32K tokens, 64 heads
// over 8 of 128: several CTAs an SM whose consumers start the loads in turns
// 177 us, a producer warp in each 155, this 143.)  Where heads and row groups are
// fewer than the warps, `lanes` groups take turns at a ring's steps and join
// their results in shared memory.
//
// K and V come by TMA as boxes of (row bytes) x (up to 32 tokens of one page) x
// (heads of the block): shared memory then holds each head's rows back to back,
// and with the 64-byte swizzle (D = 128) and the token order of `tok_of` every
// fragment read is free of bank conflicts.  Parameters come by TMA too,
// [token][head] (by cp.async where their rows are not 16 bytes and the CTA has
// not all heads); pages without a factor of 4 take K and V in 16-byte copies to
// the same places, since a box ends at its page's end.  The warps never wait for
// one another beyond the ring: each works out its segments from the lengths,
// and the loads run ahead across request borders.  Short requests are not
// shared out: a ring takes whole ones, one launch without partial results.
//
// Measured on GB300 (main and merge kernel): the 32 requests above, 814 MB,
// 141-146 us by box, 82 to 85 % of the copy peak -- bound by HBM and by SMs
// whose path to memory is slower, which the shares do not know of; one request of
// 128K tokens 44 us, of which the start is 6 and the merge 5; 256 requests of up
// to 1K tokens 47 us, where the consumers fill half of the issue slots (ALU pipe 41
// %, tensor pipe 22 %), wait the rest of the time and change requests; 16 requests of 4 x 4 rows a head
// and up to 8K tokens 37 us, where 16 rows a warp make a step 1.2 us long; 40
// whole requests of 256 tokens 14 us.
#pragma once

#include <stddef.h>

#include "gqa_common.cuh"
#include "gqa_params.h"

namespace gqa {

constexpr int kInt4Step = 32;       // tokens a stage
constexpr int kInt4MaxStages = 16;  // of a ring
constexpr int kInt4MaxRings = 4;    // of a CTA; as many producer warps
// Consumer warps of a CTA that hold NT tiles of 8 query rows, and the
// registers a thread of theirs and of the producers' warpgroup has: together
// what the CTA was launched with (20 warps of 96, or 12 of 168).  Producers that
// copy rows themselves need more than those that start TMA: a spilled value
// comes back behind all the copies under way.
__host__ __device__ constexpr int int4_consumers(int nt) { return nt == 1 ? 16 : 8; }
__host__ __device__ constexpr int int4_threads(int nt) { return 32 * (int4_consumers(nt) + 4); }
__host__ __device__ constexpr int int4_consumer_regs(int nt, bool copy) { return nt == 1 ? (copy ? 104 : 112) : 216; }
__host__ __device__ constexpr int int4_producer_regs(int nt, bool copy) { return nt == 1 ? (copy ? 64 : 32) : 72; }
static_assert(16 * int4_consumer_regs(1, false) + 4 * int4_producer_regs(1, false) == 20 * 96, "registers");
static_assert(16 * int4_consumer_regs(1, true) + 4 * int4_producer_regs(1, true) == 20 * 96, "registers");
static_assert(8 * int4_consumer_regs(2, true) + 4 * int4_producer_regs(2, true) == 12 * 168, "registers");
constexpr int kInt4WarpRequests = 256;  // up to so many requests each warp works out the schedule for itself
constexpr float kInt4NoRef = -3e38f;  // reference of a row that has seen nothing
// log2 of a row's largest weight when its reference is set.  Weights are fp16:
// at 2^7 what is rounded to nothing lies 2^-32 below the largest (at 1 it lay
// 2^-25 below, which over millions of tokens can be seen), and up to 2^15,
// where the reference moves, a step's largest may be 2^8 times the first one's.
constexpr float kInt4Top = 7.f;

// x / d for x < 2^31, d of the host's choosing: m = floor(2^(31 + l) / d) + 1, l = ceil(log2 d).  (m d lies above
// 2^(31 + l) by at most d <= 2^l, so x m / 2^(31 + l) is above x / d by less than 1 / d: the floor is right.)
struct FastDiv {
    unsigned long long m;
    int shift;
};
__device__ __forceinline__ int fast_div(int x, const FastDiv &f) { return int((unsigned long long)unsigned(x) * f.m >> f.shift); }

struct Int4Args {
    const __nv_bfloat16 *q;   // [B, Sq, Hq, D]
    const __half *params;     // [num_pages, page_size, Hkv, 4]
    const int32_t *page_table, *seq_lens;
    __nv_bfloat16 *out;
    float *lse;
    float *o_part;            // [head block, worker, 2 slots, HB, Mq, D] fp32, O / l
    float *lse_part;          // [head block, worker, 2 slots, HB, Mq] fp32, log2 domain
    int *step_prefix;         // [B + 2] first place of each request, their end, and the places shared out (several workers)
    int B, Sq, Hq, Hkv, G, Mq, page_size, pages_per_req, num_pages;
    int change;               // steps' worth of time that a change of request costs (at least 1)
    int whole;                // 1: worker w takes the whole requests w, w + workers, ...; 0: an equal share of all steps
    int next_b;               // from a worker's request to its next one: workers if whole, else 1
    int workers, HB, RG;      // workers per head block; heads of a CTA, warps (of 8 or 16 query rows) a head
    int rings, rings_max;     // rings (workers) of a CTA, and how many its warps could serve
    int lanes;                // groups of HB x RG warps that take turns at a ring's steps
    int stages, box_rows, box_pitch, stage_bytes;
    FastDiv by_page;          // page_size
    unsigned g_inv;           // ceil(2^16 / G): r / G = r * g_inv >> 16 for r < 128
    int param_tma;            // parameters by 2-D TMA, else by 8-byte cp.async
    int param_heads;          // heads between a token's parameters and the next one's in a stage
    int param_shift, param_mul;  // a box's row of the parameters' map: (first row >> shift) * mul
    int producers;            // warps that fill a ring: in turns (TMA), or a part of each step's tokens each (16-byte copies)
    const uint8_t *k_pool, *v_pool;  // for 16-byte copies
    unsigned param_pitch;     // of a box's parameters in a stage
    unsigned par8, par16;     // as tok8, tok16, of the parameters
    unsigned tok8, tok16;     // bytes from a token's row in a stage to that of the token 8, 16 later (8, 16 keep the swizzle)
    float alpha;              // scale * log2(e)
    unsigned long long wait_limit_ns;
    int fault_mode;           // test hook: 1 = the producer never issues the first stage
    unsigned *err;
};

// Shared memory of a CTA: barriers, masks, schedules and flag of its rings (at
// constant addresses), then the rings (on the swizzle's 512-byte period).
struct Int4Head {
    uint64_t full[kInt4MaxRings][kInt4MaxStages], empty[kInt4MaxRings][kInt4MaxStages];
    uint64_t ready[kInt4MaxRings], taken[kInt4MaxRings];  // lanes: results handed to the first lane, and taken
    uint32_t mask[kInt4MaxRings][kInt4MaxStages];  // tokens of a stage that are there
    int begin[kInt4MaxRings], end[kInt4MaxRings];  // steps of the ring's share
    unsigned long long first[kInt4MaxRings];  // its first request (high half), and that one's first step
    int warp_sum[20];
    int abort;
};
constexpr int kInt4HeadBytes = 2048;
static_assert(sizeof(Int4Head) <= kInt4HeadBytes && kInt4MaxStages <= 32, "head");

template <int REGS>
__device__ __forceinline__ void more_registers() {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(REGS));
}
template <int REGS>
__device__ __forceinline__ void fewer_registers() {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(REGS));
}

__device__ __forceinline__ uint32_t movmatrix_trans(uint32_t x) {
    uint32_t y;
    asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
    return y;
}

__device__ __forceinline__ uint32_t prmt4(uint32_t a, uint32_t b, uint32_t sel) {
    uint32_t r;
    asm("prmt.b32 %0, %1, %2, %3;" : "=r"(r) : "r"(a), "r"(b), "r"(sel));
    return r;
}

// Operands of a word's codes: of each half's lower byte (upper: its upper byte)
// lo has the low code u, hi the high one times 16, as fp16 subnormals in units
// of 2^-24.  The upper byte comes down by a permute that clears the rest, so
// its high code is a difference, exact, on the FMA pipe: the ALU pipe, at half
// the issue rate, is what these operands load most.
__device__ __forceinline__ void code_pairs(uint32_t word, int upper, uint32_t &lo, uint32_t &hi) {
    if (upper) {
        const uint32_t b = prmt4(word, 0, 0x4341u);
        lo = b & 0x000f000fu;
        asm("sub.f16x2 %0, %1, %2;" : "=r"(hi) : "r"(b), "r"(lo));
    } else {
        lo = word & 0x000f000fu;
        hi = word & 0x00f000f0u;
    }
}

// Larger of two fp16 pairs, half by half (a NaN gives way to the other).
__device__ __forceinline__ uint32_t hmax2(uint32_t a, uint32_t b) {
    uint32_t r;
    asm("max.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    return r;
}
// Whether a half of x, which is not negative, is above 2^15 (a NaN is not).
__device__ __forceinline__ bool above_2_15(uint32_t x) {
    const float2 f = __half22float2(*reinterpret_cast<const __half2 *>(&x));
    return fmaxf(f.x, f.y) > 32768.f;
}
// x + 0 x + 0 y, half by half: x where both are finite, else NaN.
__device__ __forceinline__ uint32_t nan_unless_finite(uint32_t x, uint32_t y) {
    uint32_t r;
    asm("{\n\t.reg .b32 t;\n\tfma.rn.f16x2 t, %1, %3, %1;\n\tfma.rn.f16x2 %0, %2, %3, t;\n\t}" : "=r"(r) : "r"(x), "r"(y), "r"(0u));
    return r;
}
// Larger of x and y; a NaN stays one.
__device__ __forceinline__ float max_nan(float x, float y) {
    float r;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(x), "f"(y));
    return r;
}

// d = A(16x16 f16) * B(16x8 f16), starting from zero
__device__ __forceinline__ void mma_f16_zero(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                             uint32_t b0, uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 "
        "{%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%10, %10, %10, %10};"
        : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(0.f));
}
// d = A * B + c
__device__ __forceinline__ void mma_f16_from(float (&d)[4], const float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                             uint32_t a3, uint32_t b0, uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 "
        "{%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%10, %11, %12, %13};"
        : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(c[0]), "f"(c[1]), "f"(c[2]), "f"(c[3]));
}
__device__ __forceinline__ void mma_f16_add(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                            uint32_t b0, uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 "
        "{%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// 3-D tiled bulk tensor load into shared memory, completing on an mbarrier.
__device__ __forceinline__ void tma_load_3d(uint32_t smem_dst, const void *tmap, uint64_t *bar, int c0, int c1,
                                            int c2) {
    asm volatile(
        "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
        " [%0], [%1, {%3, %4, %5}], [%2];" ::"r"(smem_dst),
        "l"(reinterpret_cast<uint64_t>(tmap)), "r"(smem_u32(bar)), "r"(c0), "r"(c1), "r"(c2)
        : "memory");
}

// 2-D form of it.
__device__ __forceinline__ void tma_load_2d(uint32_t smem_dst, const void *tmap, uint64_t *bar, int c0, int c1) {
    asm volatile(
        "cp.async.bulk.tensor.2d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
        " [%0], [%1, {%3, %4}], [%2];" ::"r"(smem_dst),
        "l"(reinterpret_cast<uint64_t>(tmap)), "r"(smem_u32(bar)), "r"(c0), "r"(c1)
        : "memory");
}

__device__ __forceinline__ void cp_async8(uint32_t smem_dst, const void *src) {
    asm volatile("cp.async.ca.shared.global [%0], [%1], 8;" ::"r"(smem_dst), "l"(src) : "memory");
}
__device__ __forceinline__ void cp_async16_to(uint32_t smem_dst, const void *src) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(smem_dst), "l"(src) : "memory");
}
// Arrives on the barrier (one of its expected arrivals) once every cp.async of
// this thread has landed.
__device__ __forceinline__ void cp_async_arrive(uint64_t *bar) {
    asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(smem_u32(bar)) : "memory");
}

__device__ __forceinline__ uint4 lds128(uint32_t addr) {
    uint4 v;
    asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(addr));
    return v;
}
__device__ __forceinline__ uint2 lds64(uint32_t addr) {
    uint2 v;
    asm volatile("ld.shared.v2.u32 {%0, %1}, [%2];" : "=r"(v.x), "=r"(v.y) : "r"(addr));
    return v;
}
__device__ __forceinline__ uint32_t lds32(uint32_t addr) {
    uint32_t v;
    asm volatile("ld.shared.u32 %0, [%1];" : "=r"(v) : "r"(addr));
    return v;
}

// As mbar_wait_bounded, by the barrier's shared-memory address.
__device__ __forceinline__ bool bar_try(uint32_t bar, uint32_t parity) {
    uint32_t ok;
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(ok)
        : "r"(bar), "r"(parity)
        : "memory");
    return ok != 0;
}
__device__ __forceinline__ bool bar_wait_bounded(uint32_t bar, uint32_t parity, uint64_t limit_ns,
                                                 volatile int *abort) {
    if (bar_try(bar, parity)) return true;
    const uint64_t t0 = globaltimer_ns();
    for (uint32_t it = 1;; ++it) {
        if (bar_try(bar, parity)) return true;
        if ((it & 63u) == 0u && ((abort != nullptr && *abort) || globaltimer_ns() - t0 > limit_ns)) return false;
    }
}
__device__ __forceinline__ void bar_arrive(uint32_t bar) {
    asm volatile("{\n\t.reg .b64 st;\n\tmbarrier.arrive.shared::cta.b64 st, [%0];\n\t}" ::"r"(bar) : "memory");
}

// Token (of a group of 8) in MMA row g.  A K fragment is read by the lanes of
// rows g, g + 1 together (16 bytes a lane; D = 64: rows g .. g + 3, 8 bytes a
// lane), a V fragment by the lanes of rows 0, 2, 4, 6 or 1, 3, 5, 7.  Rows lie
// D/2 bytes apart, so with D = 64 each of these sets must cover the four rows
// of a 128-byte line, and with D = 128 (two rows a line, the 64-byte swizzle
// xoring the 16-byte unit with bits 7-8 of the address) pairs of rows must
// differ in parity and V's even (odd) rows in bit 2.
template <int D>
__device__ __forceinline__ int tok_of(int g) {
    return D == 128 ? g ^ ((g >> 1) & 1) : g ^ (g >> 2);
}

// Byte of 16-byte unit `unit` in the row at offset `off` of a stage (which lies
// on the swizzle's 512-byte period).
template <int D>
__device__ __forceinline__ uint32_t swizzle(uint32_t off, int unit) {
    return D == 128 ? (uint32_t(unit) ^ ((off >> 7) & 3u)) << 4 : uint32_t(unit) << 4;
}

// First place of worker w's share of T places over W workers: floor(w T / W).
__device__ __forceinline__ int int4_share(unsigned w, int T, int W) {
    const unsigned long long x = (unsigned long long)w * unsigned(T);
    return x < (1ull << 32) ? int(unsigned(x) / unsigned(W)) : int(x / unsigned(W));
}

// COPY: K and V in 16-byte copies instead of TMA boxes (page sizes without a
// factor of 4).
template <int D, int NT, bool COPY>
__global__ void __launch_bounds__(int4_threads(NT), 1)
    gqa_paged_int4_kernel(const __grid_constant__ CUtensorMap k_map, const __grid_constant__ CUtensorMap v_map,
                          const __grid_constant__ CUtensorMap p_map, const Int4Args a) {
    constexpr int ROWB = D / 2;     // bytes of a row
    constexpr int KW = D / 32;      // K words a lane holds of a token
    constexpr int VW = D / 64;      // V words a lane holds of a token
    constexpr int DB = D / 16;      // output blocks: block j holds elements (D/8) gi + 2 j, + 2 j + 1
    constexpr int CW = int4_consumers(NT);
    constexpr uint32_t M0 = 0x000f000fu, M = 0x00ff00ffu;
    constexpr uint32_t kMinus8 = 0x80088008u, kMinus136 = 0x80888088u;  // in units of 2^-24, as the codes
    extern __shared__ __align__(1024) uint8_t smem4[];
    Int4Head *head = reinterpret_cast<Int4Head *>(smem4);
    volatile int *abort_flag = &head->abort;

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int hb0 = blockIdx.x * a.HB;
    const int nh = min(a.HB, a.Hkv - hb0);
    const int cap = a.pages_per_req * a.page_size;

    if (warp < a.rings && lane < a.stages) {  // a ring a warp, a stage a lane
        mbar_init(&head->full[warp][lane], a.param_tma ? 1 : 1 + 32 * (COPY ? a.producers : 1));  // the expect, and lanes' copies
        mbar_init(&head->empty[warp][lane], nh * a.RG);
        if (lane == 0) {
            mbar_init(&head->ready[warp], max(1, (a.lanes - 1) * nh * a.RG));
            mbar_init(&head->taken[warp], nh * a.RG);
            head->first[warp] = (unsigned long long)a.B << 32;
        }
        fence_mbarrier_init();
    }
    if (threadIdx.x == 0) {
        head->abort = 0;
        if constexpr (!COPY) {
            prefetch_tmap(&k_map);
            prefetch_tmap(&v_map);
        }
        if (a.param_tma) prefetch_tmap(&p_map);
    }
    pdl_wait_primary();  // inputs may be written by the previous kernel in the stream

    // The CW consumer warps form groups of HB x RG, `lanes` groups to a ring;
    // producer warp p serves ring p mod rings.  Warps of an SM sub-partition (warp mod 4)
    // run oldest first, and a ring is as fast as its slowest warp, so the
    // groups' warps are dealt so that each group has warps of every age.
    const int members = a.HB * a.RG, groups = a.rings_max * a.lanes;
    const int member = warp / groups;
    const int group = (warp + (groups == 2 ? member >> 1 : groups == 4 ? member : 0)) % groups;
    const int r = warp < CW ? group / a.lanes : (warp - CW) % a.rings;

    // ---- schedule.  Request b takes n_b = ceil(len_b / 32) steps and `change`
    // more for what changing requests costs (queries, output); worker w takes places
    // [w T / W, (w + 1) T / W) of the T places of all requests in order, b's
    // steps first from P_b on.  An empty request belongs to whoever holds P_b.
    bool bad = false;
    int w_begin, w_end, seg_b, seg_p;
    // no change follows the last request (an empty one keeps a place to be held)
    const int trailing = a.change - (__ldg(a.seq_lens + a.B - 1) <= 0 ? 1 : 0);
    if (a.whole) {
        const int w = r * int(gridDim.y) + int(blockIdx.y);
        w_begin = seg_p = 0;  // counted over the worker's own requests
        w_end = 0x7fffffff;
        seg_b = w < a.workers ? w : a.B;
        __syncthreads();  // the barriers are set up
    } else if (a.B <= kInt4WarpRequests) {
        // each warp for itself: a run of requests a lane, a scan, and the first
        // lane with a request that holds the share's first step
        const int run = (a.B + 31) / 32;
        const int b0 = min(a.B, lane * run), b1 = min(a.B, b0 + run);
        int mine = 0;
        for (int b = b0; b < b1; ++b) {
            const int len = __ldg(a.seq_lens + b);
            bad |= len < 0 || len > cap;
            mine += (min(max(len, 0), cap) + kInt4Step - 1) / kInt4Step + a.change;
        }
        int incl = mine;
#pragma unroll
        for (int off = 1; off < 32; off <<= 1) {
            const int y = __shfl_up_sync(0xffffffffu, incl, off);
            if (lane >= off) incl += y;
        }
        const int total = __shfl_sync(0xffffffffu, incl, 31), T = total - trailing;
        const int w = r * int(gridDim.y) + int(blockIdx.y);
        w_begin = int4_share(min(w, a.workers), T, a.workers);
        w_end = int4_share(min(w + 1, a.workers), T, a.workers);
        const bool record = a.step_prefix != nullptr && threadIdx.x < 32 && blockIdx.x == 0 && blockIdx.y == 0;
        int P = incl - mine, hit = a.B, hit_p = 0;
        for (int b = b0; b < b1; ++b) {
            const int n = run == 1 ? mine - a.change : (min(max(__ldg(a.seq_lens + b), 0), cap) + kInt4Step - 1) / kInt4Step;
            if (record) a.step_prefix[b] = P;
            if (hit == a.B && P + max(n, 1) > w_begin) hit = b, hit_p = P;
            P += n + a.change;
        }
        if (record && lane == 0) a.step_prefix[a.B] = total, a.step_prefix[a.B + 1] = T;
        const unsigned found = __ballot_sync(0xffffffffu, hit < a.B);
        const int src = found != 0 ? __ffs(found) - 1 : 0;
        seg_b = __shfl_sync(0xffffffffu, hit, src);
        seg_p = __shfl_sync(0xffffffffu, hit_p, src);
        if (bad && threadIdx.x < 32 && blockIdx.x == 0 && blockIdx.y == 0) flag_error(a.err, kErrIndex);
        bad = false;
        __syncthreads();  // the barriers are set up
    } else {
        // the CTA together: a run of requests a thread
        constexpr int NTH = int4_threads(NT);
        const int run = (a.B + NTH - 1) / NTH;
        const int b0 = min(a.B, int(threadIdx.x) * run), b1 = min(a.B, b0 + run);
        int mine = 0;
        for (int b = b0; b < b1; ++b) {
            const int len = __ldg(a.seq_lens + b);
            bad |= len < 0 || len > cap;
            mine += (min(max(len, 0), cap) + kInt4Step - 1) / kInt4Step + a.change;
        }
        int incl = mine;
#pragma unroll
        for (int off = 1; off < 32; off <<= 1) {
            const int y = __shfl_up_sync(0xffffffffu, incl, off);
            if (lane >= off) incl += y;
        }
        if (lane == 31) head->warp_sum[warp] = incl;
        __syncthreads();
        int T = 0, P = incl - mine;
        for (int w = 0; w < CW + 4; ++w) {
            T += head->warp_sum[w];
            if (w < warp) P += head->warp_sum[w];
        }
        const int total = T;
        T -= trailing;
        if (warp == 0 && lane < a.rings) {
            const int w = lane * int(gridDim.y) + int(blockIdx.y);
            head->begin[lane] = int4_share(min(w, a.workers), T, a.workers);
            head->end[lane] = int4_share(min(w + 1, a.workers), T, a.workers);
        }
        __syncthreads();
        const bool record = a.step_prefix != nullptr && blockIdx.x == 0 && blockIdx.y == 0;
        if (record && threadIdx.x == 0) a.step_prefix[a.B] = total, a.step_prefix[a.B + 1] = T;
        for (int b = b0; b < b1; ++b) {
            const int n = (min(max(__ldg(a.seq_lens + b), 0), cap) + kInt4Step - 1) / kInt4Step;
            if (record) a.step_prefix[b] = P;
            for (int k = 0; k < a.rings; ++k)
                if (P + max(n, 1) > head->begin[k])  // of those the first counts
                    atomicMin(&head->first[k], (unsigned long long)b << 32 | unsigned(P));
            P += n + a.change;
        }
        if (bad && blockIdx.x == 0 && blockIdx.y == 0) flag_error(a.err, kErrIndex);
        bad = false;
        __syncthreads();
        const int k = min(r, a.rings - 1);
        w_begin = head->begin[k];
        w_end = head->end[k];
        seg_b = int(head->first[k] >> 32);
        seg_p = int(unsigned(head->first[k]));
    }
    int seg_t = max(w_begin, seg_p);  // past the place of the request before

    const int R = a.box_rows;
    // Offsets in a stage: a token's row lies in box t / R, head h, row t % R.
    const uint32_t v_off = uint32_t(kInt4Step / R) * a.box_pitch;
    auto par_off = [&](int t, int h) { return 2 * v_off + uint32_t(t / R) * a.param_pitch + uint32_t((t % R) * a.param_heads + h) * 8; };

    // ============================================================== producers
    if (warp >= CW) {
        fewer_registers<int4_producer_regs(NT, COPY)>();
        // One warp starts a step's TMA every 0.65 us, so a ring's warps take turns
        // (one request of 1K tokens, 8 lanes on one ring: 27 -> 12 us); of
        // 16-byte copies each takes a part of every step's tokens.
        const int part = (warp - CW) / a.rings, parts = a.producers;
        if (part >= parts) return;
        const int every = COPY ? 1 : a.producers;  // takes every so many steps, and stages
        uint64_t *full = head->full[r], *empty = head->empty[r];
        uint32_t *vmask = head->mask[r];
        const uint32_t ring = smem_u32(smem4) + kInt4HeadBytes + uint32_t(r * a.stages) * a.stage_bytes;
        const uint32_t box_bytes = COPY ? 0 : uint32_t(R) * (a.HB * 2 * ROWB + (a.param_tma ? a.param_heads * 8 : 0));
        const uint32_t box_at = uint32_t(lane / R) * a.box_pitch, par_at = par_off(lane, 0);
        const bool first = lane % R == 0 && !COPY;  // of a box
        // 16-byte copies: a token's piece of the block's heads is 2^lc of them;
        // this lane always takes copy u of a token
        const int lc = 31 - __clz(a.HB) + (D == 128 ? 2 : 1);
        const int u = lane & ((1 << lc) - 1);
        const bool copies = u < nh * (ROWB / 16);
        const uint32_t row_bytes = uint32_t(a.Hkv) * ROWB, copy_at = uint32_t(u / (ROWB / 16)) * 16 * ROWB;
        const int per_part = kInt4Step / parts;
        const uint8_t *k_src = a.k_pool + size_t(hb0) * ROWB + u * 16;
        const uint8_t *v_src = a.v_pool + size_t(hb0) * ROWB + u * 16;
        int st = COPY ? 0 : part, round = 0;  // stage of this warp's next step, and times it was used
        int ahead = st;  // from the segment's first step to that one
        bool failed = false;
        while (seg_b < a.B && seg_t < w_end && !failed) {
            const int len0 = __ldg(a.seq_lens + seg_b), len = min(max(len0, 0), cap);
            bad |= len0 != len;
            const int steps_b = (len + kInt4Step - 1) / kInt4Step;
            const int seg_next = min(w_end, seg_p + steps_b);
            const int32_t *table = a.page_table + size_t(seg_b) * a.pages_per_req;
            const int t_end = min((seg_next - seg_p) * kInt4Step, len);
            int t = (seg_t - seg_p + ahead) * kInt4Step + lane;
            int at = fast_div(t, a.by_page);
            int page = t < t_end ? __ldg(table + at) : 0;
            while (t - lane < t_end) {
                const bool in = t < t_end;
                const bool ok = in && page >= 0 && page < a.num_pages;
                bad |= in && !ok;
                const int row = ok ? page * a.page_size + (t - at * a.page_size) : 0;
                // the next step's page is on its way while this one is issued
                t += kInt4Step * every;
                at = fast_div(t, a.by_page);
                if (t < t_end) page = __ldg(table + at);
                const uint32_t valid = __ballot_sync(0xffffffffu, ok);
                const bool box = ok && first;  // its first token's page holds all of a box
                const uint32_t boxes = __popc(__ballot_sync(0xffffffffu, box));
                if (round > 0) {
                    bool free = true;
                    if (lane == 0) free = mbar_wait_bounded(empty + st, (round - 1) & 1, a.wait_limit_ns, abort_flag);
                    if (!__shfl_sync(0xffffffffu, free, 0)) {
                        failed = true;
                        break;
                    }
                }
                if (!(a.fault_mode == 1 && round == 0 && st == 0)) {
                    if (lane == 0 && (!COPY || part == 0)) {
                        vmask[st] = valid;
                        mbar_arrive_expect_tx(full + st, boxes * box_bytes);
                    }
                    __syncwarp();
                    const uint32_t base = ring + uint32_t(st) * a.stage_bytes;
                    if (!COPY && box) {
                        tma_load_3d(base + box_at, &k_map, full + st, 0, row, hb0);
                        tma_load_3d(base + box_at + v_off, &v_map, full + st, 0, row, hb0);
                        if (a.param_tma) tma_load_2d(base + par_at, &p_map, full + st, hb0 * 4, (row >> a.param_shift) * a.param_mul);
                    }
                    if constexpr (COPY) {
#pragma unroll 4
                        for (int tok = part * per_part + (lane >> lc); tok < (part + 1) * per_part; tok += 32 >> lc) {
                            const uint32_t from = __shfl_sync(0xffffffffu, row, tok);
                            if ((valid >> tok & 1u) == 0 || !copies) continue;
                            const uint32_t off = (tok & 16 ? a.box_pitch : 0) + copy_at + uint32_t(tok & 15) * ROWB;
                            const uint32_t dst = base + off + swizzle<D>(off, u % (ROWB / 16));
                            const unsigned long long src = (unsigned long long)from * row_bytes;
                            cp_async16_to(dst, k_src + src);
                            cp_async16_to(dst + v_off, v_src + src);
                        }
                    }
                    if (COPY || !a.param_tma) {
                        if (ok && (!COPY || part == parts - 1)) {
                            const __half *src = a.params + (size_t(row) * a.Hkv + hb0) * 4;
                            for (int h = 0; h < nh; ++h) cp_async8(base + par_at + h * 8, src + h * 4);
                        }
                        cp_async_arrive(full + st);
                    }
                }
                st += every;
                if (st >= a.stages) st -= a.stages, ++round;
            }
            if (!COPY) ahead = (t - lane) / kInt4Step - (seg_next - seg_p);
            seg_t = seg_next;
            if (seg_next == seg_p + steps_b) {
                seg_t = seg_p = seg_next + a.change;
                seg_b += a.next_b;
            }
        }
        if (bad) flag_error(a.err, kErrIndex);
        if (failed && lane == 0) {
            flag_error(a.err, kErrTimeout);
            *abort_flag = 1;
        }
        // Every copy must land before the CTA's shared memory is released;
        // after an abort some may not have been waited for.
        for (int i = COPY ? 0 : part; i < a.stages; i += every) {
            const int last = round - (i < st ? 0 : 1);  // the last round in which stage i was filled
            if (last < 0 || (a.fault_mode == 1 && last == 0 && i == 0)) continue;
            if (lane == 0 && !mbar_wait_bounded(full + i, last & 1, a.wait_limit_ns, nullptr))
                flag_error(a.err, kErrTimeout);
        }
        return;
    }

    // ============================================================== consumers
    more_registers<int4_consumer_regs(NT, COPY)>();
    const int turn = group - r * a.lanes;
    const int lh = member / a.RG, rg = member - lh * a.RG;
    if (member >= members || r >= a.rings || lh >= nh) return;
    const int w = r * int(gridDim.y) + int(blockIdx.y);  // worker
    const uint32_t ring = smem_u32(smem4) + kInt4HeadBytes + uint32_t(r * a.stages) * a.stage_bytes;
    const int g = hb0 + lh;
    const int gi = lane >> 2, c = lane & 3;
    auto row_off = [&](int t) { return uint32_t(t / R) * a.box_pitch + uint32_t(lh * R + t % R) * ROWB; };
    const uint32_t k_row = row_off(tok_of<D>(gi));
    const uint32_t k_off = D == 128 ? k_row + swizzle<D>(k_row, c) : k_row + 8 * c;
    uint32_t vo[2];  // tokens of MMA columns 2 c, 2 c + 1
#pragma unroll
    for (int e = 0; e < 2; ++e) {
        const uint32_t r = row_off(tok_of<D>(2 * c + e));
        vo[e] = v_off + (D == 128 ? r + swizzle<D>(r, gi >> 1) + (gi & 1) * 8 : r + 4 * gi);
    }
    const int tok0 = tok_of<D>(gi);
    auto row_of = [&](int r) { return int(unsigned(r) * a.g_inv >> 16); };  // query row i of the group's row r = i G + h
    const uint32_t p_off = par_off(tok0, lh);

    const uint32_t full = smem_u32(head->full[r]), mask_at = smem_u32(head->mask[r]);
    constexpr uint32_t kEmpty = offsetof(Int4Head, empty) - offsetof(Int4Head, full);

    int done = 0;    // steps of the share before the segment
    int handed = 0;  // results handed between the lanes so far
    int st = turn;  // the stages are a multiple of the lanes: a lane sees every round of its stages
    uint32_t phase = 0;
    bool failed = false;
    // Queries as they are in memory: lane gi has row gi (+ 8 a tile), its
    // quarter c of the elements.  Loaded before the previous segment's results
    // are written, so that the latency lies under that.
    uint4 q_next[NT][KW];
    auto load_queries = [&](int b) {
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
            const int row = (rg * NT + nt) * 8 + gi;
            const int i = row_of(row);
            const __nv_bfloat16 *src = a.q + ((size_t(b) * a.Sq + i) * a.Hq + g * a.G + (row - i * a.G)) * D + (D / 4) * c;
#pragma unroll
            for (int w = 0; w < KW; ++w)
                q_next[nt][w] = row < a.Mq && b < a.B ? __ldg(reinterpret_cast<const uint4 *>(src) + w) : make_uint4(0, 0, 0, 0);
        }
    };
    load_queries(seg_b);
    // Segment of the share: steps [seg_t, seg_next) of request seg_b.
    while (seg_b < a.B && seg_t < w_end) {
        const int b = seg_b;
        const int len = min(max(__ldg(a.seq_lens + b), 0), cap);
        const int steps_b = (len + kInt4Step - 1) / kInt4Step;
        const int seg_next = min(w_end, seg_p + steps_b);
        const bool complete = seg_t == seg_p && seg_next == seg_p + steps_b;
        const int slot = seg_t == seg_p ? 1 : 0;  // of a part: a request's first steps, or what follows

        // ---- queries.  Lane gi holds row gi (+ 8 a tile) at the elements of
        // its quarter c, times a power of two that brings the row's largest
        // element near 2^14 (bf16 values stay exact in fp16 down to 2^-27 of
        // it).  The second code of a half is 16 u, so its q is q / 16.
        uint32_t qf[NT][2 * KW][2];
        float A[NT][2], qs[NT][2], R_[NT][2], l[NT][2], z[NT][2];
        float o[NT][DB][4];
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
            float x[KW][8];
            float mx = 0.f;
#pragma unroll
            for (int w = 0; w < KW; ++w) {
                const uint32_t rw[4] = {q_next[nt][w].x, q_next[nt][w].y, q_next[nt][w].z, q_next[nt][w].w};
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    x[w][2 * j] = __uint_as_float(rw[j] << 16);
                    x[w][2 * j + 1] = __uint_as_float(rw[j] & 0xffff0000u);
                    mx = fmaxf(mx, fmaxf(fabsf(x[w][2 * j]), fabsf(x[w][2 * j + 1])));
                }
            }
            mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 1));
            mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 2));
            // exponent of mx, kept where 2^-ex and 2^ex are normal
            const bool inf = mx > 3.4e38f;
            const int ex = inf ? 0 : max(int(__float_as_uint(mx) >> 23) - 127 - 14, -100);
            const float down = __uint_as_float(uint32_t(127 - ex) << 23);
            float sum = 0.f;
#pragma unroll
            for (int w = 0; w < KW; ++w) {
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    x[w][j] *= down;
                    sum += x[w][j];
                }
                qf[nt][2 * w][0] = pack_f16x2(x[w][0], x[w][4]);
                qf[nt][2 * w][1] = pack_f16x2(x[w][1] * 0.0625f, x[w][5] * 0.0625f);
                qf[nt][2 * w + 1][0] = pack_f16x2(x[w][2], x[w][6]);
                qf[nt][2 * w + 1][1] = pack_f16x2(x[w][3] * 0.0625f, x[w][7] * 0.0625f);
            }
            sum += __shfl_xor_sync(0xffffffffu, sum, 1);
            sum += __shfl_xor_sync(0xffffffffu, sum, 2);
            // score in the log2 domain = A (ks acc + kz qs), acc = 2^-24 sum q u
            // (an infinite query, or scale * mx past 2^103: every score NaN by the
            // zeros' part.  Up to there the least of all scores, D = 128 elements
            // of a K of -65504, lies above -2^127.6; scores below kInt4NoRef would
            // look like no token.)
            const float factor = a.alpha * __uint_as_float(uint32_t(127 + ex) << 23) * 16777216.f;
            const float row_a = fmaxf(factor, 1e-37f);
            const float row_qs = inf || factor > 1.4982e34f ? NAN : sum * (1.f / 16777216.f);  // log2(e) 2^113
#pragma unroll
            for (int e = 0; e < 2; ++e) {  // rows of this lane's scores: 2 c + e
                A[nt][e] = __shfl_sync(0xffffffffu, row_a, 4 * (2 * c + e));
                qs[nt][e] = __shfl_sync(0xffffffffu, row_qs, 4 * (2 * c + e));
                R_[nt][e] = kInt4NoRef;
                l[nt][e] = z[nt][e] = 0.f;
            }
#pragma unroll
            for (int j = 0; j < DB; ++j) o[nt][j][0] = o[nt][j][1] = o[nt][j][2] = o[nt][j][3] = 0.f;
        }
        const int n_seg = seg_next - seg_t;
        // from this many steps before the segment's end some row may not see a
        // token (row 0 sees none past len - Sq)
        const int n_causal = a.Sq > 1 ? min(n_seg, n_seg - (max(len - a.Sq + 1, 0) / kInt4Step - (seg_t - seg_p))) : 0;

        // this lane's steps of the segment: every lanes-th of the share's
        const int skip = a.lanes == 1 ? 0 : (turn + a.lanes - done % a.lanes) % a.lanes;
        for (int left = n_seg - skip; left > 0; left -= a.lanes) {
            const bool ok = bar_wait_bounded(full + 8 * st, phase, a.wait_limit_ns, abort_flag);
            if (!__all_sync(0xffffffffu, ok)) {
                failed = true;
                break;
            }
            const uint32_t base = ring + uint32_t(st) * a.stage_bytes;
            const uint32_t mask = lds32(mask_at + 4 * st);
            uint32_t kw[4][KW];  // token group j: tokens tok0 + 8 j
            uint2 par[4];
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const uint32_t at = base + k_off + (j & 1) * a.tok8 + (j >> 1) * a.tok16;
                if constexpr (KW == 4) {
                    const uint4 x = lds128(at);
                    kw[j][0] = x.x, kw[j][1] = x.y, kw[j][2] = x.z, kw[j][3] = x.w;
                } else {
                    const uint2 x = lds64(at);
                    kw[j][0] = x.x, kw[j][1] = x.y;
                }
                par[j] = lds64(base + p_off + (j & 1) * a.par8 + (j >> 1) * a.par16);
            }
            // ---- scores of 2 x 16 tokens
            float acc[NT][2][4];
#pragma unroll
            for (int w = 0; w < KW; ++w)
#pragma unroll
                for (int h = 0; h < 2; ++h)
#pragma unroll
                    for (int t = 0; t < 2; ++t) {
                        // codes 0, 4 and 1, 5 of the word, or 2, 6 and 3, 7
                        uint32_t lo0, hi0, lo1, hi1;
                        code_pairs(kw[2 * t][w], h, lo0, hi0);
                        code_pairs(kw[2 * t + 1][w], h, lo1, hi1);
#pragma unroll
                        for (int nt = 0; nt < NT; ++nt) {
                            const uint32_t b0 = qf[nt][2 * w + h][0], b1 = qf[nt][2 * w + h][1];
                            if (w == 0 && h == 0)
                                mma_f16_zero(acc[nt][t], lo0, lo1, hi0, hi1, b0, b1);
                            else
                                mma_f16_add(acc[nt][t], lo0, lo1, hi0, hi1, b0, b1);
                        }
                    }

            // ---- weights.  acc[t][2 i + e]: token group j = 2 t + i, row 2 c + e.
            float vs[4], vz[4];
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                // a token with a NaN or infinite parameter has a score of NaN, so that no weight of 0 hides it
                const uint32_t pk = nan_unless_finite(par[j].x, par[j].y);
                const float2 k2 = __half22float2(*reinterpret_cast<const __half2 *>(&pk));
                const float2 v2 = __half22float2(*reinterpret_cast<const __half2 *>(&par[j].y));
                vs[j] = max_nan(v2.x, 5.9604644775390625e-8f);  // fp16's smallest: a weight of 0 would hide its score
                vz[j] = v2.y;
#pragma unroll
                for (int nt = 0; nt < NT; ++nt) {
                    float *y = &acc[nt][j >> 1][2 * (j & 1)];
                    // rounded here, so that a score less itself is 0 at any size
                    const float2 x = mul2(make_float2(fmaf(y[0], k2.x, k2.y * qs[nt][0]), fmaf(y[1], k2.x, k2.y * qs[nt][1])),
                                          make_float2(A[nt][0], A[nt][1]));
                    y[0] = x.x, y[1] = x.y;
                }
            }
            if (mask != 0xffffffffu || left <= n_causal) {  // tokens that are not there, or not seen by all rows
                const int s0 = (seg_next - seg_p - left) * kInt4Step;  // the step's first token
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const bool there = (mask >> (tok0 + 8 * j)) & 1u;
                    // a slot that is not there may hold anything; a NaN or infinity of V would pass a weight of
                    // 0 in the rows that do not see its token, and those that do have it by the score
                    const bool odd = !(fmaxf(vs[j], fabsf(vz[j])) <= 65504.f && vs[j] == vs[j] && vz[j] == vz[j]);
                    if (!there || odd) vs[j] = vz[j] = 0.f;
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                        for (int e = 0; e < 2; ++e) {
                            const int r = (rg * NT + nt) * 8 + 2 * c + e;
                            const bool seen = there && s0 + tok0 + 8 * j <= len - a.Sq + (r < a.Mq ? row_of(r) : a.Sq);
                            if (!seen) acc[nt][j >> 1][2 * (j & 1) + e] = -INFINITY;
                        }
                }
            }
#pragma unroll
            for (int j = 0; j < 4; ++j) vz[j] = fmaf(8.f, vs[j], vz[j]);  // the value of V's middle code
            // Weights of V as fp16 pairs (rows 2 c, 2 c + 1), the step's sums of
            // p and p vz, and the largest weight.
            uint32_t wt[NT][4], top = 0;
            float sp[NT][2], sz[NT][2];
            auto weigh = [&] {
#pragma unroll
                for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
                    for (int e = 0; e < 2; ++e) sp[nt][e] = sz[nt][e] = 0.f;
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        float p[2];
                        const float2 d = add2(make_float2(acc[nt][j >> 1][2 * (j & 1)], acc[nt][j >> 1][2 * (j & 1) + 1]),
                                              make_float2(-R_[nt][0], -R_[nt][1]));
#pragma unroll
                        for (int e = 0; e < 2; ++e) {
                            p[e] = fast_exp2(e == 0 ? d.x : d.y);
                            sp[nt][e] += p[e];
                            sz[nt][e] = fmaf(p[e], vz[j], sz[nt][e]);
                        }
                        wt[nt][j] = pack_f16x2(p[0] * vs[j], p[1] * vs[j]);
                        top = hmax2(top, wt[nt][j]);
                    }
                }
            };
            weigh();
            if (__any_sync(0xffffffffu, above_2_15(top))) {
                // Move references up to the step's largest score + log2(V scale)
                // - kInt4Top: the row's largest weight is then 2^kInt4Top.  Only of
                // rows past the limit themselves (by more than the roundings of
                // the test above), so that no row's bits depend on another row.
#pragma unroll
                for (int nt = 0; nt < NT; ++nt) {
                    float corr[2];
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        float m = kInt4NoRef;
#pragma unroll
                        for (int j = 0; j < 4; ++j) {
                            const float y = acc[nt][j >> 1][2 * (j & 1) + e];
                            if (!(vs[j] > 0.f && vs[j] <= 65504.f)) continue;
                            const float top_j = log2f(vs[j]) - kInt4Top;
                            float m_j = y + top_j;
                            // a score of 2^28 has steps of 32: rounded down, the weight could pass fp16
                            if (y - m_j > 8.f - top_j) m_j = __fadd_ru(y, top_j);
                            m = fmaxf(m, m_j);
                        }
                        m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, 4));
                        m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, 8));
                        m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, 16));
                        m = m > R_[nt][e] + (15.f - kInt4Top + 0.00390625f) ? m : R_[nt][e];
                        corr[e] = fast_exp2(R_[nt][e] - m);
                        R_[nt][e] = m;
                        l[nt][e] *= corr[e];
                        z[nt][e] *= corr[e];
                    }
#pragma unroll
                    for (int j = 0; j < DB; ++j) {
                        o[nt][j][0] *= corr[0];
                        o[nt][j][1] *= corr[1];
                        o[nt][j][2] *= corr[0];
                        o[nt][j][3] *= corr[1];
                    }
                }
                weigh();
            }
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    l[nt][e] += sp[nt][e];
                    z[nt][e] += sz[nt][e];
                }
                // to row gi's weights for the tokens of columns 2 c, 2 c + 1 of group j
#pragma unroll
                for (int j = 0; j < 4; ++j) wt[nt][j] = movmatrix_trans(wt[nt][j]);
            }
            // what the sums start from: every code 8 less, every whole byte 8 + 16 x 8
            float middle[NT][4];
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
                mma_f16_zero(middle[nt], kMinus8, kMinus136, kMinus8, kMinus136, wt[nt][0], wt[nt][1]);
                mma_f16_add(middle[nt], kMinus8, kMinus136, kMinus8, kMinus136, wt[nt][2], wt[nt][3]);
            }

            uint32_t vw[8][VW];  // token pair j: tokens of columns 2 c, 2 c + 1, 8 j later
#pragma unroll
            for (int j = 0; j < 4; ++j)
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    const uint32_t at = base + vo[e] + (j & 1) * a.tok8 + (j >> 1) * a.tok16;
                    if constexpr (VW == 2) {
                        const uint2 x = lds64(at);
                        vw[2 * j + e][0] = x.x, vw[2 * j + e][1] = x.y;
                    } else {
                        vw[2 * j + e][0] = lds32(at);
                    }
                }
            __syncwarp();
            if (lane == 0) bar_arrive(full + kEmpty + 8 * st);
            st += a.lanes;
            if (st >= a.stages) st -= a.stages, phase ^= 1;

            // ---- O^T += (V - 8)^T . weights, 32 tokens at a time.  The tensor
            // cores cut off what does not fit their sums, always towards zero,
            // so over a long walk the cuts would add up.  The sum over the
            // steps is rounded instead.
#pragma unroll
            for (int w = 0; w < VW; ++w)
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    const uint32_t sel = h ? 0x7632u : 0x5410u;
                    float sum[NT][2][4];
#pragma unroll
                    for (int t = 0; t < 2; ++t) {
                        const uint32_t x = prmt4(vw[4 * t][w], vw[4 * t + 1][w], sel);
                        const uint32_t y = prmt4(vw[4 * t + 2][w], vw[4 * t + 3][w], sel);
                        // element 2 j: its codes; element 2 j + 1: whole bytes
                        // (16 times its codes more than that), taken apart in the epilogue
                        const uint32_t x8 = prmt4(x, 0, 0x4341u), y8 = prmt4(y, 0, 0x4341u);
#pragma unroll
                        for (int nt = 0; nt < NT; ++nt) {
                            const uint32_t b0 = wt[nt][2 * t], b1 = wt[nt][2 * t + 1];
                            if (t == 0) {
                                mma_f16_from(sum[nt][0], middle[nt], x & M0, x & M, y & M0, y & M, b0, b1);
                                mma_f16_from(sum[nt][1], middle[nt], x8 & M0, x8, y8 & M0, y8, b0, b1);
                            } else {
                                mma_f16_add(sum[nt][0], x & M0, x & M, y & M0, y & M, b0, b1);
                                mma_f16_add(sum[nt][1], x8 & M0, x8, y8 & M0, y8, b0, b1);
                            }
                        }
                    }
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                        for (int k = 0; k < 2; ++k)
#pragma unroll
                            for (int e = 0; e < 4; e += 2) {
                                float(&acc_o)[4] = o[nt][4 * w + 2 * h + k];
                                const float2 r2 = add2(make_float2(acc_o[e], acc_o[e + 1]), make_float2(sum[nt][k][e], sum[nt][k][e + 1]));
                                acc_o[e] = r2.x, acc_o[e + 1] = r2.y;
                            }
                }
        }
        if (failed) break;
        load_queries(b + a.next_b);
        done += n_seg;

        // ---- lanes: the first one takes the others' results, which lie in
        // shared memory behind the rings, thread for thread.  (Waits on
        // barriers with a limit, so that a lane that gave up stops the others.)
        if (a.lanes > 1 && n_seg > 0) {
            constexpr int kWords = NT * (4 * DB + 6);
            const uint32_t round = handed++ & 1;
            float *box = reinterpret_cast<float *>(smem4 + kInt4HeadBytes + a.rings * a.stages * a.stage_bytes) +
                         (r * (a.lanes - 1) * members + member) * kWords * 32 + lane;
            const uint32_t ready = smem_u32(&head->ready[r]), taken = smem_u32(&head->taken[r]);
            const bool wait = turn == 0 || handed > 1;
            if (wait && !__all_sync(0xffffffffu, bar_wait_bounded(turn == 0 ? ready : taken, turn == 0 ? round : round ^ 1,
                                                                  a.wait_limit_ns, abort_flag))) {
                failed = true;
                break;
            }
            if (turn > 0) {
                box += (turn - 1) * members * kWords * 32;
#pragma unroll
                for (int nt = 0; nt < NT; ++nt) {
                    float *p = box + nt * (4 * DB + 6) * 32;
#pragma unroll
                    for (int j = 0; j < DB; ++j)
#pragma unroll
                        for (int e = 0; e < 4; ++e) p[(4 * j + e) * 32] = o[nt][j][e];
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        p[(4 * DB + e) * 32] = R_[nt][e];
                        p[(4 * DB + 2 + e) * 32] = l[nt][e];
                        p[(4 * DB + 4 + e) * 32] = z[nt][e];
                    }
                }
                __syncwarp();
                if (lane == 0) bar_arrive(ready);
            } else {
                for (int k = 1; k < a.lanes; ++k, box += members * kWords * 32) {
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt) {
                        const float *p = box + nt * (4 * DB + 6) * 32;
                        float mine[2], other[2];
#pragma unroll
                        for (int e = 0; e < 2; ++e) {
                            const float x = p[(4 * DB + e) * 32], m = fmaxf(x, R_[nt][e]);
                            mine[e] = fast_exp2(R_[nt][e] - m);
                            other[e] = fast_exp2(x - m);
                            R_[nt][e] = m;
                            l[nt][e] = l[nt][e] * mine[e] + p[(4 * DB + 2 + e) * 32] * other[e];
                            z[nt][e] = z[nt][e] * mine[e] + p[(4 * DB + 4 + e) * 32] * other[e];
                        }
#pragma unroll
                        for (int j = 0; j < DB; ++j)
#pragma unroll
                            for (int e = 0; e < 4; ++e)
                                o[nt][j][e] = o[nt][j][e] * mine[e & 1] + p[(4 * j + e) * 32] * other[e & 1];
                    }
                }
                __syncwarp();
                if (lane == 0) bar_arrive(taken);
            }
        }

        // ---- epilogue of the segment: row 2 c + e of a tile, elements (D/8) gi .. + D/8 - 1
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                float L = l[nt][e], Z = z[nt][e];
#pragma unroll
                for (int off = 4; off < 32; off *= 2) {
                    L += __shfl_xor_sync(0xffffffffu, L, off);
                    Z += __shfl_xor_sync(0xffffffffu, Z, off);
                }
                const int r = (rg * NT + nt) * 8 + 2 * c + e;
                if (r >= a.Mq || turn > 0) continue;
                const float f = L == 0.f ? 0.f : __fdividef(1.f, L);  // NaN stays
                const float lse2 = L == 0.f ? -INFINITY : R_[nt][e] + __log2f(L);
                const float f24 = f * 16777216.f, f20 = f * 1048576.f, zf = Z * f;
                float x[2 * DB];
#pragma unroll
                for (int j = 0; j < DB; ++j) {
                    x[2 * j] = fmaf(o[nt][j][e], f24, zf);
                    x[2 * j + 1] = fmaf(o[nt][j][2 + e] - o[nt][j][e], f20, zf);
                }
                if (!complete) {
                    const size_t prow = ((((size_t(blockIdx.x) * a.workers + w) * 2 + slot) * a.HB + lh) * a.Mq) + r;
                    float *dst = a.o_part + prow * D + (D / 8) * gi;
#pragma unroll
                    for (int j = 0; j < 2 * DB; j += 4)
                        *reinterpret_cast<float4 *>(dst + j) = make_float4(x[j], x[j + 1], x[j + 2], x[j + 3]);
                    if (gi == 0) a.lse_part[prow] = lse2;
                    continue;
                }
                const int i = row_of(r), h = g * a.G + (r - i * a.G);
                __nv_bfloat16 *dst = a.out + ((size_t(b) * a.Sq + i) * a.Hq + h) * D + (D / 8) * gi;
#pragma unroll
                for (int j = 0; j < 2 * DB; j += 8)
                    *reinterpret_cast<uint4 *>(dst + j) =
                        make_uint4(pack_bf16x2(x[j], x[j + 1]), pack_bf16x2(x[j + 2], x[j + 3]),
                                   pack_bf16x2(x[j + 4], x[j + 5]), pack_bf16x2(x[j + 6], x[j + 7]));
                if (a.lse != nullptr && gi == 0)
                    a.lse[(size_t(b) * a.Hq + h) * a.Sq + i] = lse2 * 0.69314718055994530942f;
            }
        seg_t = seg_next;
        if (seg_next == seg_p + steps_b) {
            seg_t = seg_p = seg_next + a.change;
            seg_b += a.next_b;
        }
    }
    if (failed && lane == 0) {
        flag_error(a.err, kErrTimeout);
        *abort_flag = 1;
    }
}

// Merge of the partials of requests that several workers share.  CTA (x, b):
// with SPLIT, row x of request b, whose partials are dealt in runs to all warps
// and their results merged in warp order -- few rows, many partials each;
// without, one row a warp.  A warp reads 32 partials' LSEs at once, one a lane,
// which gives their weights, then adds them up in order, several in flight: the
// same bits every time.  A few us, most of them the launch.
__host__ __device__ constexpr int int4_merge_batch(bool split) { return split ? 8 : 4; }  // partials in flight
__host__ __device__ constexpr int int4_merge_warps(bool split) { return split ? 16 : 8; }

template <int D, bool SPLIT>
__global__ void __launch_bounds__(32 * int4_merge_warps(SPLIT), SPLIT ? 2 : 5) gqa_paged_int4_merge_kernel(const Int4Args a) {
    constexpr int V = D / 32, NW = int4_merge_warps(SPLIT), BATCH = int4_merge_batch(SPLIT);
    __shared__ float sm_m[NW], sm_l[NW], sm_o[SPLIT ? NW : 1][D];
    pdl_wait_primary();
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int b = blockIdx.y, rr = SPLIT ? int(blockIdx.x) : int(blockIdx.x) * NW + warp;
    const int W = a.workers;
    const int P = a.step_prefix[b], n = a.step_prefix[b + 1] - P - a.change, T = a.step_prefix[a.B + 1];
    if (n == 0) return;  // an empty request: written by the main kernel
    // worker of step s: the largest w with floor(w T / W) <= s
    auto holder = [&](int s) {
        const unsigned long long x = (unsigned long long)(s + 1) * unsigned(W) - 1;
        return x < (1ull << 32) ? int(unsigned(x) / unsigned(T)) : int(x / unsigned(T));
    };
    const int w_first = holder(P), w_last = holder(P + n - 1);
    if (w_first == w_last) return;  // one worker: written by the main kernel
    if (rr >= a.Hkv * a.Mq) return;
    const int g = rr / a.Mq, r = rr - g * a.Mq;
    const int hb = g / a.HB, lh = g - hb * a.HB;
    const int parts = w_last - w_first + 1;
    const int each = SPLIT ? (parts + NW - 1) / NW : parts;
    const int from = SPLIT ? warp * each : 0, to = min(parts, from + each);

    float m = -INFINITY, L = 0.f, acc[V];
#pragma unroll
    for (int v = 0; v < V; ++v) acc[v] = 0.f;
    for (int k0 = from; k0 < to; k0 += 32) {
        // one partial a lane: its LSE gives the weights of the 32
        const int part = k0 + lane, w = w_first + part;
        float l2 = -INFINITY;
        // a worker without a step (T < W) holds nothing
        const bool there = part < to && !(T < W && int4_share(w, T, W) == int4_share(w + 1, T, W));
        const size_t prow = ((((size_t(hb) * W + w) * 2 + (part == 0 ? 1 : 0)) * a.HB + lh) * a.Mq) + r;
        if (there) l2 = __ldg(a.lse_part + prow);
        float mn = l2;
#pragma unroll
        for (int off = 16; off > 0; off >>= 1) mn = fmaxf(mn, __shfl_xor_sync(0xffffffffu, mn, off));
        mn = fmaxf(mn, m);
        const float sc = m == -INFINITY ? 0.f : fast_exp2(m - mn);
        const float wgt = l2 == -INFINITY ? 0.f : fast_exp2(l2 - mn);
        float sum = wgt;
#pragma unroll
        for (int off = 16; off > 0; off >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, off);
        L = L * sc + sum;
#pragma unroll
        for (int v = 0; v < V; ++v) acc[v] *= sc;
        m = mn;
        const size_t step = size_t(2) * a.HB * a.Mq * D;  // from a worker's partial to the next one's
        const float *first = a.o_part + ((((size_t(hb) * W + w_first + k0) * 2) * a.HB + lh) * a.Mq + r) * D + lane * V;
        const int n_here = min(32, to - k0);
        for (int j0 = 0; j0 < n_here; j0 += BATCH) {
            float x[BATCH][V];
#pragma unroll
            for (int j = 0; j < BATCH; ++j) {
                const float f = __shfl_sync(0xffffffffu, wgt, (j0 + j) & 31);
#pragma unroll
                for (int v = 0; v < V; ++v) x[j][v] = 0.f;
                if (j0 + j >= n_here || f == 0.f) continue;  // a partial without weight may hold anything
                const float *src = first + (j0 + j) * step + (k0 + j0 + j == 0 ? step / 2 : 0);
                if constexpr (V == 4) {
                    const float4 t = __ldg(reinterpret_cast<const float4 *>(src));
                    x[j][0] = t.x, x[j][1] = t.y, x[j][2] = t.z, x[j][3] = t.w;
                } else {
                    const float2 t = __ldg(reinterpret_cast<const float2 *>(src));
                    x[j][0] = t.x, x[j][1] = t.y;
                }
            }
#pragma unroll
            for (int j = 0; j < BATCH; ++j) {
                const float f = __shfl_sync(0xffffffffu, wgt, (j0 + j) & 31);
#pragma unroll
                for (int v = 0; v < V; ++v) acc[v] = fmaf(f, x[j][v], acc[v]);
            }
        }
    }
    if constexpr (SPLIT) {
        if (lane == 0) sm_m[warp] = m, sm_l[warp] = L;
#pragma unroll
        for (int v = 0; v < V; ++v) sm_o[warp][lane * V + v] = acc[v];
        __syncthreads();
        if (warp > 0) return;
        m = -INFINITY;
#pragma unroll
        for (int w = 0; w < NW; ++w) m = fmaxf(m, sm_m[w]);
        L = 0.f;
#pragma unroll
        for (int v = 0; v < V; ++v) acc[v] = 0.f;
#pragma unroll
        for (int w = 0; w < NW; ++w) {
            if (sm_l[w] == 0.f) continue;
            const float f = fast_exp2(sm_m[w] - m);
            L += f * sm_l[w];
#pragma unroll
            for (int v = 0; v < V; ++v) acc[v] += f * sm_o[w][lane * V + v];
        }
    }
    const float inv = L == 0.f ? 0.f : 1.f / L;
    const int i = r / a.G, h = g * a.G + (r - i * a.G);
    const size_t row = (size_t(b) * a.Sq + i) * a.Hq + h;
#pragma unroll
    for (int v = 0; v < V; v += 2)
        *reinterpret_cast<uint32_t *>(a.out + row * D + lane * V + v) = pack_bf16x2(acc[v] * inv, acc[v + 1] * inv);
    if (a.lse != nullptr && lane == 0)
        a.lse[(size_t(b) * a.Hq + h) * a.Sq + i] = L == 0.f ? -INFINITY : (m + log2f(L)) * 0.69314718055994530942f;
}

}  // namespace gqa
