// gqa_prefill_kernel.cuh -- prompt attention on the fifth-generation tensor cores (tcgen05 + TMEM).
//
//   s_j = scale q.k_j over the keys that a row sees,  out = sum_j exp(s_j - lse) v_j
//
// One persistent CTA an SM walks its pieces of the plan (gqa_prefill_plan.cuh).  A tile is 128 query rows: tok_tile
// consecutive tokens x g_tile query heads of one KV head (TMA lays them out so), so that one token of a grouped model still
// fills rows, and K and V are read once for all of them.  Steps of 128 keys:
//   S_t = Q_t K^T  (128 x 128, K = Dqk)   P_t = exp2(alpha S_t - reference)   O_t += P_t V  (128 x Dv, K = 128)
// with two tiles t = 0, 1 in TMEM (S 128 columns and O Dv columns each; P_t overwrites S_t as 16-bit values and is the A
// operand of the second product).  The tensor core works on one tile's products while the other tile's softmax runs: the
// issue order is P_t V of a step, then Q_t K^T of tile t's next step, then the same for the other tile.  An item with rows for
// one tile only gives its steps to the two row groups in turns and joins their (reference, sum, O) at the end.
//
// Roles: warps 0-3 and 4-7 softmax of tile 0 and 1, a thread a row; warp 8 issues the products; warp 9 loads Q and K, warp
// 10 V, by TMA; warp 11 clears, in steps past what some row sees, the V rows that no row may see (0 x NaN is NaN) and
// elements of V that are not finite, which rows that see them get back at the end; such steps land on a barrier of their own
// and warp 11 hands them on.
// Pools that TMA cannot bring as they are wanted (codes; bf16 pages of odd sizes) have four more warps that copy or convert
// K and V through registers (gqa_prefill_load.cuh); warp 9 then loads Q only.  Codes enter the products as fp16: FP8 and int8
// codes as they are (exact), 4-bit codes of K as they are, with scale and zero applied to the scores, those of V as values.
// Q is converted to fp16 in place, each row times a power of two (exact but for elements 2^-28 below the row's largest).
// Tensor products run in the order of their issue, so S_t of a step being there says that O_t of the step before is too.
//
// Two tiles because one chain of scores, softmax (1.4K cycles a step), weights and output leaves the tensor core (1K cycles a
// step and tile at d 128) idle more than half of the time; 128 keys a step because S, P and O of both tiles then fill TMEM.
// Measured (GB300; a call alone after an L2 flush, and in brackets among others, where the power limit holds the long ones; of
// 1.89 PFLOP/s measured for a large library product).  64/8 heads of 128: one causal prompt of 16K tokens 2.64 (2.76-2.89) ms =
// 1.67 (1.53-1.59) PFLOP/s, 2K rows over 128K bf16 keys 5.12 (5.52-5.71) ms = 1.70 (1.53-1.58) PFLOP/s; the tensor pipe is 69 %
// active at 8K tokens; 8 rows for each of 16 requests of 8K-32K keys 240 (226) us, 206 in the kernel = 6.45 TB/s (HBM); a
// mixed step over an FP8 cache 1.23 (1.15-1.18) ms = 1.1 PFLOP/s (the converting warps, 2.6K cycles a step).  Short items are bound
// by their chain: some 8K cycles beside their steps, of which the epilogue is 5K.  At d 64 a step's products halve and its
// softmax does not: one prompt of 8K tokens 658 (611) us = 0.84-0.89 PFLOP/s.  Single tokens over codes convert every code for a
// tile that is a sixteenth full: 32 tokens over 16K-32K keys FP8 459 (451) us, 4 bits 750 (745), where the paged decode calls
// take 273 and 141-146.
#pragma once

#include "gqa_prefill_load.cuh"
#include "gqa_umma.cuh"

namespace gqa {

// A row's largest weight is 2^TOP when its reference is set, and the reference moves when a later one would pass 2^8 times that.
// bf16 weights have fp32's range (TOP 0); fp16 ones lose what lies below 2^-25, so they start at 2^7 and use fp16's range up to
// 2^15: what is rounded to nothing lies 2^-32 below the largest (from 1 on it lay 2^-25 below, and a row with one large
// score among 2^20 small ones came out 2 % small, its sum being taken before the rounding).
constexpr float kPreRescaleLog2 = 8.f, kPreTopF16 = 7.f;

// Steps of a row group after which its O goes to global memory, in fp32, and starts anew.  The tensor core cuts a product off some
// 2^-25 below the sum that it is added to: over 2^20 keys values of one sign came out 0.7 % small, and the others' part was
// missing where one key's weight was 2^25 times theirs.  Over 256 steps that is 2^-10 of the sum at most.  Items of up to 32K keys
// never come to it.  It takes some 6 us, as all SMs move their 128 KB at about the same time (2K rows over 128K keys: every 256
// steps 5690 us, every 128 some 60 more, never 5610).
constexpr int kPreDrain = 256;
static_assert((kPreDrain & (kPreDrain - 1)) == 0 && kPreDrain > kPreMinSplit + kPreSnap, "only items with room for partial results");

__device__ __forceinline__ void tma_load_3d(void *smem_dst, const void *tmap, uint64_t *bar, int c0, int c1, int c2) {
    asm volatile(
        "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
        " [%0], [%1, {%3, %4, %5}], [%2];" ::"r"(smem_u32(smem_dst)),
        "l"(reinterpret_cast<uint64_t>(tmap)), "r"(smem_u32(bar)), "r"(c0), "r"(c1), "r"(c2)
        : "memory");
}

// Adds to a row's result (bf16 out, or fp32 part) the elements of V's rows key0 .. key1 - 1 that are not finite: the
// products had zeros there.  (What is added is the value without its scale and weight: infinite or NaN all the same.)  Eight
// elements of eight keys at a time, then into the result: where all of V is NaN a batch of 256 prompts of 128 tokens takes 4.4 ms
// (element by element into the result 71, which is longer than the least limit of the other warps' waits).
template <int DV, int SRC, typename T>
__device__ __noinline__ void prefill_add_not_finite(const PrefillArgs &a, int req, int k_row, int g, int key0, int key1, T *dst) {
    if constexpr (SRC == kPreInt8) return;  // every code is finite
    constexpr int KEYS = 8, WORDS = SRC == kPreInt4 ? 1 : SRC == kPreFp8 ? 2 : 4;  // keys on their way, words of one's elements
#pragma unroll 1
    for (int d = 0; d < DV; d += 8) {
        float add[8] = {};
        bool some = false;
#pragma unroll 1
        for (int key = key0; key < key1; key += KEYS) {
            long long at[KEYS];
            uint32_t w[KEYS][WORDS] = {};
#pragma unroll
            for (int i = 0; i < KEYS; ++i) {
                at[i] = -1;
                if (key + i < key1) at[i] = SRC == kPreDense ? k_row + key + i : prefill_pool_row(a, req, key + i);
            }
#pragma unroll
            for (int i = 0; i < KEYS; ++i) {
                if (at[i] < 0) continue;
                const long long head = at[i] * a.Hkv + g;
                if constexpr (SRC == kPreInt4) {
                    w[i][0] = reinterpret_cast<const uint32_t *>(a.params)[head * 2 + 1];
                } else if constexpr (SRC == kPreFp8) {
                    const uint2 x = *reinterpret_cast<const uint2 *>(a.v_pool + head * DV + d);
                    w[i][0] = x.x, w[i][1] = x.y;
                } else {
                    const __nv_bfloat16 *v = SRC == kPreDense ? a.v + at[i] * a.v_stride + g * DV : reinterpret_cast<const __nv_bfloat16 *>(a.v_pool) + head * DV;
                    const uint4 x = *reinterpret_cast<const uint4 *>(v + d);
                    w[i][0] = x.x, w[i][1] = x.y, w[i][2] = x.z, w[i][3] = x.w;
                }
            }
            bool found = false;
#pragma unroll
            for (int i = 0; i < KEYS; ++i)
#pragma unroll
                for (int x = 0; x < WORDS; ++x)
                    found |= SRC == kPreFp8 ? __vcmpeq4(w[i][x] & 0x7f7f7f7fu, 0x7f7f7f7fu) != 0 : not_finite2<SRC == kPreInt4>(w[i][x]);
            if (!found) continue;
            some = true;
#pragma unroll
            for (int i = 0; i < KEYS; ++i)
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    if constexpr (SRC == kPreInt4) {
                        if (not_finite2<true>(w[i][0])) add[e] = NAN;
                    } else if constexpr (SRC == kPreFp8) {
                        if ((w[i][e >> 2] >> (e & 3) * 8 & 0x7f) == 0x7f) add[e] = NAN;
                    } else {
                        const float f = __uint_as_float(e & 1 ? w[i][e >> 1] & 0xffff0000u : w[i][e >> 1] << 16);
                        if (!isfinite(f)) add[e] += f;
                    }
                }
        }
        if (!some) continue;
#pragma unroll
        for (int e = 0; e < 8; ++e) dst[d + e] = T(float(dst[d + e]) + add[e]);
    }
}

__device__ __forceinline__ bool elect_one() {
    uint32_t p;
    asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(p));
    return p != 0;
}

// Shared-memory matrix descriptors of 128-byte-swizzled operands (smem_desc_sw128) in two words: the low one moves by
// offset / 16, the high one is the same for all (1024 bytes between groups of 8 rows).
__device__ __forceinline__ uint32_t desc_lo(uint32_t addr, uint32_t lbo) { return (addr & 0x3FFFFu) >> 4 | lbo >> 4 << 16; }
constexpr uint32_t kDescHi = (1024 >> 4) | 1u << 14 | 2u << 29;

// D[tmem] (+)= A[smem] B[smem], and with A in tensor memory.
template <bool ADD>
__device__ __forceinline__ void umma_ss(uint32_t d, uint32_t a, uint32_t b, uint32_t idesc) {
    asm volatile(
        "{\n\t.reg .pred p;\n\t.reg .b64 x, y;\n\tmov.b64 x, {%1, %3};\n\tmov.b64 y, {%2, %3};\n\tsetp.ne.b32 p, %5, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], x, y, %4, p;\n\t}" ::"r"(d), "r"(a), "r"(b), "r"(kDescHi), "r"(idesc), "n"(int(ADD))
        : "memory");
}
template <bool ADD>
__device__ __forceinline__ void umma_ts(uint32_t d, uint32_t a, uint32_t b, uint32_t idesc) {
    asm volatile(
        "{\n\t.reg .pred p;\n\t.reg .b64 y;\n\tmov.b64 y, {%2, %3};\n\tsetp.ne.b32 p, %5, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], y, %4, p;\n\t}" ::"r"(d), "r"(a), "r"(b), "r"(kDescHi), "r"(idesc), "n"(int(ADD))
        : "memory");
}

// Lanes without bit d keep word a and get the partner's a for b; lanes with it the other way round.
__device__ __forceinline__ void swap_words(uint32_t &a, uint32_t &b, int d, bool up) {
    const uint32_t got = __shfl_xor_sync(0xffffffffu, up ? a : b, d);
    a = up ? got : a;
    b = up ? b : got;
}

// Lane q of four gets piece q (words 4 q ..) of each of the four lanes.
__device__ __forceinline__ void quad_transpose(uint32_t (&x)[16], int lane) {
    const bool up1 = (lane & 1) != 0, up2 = (lane & 2) != 0;
#pragma unroll
    for (int w = 0; w < 4; ++w) {
        swap_words(x[w], x[4 + w], 1, up1);
        swap_words(x[8 + w], x[12 + w], 1, up1);
    }
#pragma unroll
    for (int w = 0; w < 4; ++w) {
        swap_words(x[w], x[8 + w], 2, up2);
        swap_words(x[4 + w], x[12 + w], 2, up2);
    }
}

// The row's 8 elements of one 16-byte unit as fp16, times `scale`; the order that 4-bit codes come in for those.
template <int SRC>
__device__ __forceinline__ uint4 prefill_q_unit(uint4 x, float scale) {
    float f[8];
    const uint32_t w[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        f[2 * i] = __uint_as_float(w[i] << 16) * scale;
        f[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u) * scale;
    }
    if constexpr (SRC == kPreInt4)
        return make_uint4(pack_f16x2(f[0], f[4]), pack_f16x2(f[1], f[5]), pack_f16x2(f[2], f[6]), pack_f16x2(f[3], f[7]));
    return make_uint4(pack_f16x2(f[0], f[1]), pack_f16x2(f[2], f[3]), pack_f16x2(f[4], f[5]), pack_f16x2(f[6], f[7]));
}

// A row group's O (at o_at, a thread a row) goes to global memory with the row's reference, added to what is there (some); last:
// that sum goes back into O instead.  The place is the warp's rows of the worker's last place for partial results, which nothing
// else uses before the epilogue of the worker's last piece; four elements of each of 32 rows in turn, so that a warp's
// accesses are whole lines.  (Not inline: two copies in the softmax's code cost short items 4 %.)
template <int DV>
__device__ __noinline__ void prefill_drain(const PrefillArgs &a, uint32_t o_at, int t, float m_ref, bool some, bool last) {
    const long long place = ((2LL * blockIdx.x + 1) * 2 + t) * kPreTile + (threadIdx.x >> 5 & 3) * 32;  // of the warp's rows
    float4 *at = reinterpret_cast<float4 *>(a.o_part + place * DV) + (threadIdx.x & 31);
    float *ref = a.lse_part + place + (threadIdx.x & 31);
    float corr = 1.f;
    if (some && *ref != m_ref) corr = fast_exp2(*ref - m_ref);
    if (!last) *ref = m_ref;
#pragma unroll 1
    for (int c = 0; c < DV; c += 64) {
        uint32_t ov[2][32];
        float4 y[16] = {};
        if (some) {
#pragma unroll
            for (int e = 0; e < 16; ++e) y[e] = at[(c / 4 + e) * 32];
        }
        tmem_ld32(o_at + c, ov[0]);
        tmem_ld32(o_at + c + 32, ov[1]);
        tmem_wait_ld();
#pragma unroll
        for (int e = 0; e < 16; ++e) {
            float *x = reinterpret_cast<float *>(&y[e]);
#pragma unroll
            for (int z = 0; z < 4; ++z) {
                uint32_t &o = ov[e / 8][4 * e % 32 + z];
                x[z] = fmaf(x[z], corr, __uint_as_float(o));
                o = __float_as_uint(x[z]);
            }
            if (!last) at[(c / 4 + e) * 32] = y[e];
        }
        if (last) {
            tmem_st32(o_at + c, ov[0]);
            tmem_st32(o_at + c + 32, ov[1]);
        }
    }
    if (last) tmem_wait_st();
    __syncwarp();  // every lane has read its part of the place, which may be the piece's own
}

template <int DQK, int DV, int SRC>
__global__ void __launch_bounds__(PrefillCfg<DQK, DV, SRC>::THREADS, 1)
    gqa_prefill_kernel(const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_k,
                       const __grid_constant__ CUtensorMap tm_v, const __grid_constant__ PrefillArgs a) {
    using C = PrefillCfg<DQK, DV, SRC>;
    extern __shared__ uint8_t smem_raw[];
    uint8_t *smem = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    float2 *stat = reinterpret_cast<float2 *>(smem + C::STAT_OFF);
    uint64_t *q_full = reinterpret_cast<uint64_t *>(smem + C::BAR_OFF);  // [1] a piece's rows have landed
    uint64_t *q_empty = q_full + 1;     // [1] ... and its last score product is done
    uint64_t *k_full = q_empty + 1;     // [KST]
    uint64_t *k_empty = k_full + C::KST;
    uint64_t *v_full = k_empty + C::KST;  // [VST]
    uint64_t *v_empty = v_full + C::VST;
    uint64_t *v_raw = v_empty + C::VST;  // [VST] V of a step past what some row sees, not cleared yet
    uint64_t *s_full = v_raw + C::VST;     // [2] a tile's scores are there
    uint64_t *p_full = s_full + 2;         // [2] a tile's weights are
    uint64_t *o_full = p_full + 2;         // [2] a tile's last product of the piece is done
    uint64_t *q_ready = o_full + 2;        // [2] a tile's rows are fp16
    uint64_t *stat_full = q_ready + 2;      // [1] row group 1's references and sums are in `stat`
    uint64_t *stat_free = stat_full + 1;   // [1] ... and joined, its O too
    uint64_t *piece_full = stat_free + 1;  // [kPrePieces]
    uint64_t *piece_empty = piece_full + kPrePieces;
    uint64_t *fin = piece_empty + kPrePieces;  // [1] every product is done
    uint32_t *tmem_base_s = reinterpret_cast<uint32_t *>(fin + 1);
    volatile int *abort_flag = reinterpret_cast<volatile int *>(tmem_base_s + 1);
    volatile int *bad_v = abort_flag + 1;  // elements of V that are not finite were cleared, in this piece or an earlier one
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const uint64_t limit = a.wait_limit_ns;

    if (threadIdx.x == 0) {
        mbar_init(q_full, 1);
        mbar_init(q_empty, 1);
        constexpr int loaders = C::TMA ? 1 : 128;
        for (int s = 0; s < C::KST; ++s) mbar_init(&k_full[s], loaders), mbar_init(&k_empty[s], 1);
        for (int s = 0; s < C::VST; ++s) mbar_init(&v_full[s], loaders), mbar_init(&v_empty[s], 1), mbar_init(&v_raw[s], 1);
        for (int t = 0; t < 2; ++t) mbar_init(&s_full[t], 1), mbar_init(&p_full[t], 128), mbar_init(&o_full[t], 1), mbar_init(&q_ready[t], 128);
        mbar_init(stat_full, 128);
        mbar_init(stat_free, 128);
        // read by the softmax warps, the issuer, and V's loader and cleaner or the four that convert
        for (int i = 0; i < kPrePieces; ++i) mbar_init(&piece_full[i], 1), mbar_init(&piece_empty[i], 8 + 1 + (C::TMA ? 2 : 4));
        mbar_init(fin, 1);
        *abort_flag = 0;
        *bad_v = 0;
        fence_mbarrier_init();
    }
    if (warp == 8) tmem_alloc(tmem_base_s, C::TMEM_COLS);
    if (threadIdx.x == 288) {
        prefetch_tmap(&tm_q);
        if constexpr (C::TMA) prefetch_tmap(&tm_k), prefetch_tmap(&tm_v);
    }
    tc_fence_before_sync();
    __syncthreads();
    tc_fence_after_sync();
    const uint32_t tbase = *tmem_base_s;
    pdl_wait_primary();  // the plan, and whatever wrote the inputs

    bool ok = true;
    PrefillPiece *pieces = reinterpret_cast<PrefillPiece *>(smem + C::PIECE_OFF);
    PieceFeed feed(pieces, piece_full, piece_empty);
    if (!C::TMA && warp >= 12) {
        if constexpr (!C::TMA) {
            set_registers<C::LAUNCH_REGS, C::LOAD_REGS>();
            ok = prefill_load<DQK, DV, SRC>(a, smem, k_full, k_empty, v_full, v_empty, feed, abort_flag, bad_v);
        }
        if (!ok && lane == 0) {
            flag_error(a.err, kErrTimeout);
            *abort_flag = 1;
        }
        __syncwarp();
    } else if (warp >= 8) {
        set_registers<C::LAUNCH_REGS, C::OTHER_REGS>();
        if (warp == 8) {
            // -------------------------------------------------------- products
            // One lane; descriptors are a base and a constant and ring places are counted, so that the next product is issued
            // before the one under way ends (rebuilding descriptors took 134 cycles a product beside two softmax warps, where
            // the tensor core takes 64).
            constexpr uint32_t fmt = C::F16 ? ~((1u << 7) | (1u << 10)) : ~0u;
            constexpr uint32_t idesc_qk = idesc_bf16_f32(kPreTile, kPreKeys, false, false) & fmt;
            constexpr uint32_t idesc_pv = idesc_bf16_f32(kPreTile, DV, false, true) & fmt;
            if (elect_one()) {
                const uint32_t q_desc = desc_lo(smem_u32(smem + C::Q_OFF), 16), k_desc = desc_lo(smem_u32(smem + C::K_OFF), 16);
                const uint32_t v_desc = desc_lo(smem_u32(smem + C::V_OFF), kPreKeys * 128);
                uint32_t q_phase = 0, p_phase = 0, k_phase = 0, v_phase = 0;
                int ks = 0, vs = 0;  // stages in turn
                while (ok) {
                    const volatile PrefillPiece *p = feed.next(limit, abort_flag, &ok);
                    if (p == nullptr) break;
                    const int units = p->units;
                    const bool two = p->two;
                    feed.done();
                    feed.step();
                    if (units == 0) continue;
                    if constexpr (C::F16)
                        ok = mbar_wait_bounded(&q_ready[0], q_phase, limit, abort_flag) &&
                             mbar_wait_bounded(&q_ready[1], q_phase, limit, abort_flag);
                    else
                        ok = mbar_wait_bounded(q_full, q_phase, limit, abort_flag);
                    q_phase ^= 1;
                    auto qk = [&](int u) {
                        const uint32_t t = u & 1;
                        if (!two || t == 0) {
                            ok = mbar_wait_bounded(&k_full[ks], k_phase, limit, abort_flag);
                            if (!ok) return;
                        }
                        tc_fence_after_sync();
                        const uint32_t d = tbase + C::S_COL + t * kPreKeys;
                        const uint32_t qd = q_desc + t * (C::Q_BYTES >> 4), kd = k_desc + ks * (C::K_BYTES >> 4);
#pragma unroll
                        for (int kk = 0; kk < DQK / 16; ++kk) {
                            const uint32_t off = (kk >> 2) * (kPreTile * 128 >> 4) + (kk & 3) * 2;
                            if (kk == 0) umma_ss<false>(d, qd, kd, idesc_qk);
                            else umma_ss<true>(d, qd + off, kd + off, idesc_qk);
                        }
                        umma_commit(&s_full[t]);
                        if (!two || t == 1) {
                            umma_commit(&k_empty[ks]);
                            if (++ks == C::KST) ks = 0, k_phase ^= 1;
                        }
                        if (u == units - 1) umma_commit(q_empty);
                    };
                    if (ok) qk(0);
                    if (ok && units > 1) qk(1);
                    for (int u = 0; ok && u < units; ++u) {
                        const uint32_t t = u & 1;
                        if (!two || t == 0) ok = mbar_wait_bounded(&v_full[vs], v_phase, limit, abort_flag);
                        ok = ok && mbar_wait_bounded(&p_full[t], p_phase >> t & 1, limit, abort_flag);
                        p_phase ^= 1u << t;
                        if (!ok) break;
                        tc_fence_after_sync();
                        const uint32_t d = tbase + C::O_COL + t * DV, w = tbase + C::S_COL + t * kPreKeys;
                        const uint32_t vd = v_desc + vs * (C::V_BYTES >> 4);
                        if ((u >> 1) & (kPreDrain - 1)) umma_ts<true>(d, w, vd, idesc_pv);
                        else umma_ts<false>(d, w, vd, idesc_pv);
#pragma unroll
                        for (int kg = 1; kg < kPreKeys / 16; ++kg) umma_ts<true>(d, w + kg * 8, vd + kg * (2048 >> 4), idesc_pv);
                        if (!two || t == 1) {
                            umma_commit(&v_empty[vs]);
                            if (++vs == C::VST) vs = 0, v_phase ^= 1;
                        }
                        if (u + 2 >= units) umma_commit(&o_full[t]);
                        else qk(u + 2);
                    }
                }
                if (!ok) {
                    flag_error(a.err, kErrTimeout);
                    *abort_flag = 1;
                }
                umma_commit(fin);
                mbar_wait_bounded(fin, 0, limit, nullptr);
            }
        } else if (warp == 9 || (C::TMA && warp == 10)) {
            // -------------------------------------------------------- loads: Q and K, or V
            const bool is_k = warp == 9;
            const int stages = is_k ? C::KST : C::VST, chunks = is_k ? C::QC : C::VC;
            const int stage_bytes = is_k ? C::K_BYTES : C::V_BYTES;
            uint64_t *full = is_k ? k_full : v_full, *empty = is_k ? k_empty : v_empty;
            uint8_t *ring = smem + (is_k ? C::K_OFF : C::V_OFF);
            const CUtensorMap *map = is_k ? &tm_k : &tm_v;
            int n_piece = 0, at = 0;
            uint32_t raw_next = 0, raw_last = 0;  // a bit a stage: parity of its next uncleared step, whether its last was one
            auto load_piece = [&](const PrefillPiece &p) {
                if (p.units <= 0) return;
                if (is_k) {
                    ok = n_piece == 0 || mbar_wait_bounded(q_empty, (n_piece - 1) & 1, limit, abort_flag);
                    ok = __all_sync(0xffffffffu, ok);
                    if (!ok) return;
                    ++n_piece;
                    if (lane == 0) {
                        const int tiles = p.units > 1 ? 2 : 1;
                        mbar_arrive_expect_tx(q_full, tiles * C::QC * a.g_tile * a.tok_tile * 128);
                        for (int t = 0; t < tiles; ++t)
#pragma unroll
                            for (int c = 0; c < C::QC; ++c)
                                tma_load_3d(smem + C::Q_OFF + t * C::Q_BYTES + c * (kPreTile * 128), &tm_q, q_full, c * 64,
                                            p.g * a.G + p.hb * a.g_tile, p.q_row + (p.two ? t * a.tok_tile : 0));
                    }
                    __syncwarp();
                }
                for (int step = p.s0; C::TMA && ok && step < p.s1; ++step, ++at) {
                    const int st = at % stages;
                    int row = 0;  // of this lane's box
                    bool there = false;
                    if constexpr (SRC == kPrePages) {
                        const int key = step * kPreKeys + lane * a.box_rows;
                        there = lane * a.box_rows < kPreKeys && key < p.L;
                        if (there) row = prefill_pool_row(a, p.req, key);
                        if (row < 0) row = a.num_pages * a.page_size;  // past the end: zeros
                    }
                    ok = at < stages || mbar_wait_bounded(&empty[st], (at / stages - 1) & 1, limit, abort_flag);
                    ok = __all_sync(0xffffffffu, ok);
                    if (!ok) break;
                    if (a.fault_mode == 1 && is_k && at == 0) continue;  // test hook: this stage never fills
                    uint8_t *dst = ring + st * stage_bytes;
                    uint64_t *bar = &full[st];
                    raw_last &= ~(1u << st);
                    if (!is_k && (step + 1) * kPreKeys > p.first_limit) {
                        bar = &v_raw[st];
                        raw_last |= 1u << st;
                        raw_next ^= 1u << st;
                    }
                    if constexpr (SRC == kPreDense) {
                        if (lane == 0) {
                            mbar_arrive_expect_tx(bar, stage_bytes);
                            for (int c = 0; c < chunks; ++c)
                                tma_load_3d(dst + c * (kPreKeys * 128), map, bar, c * 64, p.g, p.k_row + step * kPreKeys);
                        }
                    } else {
                        const int boxes = __popc(__ballot_sync(0xffffffffu, there));
                        if (lane == 0) mbar_arrive_expect_tx(bar, boxes * chunks * a.box_rows * 128);
                        __syncwarp();
                        if (there)
                            for (int c = 0; c < chunks; ++c)
                                tma_load_3d(dst + c * (kPreKeys * 128) + lane * a.box_rows * 128, map, bar, c * 64, p.g, row);
                    }
                    __syncwarp();
                }
            };
            PrefillPiece p;
            if (is_k) {
                // This warp walks the plan for all of them, a piece ahead of its own loads.
                auto publish = [&](int n) {
                    ok = n < kPrePieces || mbar_wait_bounded(&piece_empty[n % kPrePieces], (n / kPrePieces - 1) & 1, limit, abort_flag);
                    ok = __all_sync(0xffffffffu, ok);
                    if (ok && lane == 0) {
                        pieces[n % kPrePieces] = p;
                        mbar_arrive(&piece_full[n % kPrePieces]);
                    }
                    __syncwarp();
                };
                if (a.direct) {
                    const bool some = direct_piece<SRC != kPreDense>(a, blockIdx.x, &p);
                    if (some) publish(0);
                    if (some) load_piece(p);
                    p.units = -1;
                    if (ok) publish(some ? 1 : 0);
                } else {
                    PrefillWalk walk(a, blockIdx.x);
                    for (int n = 0; ok; ++n) {
                        walk.next(&p);
                        publish(n);
                        if (!ok || p.units < 0) break;
                        load_piece(p);
                    }
                }
            } else {
                while (ok) {
                    const volatile PrefillPiece *x = feed.next(limit, abort_flag, &ok);
                    ok = __all_sync(0xffffffffu, ok);
                    if (!ok || x == nullptr) break;
                    p.units = x->units, p.L = x->L, p.req = x->req, p.k_row = x->k_row, p.g = x->g, p.s0 = x->s0, p.s1 = x->s1;
                    p.first_limit = x->first_limit;
                    __syncwarp();
                    if (lane == 0) feed.done();
                    feed.step();
                    load_piece(p);
                }
            }
            if (!ok && lane == 0) {
                flag_error(a.err, kErrTimeout);
                *abort_flag = 1;
            }
            if (lane == 0 && (!ok || *abort_flag)) {
                // copies in flight land before the CTA goes
                for (int i = max(0, at - stages); i < at; ++i) {
                    const int st = i % stages;
                    if (a.fault_mode == 1 && is_k && i == 0) continue;
                    if (raw_last >> st & 1) mbar_wait_bounded(&v_raw[st], raw_next >> st & 1 ^ 1, limit, nullptr);
                    else mbar_wait_bounded(&full[st], (i / stages) & 1, limit, nullptr);
                }
                if (is_k && n_piece > 0) mbar_wait_bounded(q_full, (n_piece - 1) & 1, limit, nullptr);
            }
        } else if (C::TMA) {
            // -------------------------------------------------------- V rows that no row may see
            int at = 0;
            uint32_t raw_phase = 0;
            while (ok) {
                const volatile PrefillPiece *x = feed.next(limit, abort_flag, &ok);
                ok = __all_sync(0xffffffffu, ok);
                if (!ok || x == nullptr) break;
                const int s0 = x->s0, s1 = x->s1, first_limit = x->first_limit, L = x->L;
                __syncwarp();
                if (lane == 0) feed.done();
                feed.step();
                for (int step = s0; ok && step < s1; ++step) {
                    const int st = (at + step - s0) % C::VST;
                    if ((step + 1) * kPreKeys <= first_limit) continue;
                    ok = mbar_wait_bounded(&v_raw[st], raw_phase >> st & 1, limit, abort_flag);
                    raw_phase ^= 1u << st;
                    ok = __all_sync(0xffffffffu, ok);
                    if (!ok) break;
                    bool found = false;
                    uint8_t *tile = smem + C::V_OFF + st * C::V_BYTES;
                    const int from = max(0, first_limit - step * kPreKeys), gone = max(0, min(kPreKeys, L - step * kPreKeys));
                    // a quarter warp a 128-byte row piece; the swizzle permutes 16-byte units within it
#pragma unroll
                    for (int c = 0; c < C::VC; ++c) {
                        uint4 *x = reinterpret_cast<uint4 *>(tile + c * (kPreKeys * 128));
                        for (int i = gone * 8 + lane; i < kPreKeys * 8; i += 32) x[i] = make_uint4(0, 0, 0, 0);
                        uint32_t most = 0;  // largest magnitude's bits, two 16-bit halves; infinities and NaN are above all others
#pragma unroll 8
                        for (int i = from * 8 + lane; i < gone * 8; i += 32) {
                            const uint4 y = x[i];
                            most = __vmaxu2(__vmaxu2(most, __vmaxu2(y.x & 0x7fff7fffu, y.y & 0x7fff7fffu)),
                                            __vmaxu2(y.z & 0x7fff7fffu, y.w & 0x7fff7fffu));
                        }
                        if (__any_sync(0xffffffffu, not_finite2<C::F16>(most))) {
                            found = true;
                            for (int i = from * 8 + lane; i < gone * 8; i += 32) {
                                const uint4 y = x[i];
                                x[i] = make_uint4(finite2<C::F16>(y.x), finite2<C::F16>(y.y), finite2<C::F16>(y.z), finite2<C::F16>(y.w));
                            }
                        }
                    }
                    if (found) *bad_v = 1;
                    fence_proxy_async_shared();
                    __threadfence_block();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(&v_full[st]);
                }
                at += s1 - s0;
            }
            if (!ok && lane == 0) {
                flag_error(a.err, kErrTimeout);
                *abort_flag = 1;
            }
        }
        __syncwarp();
    } else {
        // ------------------------------------------------------------ softmax and epilogue: a thread a row
        set_registers<C::LAUNCH_REGS, C::SOFT_REGS>();
        const int t = warp >> 2;
        const int row = threadIdx.x & 127;
        const int tok_in = row / a.g_tile, head_in = row - tok_in * a.g_tile;
        const uint32_t lane_base = tbase + (uint32_t((warp & 3) * 32) << 16);
        const uint32_t s_at = lane_base + C::S_COL + t * kPreKeys;
        uint32_t s_phase = 0, o_phase = 0, stat_phase = 0, q_phase = 0;
        int par_at = 0;  // steps before this piece
        while (ok) {
            const volatile PrefillPiece *p = feed.next(limit, abort_flag, &ok);
            ok = __all_sync(0xffffffffu, ok);
            if (!ok || p == nullptr) break;
            const int tok = tok_in + (p->two ? t * a.tok_tile : 0);
            const bool real = tok_in < a.tok_tile && tok < p->n_tok && p->hb * a.g_tile + head_in < a.G;
            const int seen = !real ? 0 : a.causal ? min(max(p->limit0 + tok, 0), p->L) : p->L;
            const bool idle = !__any_sync(0xffffffffu, real);  // nothing in this warp's rows: it only keeps step
            const int all_see = __reduce_min_sync(0xffffffffu, real ? seen : 0x7fffffff);
            const int most_see = __reduce_max_sync(0xffffffffu, seen);
            const int n_units = p->two ? p->s1 - p->s0 : (p->s1 - p->s0 + 1 - t) / 2;
            float alpha = a.alpha, v_scale = a.v_scale;
            if constexpr (C::F16) {
                if (a.k_scales != nullptr) {
                    alpha *= a.k_scales[a.n_scales > 1 ? p->g : 0];
                    v_scale = a.v_scales[a.n_scales > 1 ? p->g : 0];
                }
            }
            float q_sum = 0.f;  // of the row as the product takes it
            if constexpr (C::F16) {
                if (p->units > 0) {
                    ok = mbar_wait_bounded(q_full, q_phase, limit, abort_flag);
                    q_phase ^= 1;
                    ok = __all_sync(0xffffffffu, ok);
                    if (!ok) break;
                    if (!idle && n_units > 0) {
                        uint8_t *q = smem + C::Q_OFF + t * C::Q_BYTES + row * 128;
                        auto unit = [&](int u) {
                            return reinterpret_cast<uint4 *>(q + (u >> 3) * (kPreTile * 128) + (((u & 7) ^ (row & 7)) << 4));
                        };
                        uint32_t top = 0;  // of the magnitudes' bits, two 16-bit halves
#pragma unroll 4
                        for (int u = 0; u < DQK / 8; ++u) {
                            const uint4 x = *unit(u);
                            top = __vmaxu2(__vmaxu2(top, __vmaxu2(x.x & 0x7fff7fffu, x.y & 0x7fff7fffu)),
                                           __vmaxu2(x.z & 0x7fff7fffu, x.w & 0x7fff7fffu));
                        }
                        const int e = int(max(top & 0xffffu, top >> 16) >> 7);  // exponent field of the largest
                        // the largest comes to [2^14, 2^15); rows of zeros, infinities and NaN stay as they are, and rows
                        // below 2^-113 end lower
                        const int up = e == 0xff ? 0 : min(141 - e, 127);
                        const float two_up = __int_as_float((up + 127) << 23);
                        const float flip = alpha < 0.f ? -two_up : two_up;  // a negative scale goes into Q: the maximum wants a positive one
#pragma unroll 4
                        for (int u = 0; u < DQK / 8; ++u) {
                            const uint4 x = prefill_q_unit<SRC>(*unit(u), flip);
                            if constexpr (C::K_PARAMS) {
                                const uint32_t w[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
                                for (int i = 0; i < 4; ++i) {
                                    const float2 f = __half22float2(*reinterpret_cast<const __half2 *>(&w[i]));
                                    q_sum += f.x + f.y;
                                }
                            }
                            *unit(u) = x;
                        }
                        alpha = ldexpf(fabsf(alpha), -up);
                        fence_proxy_async_shared();
                    }
                    mbar_arrive(&q_ready[t]);
                }
            }
            if (alpha < 1e-37f) alpha = 1e-37f;  // a scale of zero must not make NaN of a masked score
            float m_ref = -INFINITY, l = 0.f;  // reference (log2 domain), sum of the weights
            for (int first = 0; ok && first < n_units; first += kPreDrain) {
                if (first > 0) {  // (a look at the next step's scores, which the loop below waits for)
                    ok = __all_sync(0xffffffffu, mbar_wait_bounded(&s_full[t], s_phase, limit, abort_flag));
                    if (!ok) break;
                    if (!idle) {
                        tc_fence_after_sync();
                        prefill_drain<DV>(a, lane_base + C::O_COL + t * DV, t, m_ref, first > kPreDrain, false);
                    }
                }
                const int stop = min(n_units, first + kPreDrain);
#pragma unroll 1
                for (int i = first; i < stop; ++i) {
                    ok = mbar_wait_bounded(&s_full[t], s_phase, limit, abort_flag);
                    s_phase ^= 1;
                    ok = __all_sync(0xffffffffu, ok);
                    if (!ok) break;
                    if (!idle) {
                        tc_fence_after_sync();
                        const int step = p->s0 + (p->two ? i : 2 * i + t), key0 = step * kPreKeys;
                        const bool masked = key0 + kPreKeys > all_see;
                        const int left = seen - key0;
                        float m4[4];
                        // Scores stay raw: the scale enters through the maximum (exact: it is positive) and one fma a weight.
                        auto hide = [&](uint32_t (&x)[32], int h) {
                            const int n = left - h * 32;
#pragma unroll
                            for (int c = 0; c < 32; ++c)
                                if (c >= n) x[c] = __float_as_uint(-INFINITY);
                        };
                        auto maximum = [&](const uint32_t (&x)[32]) {  // four chains of three-input maxima (exact)
#pragma unroll
                            for (int c = 0; c < 32; c += 2)
                                m4[(c >> 1) & 3] = fmax3(m4[(c >> 1) & 3], __uint_as_float(x[c]), __uint_as_float(x[c + 1]));
                        };
                        float2 sum2[2];
                        // weights exp2(alpha s - reference), two keys at a time (each lane rounded as fmaf would), summed in fp32
                        // before they are rounded for the product
                        const float2 al2 = make_float2(alpha, alpha);
                        auto weigh = [&](const uint32_t (&x)[32], uint32_t *pk, float2 nm2) {
#pragma unroll
                            for (int c = 0; c < 32; c += 2) {
                                const float2 y = fma2(make_float2(__uint_as_float(x[c]), __uint_as_float(x[c + 1])), al2, nm2);
                                const float2 w = make_float2(fast_exp2(y.x), fast_exp2(y.y));
                                sum2[(c >> 1) & 1] = add2(sum2[(c >> 1) & 1], w);
                                pk[c / 2] = C::F16 ? pack_f16x2(w.x, w.y) : pack_bf16x2(w.x, w.y);
                            }
                        };
                        // A row's reference follows its maximum when that passes it by too much; O and the sum then change with it.
                        auto follow = [&]() {
                            constexpr float top = C::F16 ? kPreTopF16 : 0.f;
                            constexpr float most = kPreRescaleLog2 + top - (C::K_PARAMS ? kPreLargeV : 0);
                            // (Rounded one by one: contracted with the product, a difference to a reference of great magnitude would
                            // not be small once the reference has moved.  The sum rounds down, so that past 2^27 no weight passes 2^15.)
                            const float mx = __fmul_rn(fmaxf(fmaxf(m4[0], m4[1]), fmaxf(m4[2], m4[3])), alpha);
                            const bool renew = mx > __fadd_rd(m_ref, most);
                            const bool rescale = renew && i > 0 && m_ref != -INFINITY;
                            const float ref = C::F16 ? __fsub_rn(mx, top) : mx;
                            if (__any_sync(0xffffffffu, rescale)) {
                                const float corr = rescale ? fast_exp2(m_ref - ref) : 1.f;
#pragma unroll 1
                                for (int c = 0; c < DV / 32; ++c) {
                                    uint32_t ov[32];
                                    tmem_ld32(lane_base + C::O_COL + t * DV + c * 32, ov);
                                    tmem_wait_ld();
#pragma unroll
                                    for (int e = 0; e < 32; e += 2) {
                                        const float2 o2 = mul2(make_float2(__uint_as_float(ov[e]), __uint_as_float(ov[e + 1])),
                                                               make_float2(corr, corr));
                                        ov[e] = __float_as_uint(o2.x);
                                        ov[e + 1] = __float_as_uint(o2.y);
                                    }
                                    tmem_st32(lane_base + C::O_COL + t * DV + c * 32, ov);
                                }
                                l *= corr;
                            }
                            if (renew) m_ref = ref;
                            return renew;
                        };
                        if constexpr (C::K_PARAMS) {
                            // Scale and zero of the keys applied first, 32 keys after the other, and the scores put back (held in
                            // registers they spilled: 350 us against 331 on chunks of 300 tokens); parameters and scores of the
                            // next are under way meanwhile (beside the tensor core's reads of shared memory theirs take long).
                            const float4 *par = reinterpret_cast<const float4 *>(smem + C::PAR_OFF + (par_at + step - p->s0) % C::PST * C::PAR_BYTES);
                            const float2 qs2 = make_float2(q_sum, q_sum);
                            float4 pr[2][8];  // scales and zeros of two keys each
                            uint32_t x[2][32];
                            m4[0] = m4[1] = m4[2] = m4[3] = -INFINITY;
                            tmem_ld32(s_at, x[0]);
#pragma unroll
                            for (int e = 0; e < 8; ++e) pr[0][e] = par[e];
#pragma unroll
                            for (int h = 0; h < 4; ++h) {
                                tmem_wait_ld();
                                if (h < 3) tmem_ld32(s_at + (h + 1) * 32, x[(h + 1) & 1]);
                                uint32_t (&y)[32] = x[h & 1];
#pragma unroll
                                for (int half = 0; half < 2; ++half) {
                                    if (h < 3 || half == 0) {
#pragma unroll
                                        for (int e = 0; e < 8; ++e) pr[(half + 1) & 1][e] = par[(h * 2 + half + 1) * 8 + e];
                                    }
#pragma unroll
                                    for (int e = 0; e < 8; ++e) {
                                        const float4 z = pr[half][e];
                                        const int c = half * 16 + 2 * e;
                                        const float2 v = fma2(make_float2(__uint_as_float(y[c]), __uint_as_float(y[c + 1])), make_float2(z.x, z.y),
                                                              mul2(qs2, make_float2(z.z, z.w)));
                                        y[c] = __float_as_uint(v.x);
                                        y[c + 1] = __float_as_uint(v.y);
                                    }
                                }
                                if (masked) hide(y, h);
                                maximum(y);
                                tmem_st32(s_at + h * 32, y);
                            }
                            tmem_wait_st();
                            follow();
                            const float m_use = m_ref == -INFINITY ? 0.f : m_ref;
                            uint32_t pk[kPreKeys / 2];
                            tmem_ld32(s_at, x[0]);
                            sum2[0] = sum2[1] = make_float2(0.f, 0.f);
#pragma unroll
                            for (int h = 0; h < 4; ++h) {
                                tmem_wait_ld();
                                if (h < 3) tmem_ld32(s_at + (h + 1) * 32, x[(h + 1) & 1]);
                                weigh(x[h & 1], pk + h * 16, make_float2(-m_use, -m_use));
                            }
#pragma unroll
                            for (int h = 0; h < 2; ++h) tmem_st32(s_at + h * 32, *reinterpret_cast<const uint32_t (*)[32]>(&pk[h * 32]));
                            // 32 keys each whose values are divided: their weights once more, times 2^4 (in the loop above, or in
                            // registers behind it, this cost every step 3 to 6 %)
                            const unsigned large = *reinterpret_cast<const unsigned *>(&par[kPreKeys / 2]);
                            if (large != 0) {
                                tmem_wait_st();
#pragma unroll 1
                                for (int h = 0; h < 2; ++h) {
                                    tmem_ld32(s_at + h * 32, x[0]);
                                    tmem_wait_ld();
#pragma unroll
                                    for (int c = 0; c < 32; ++c) {
                                        const __half2 by = __float2half2_rn(large >> (h * 16 + c / 16 * 8) & 1 ? 16.f : 1.f);
                                        const __half2 y = __hmul2(*reinterpret_cast<const __half2 *>(&x[0][c]), by);
                                        x[0][c] = *reinterpret_cast<const uint32_t *>(&y);
                                    }
                                    tmem_st32(s_at + h * 32, x[0]);
                                }
                            }
                        } else if (masked) {
                            // 32 keys after the other, those that no row of the warp sees left out (in short prompts half of them):
                            // the maximum, then the weights from scores read once more
                            const int most = most_see - key0;
                            m4[0] = m4[1] = m4[2] = m4[3] = -INFINITY;
#pragma unroll 1
                            for (int h = 0; h * 32 < min(most, kPreKeys); ++h) {
                                uint32_t x[32];
                                tmem_ld32(s_at + h * 32, x);
                                tmem_wait_ld();
                                hide(x, h);
                                maximum(x);
                            }
                            follow();
                            const float m_use = m_ref == -INFINITY ? 0.f : m_ref;
                            sum2[0] = sum2[1] = make_float2(0.f, 0.f);
#pragma unroll 1
                            for (int h = 0; h < kPreKeys / 32; ++h) {
                                uint32_t w[16] = {};
                                if (h * 32 < most) {
                                    uint32_t x[32];
                                    tmem_ld32(s_at + h * 32, x);
                                    tmem_wait_ld();
                                    hide(x, h);
                                    weigh(x, w, make_float2(-m_use, -m_use));
                                }
                                tmem_st16(s_at + h * 16, w);  // (columns whose scores have been read)
                            }
                        } else if constexpr (C::TMA) {
                            // a row's scores in registers: the maximum, then the weights
                            uint32_t pk[kPreKeys / 2];
                            uint32_t sr[4][32];
#pragma unroll
                            for (int h = 0; h < 4; ++h) tmem_ld32(s_at + h * 32, sr[h]);
                            tmem_wait_ld();
                            m4[0] = m4[1] = m4[2] = m4[3] = -INFINITY;
#pragma unroll
                            for (int h = 0; h < 4; ++h) {
                                maximum(sr[h]);
                            }
                            follow();
                            const float m_use = m_ref == -INFINITY ? 0.f : m_ref;
                            sum2[0] = sum2[1] = make_float2(0.f, 0.f);
#pragma unroll
                            for (int h = 0; h < 4; ++h) {
                                weigh(sr[h], pk + h * 16, make_float2(-m_use, -m_use));
                            }
                            // All of them at the end: a store holds its registers for some 180 cycles, which stores between the
                            // pieces would wait for.
#pragma unroll
                            for (int h = 0; h < 2; ++h) tmem_st32(s_at + h * 32, *reinterpret_cast<const uint32_t (*)[32]>(&pk[h * 32]));
                        } else {
                            // Registers for half of them: maximum and weights in one pass with the reference as it is, once more in the
                            // few steps whose maximum passes it (read a second time for the weights always: mixed step over an FP8
                            // cache 1652 us against 1243).
                            uint32_t pk[kPreKeys / 2];
#pragma unroll 1
                            for (int pass = 0; pass < 2; ++pass) {
                                const float m_use = m_ref == -INFINITY ? 0.f : m_ref;
                                const float2 nm2 = make_float2(-m_use, -m_use);
                                m4[0] = m4[1] = m4[2] = m4[3] = -INFINITY;
                                sum2[0] = sum2[1] = make_float2(0.f, 0.f);
                                uint32_t sr[2][32];
                                tmem_ld32(s_at, sr[0]);
#pragma unroll
                                for (int h = 0; h < 4; ++h) {
                                    tmem_wait_ld();
                                    if (h < 3) tmem_ld32(s_at + (h + 1) * 32, sr[(h + 1) & 1]);
                                    maximum(sr[h & 1]);
                                    weigh(sr[h & 1], pk + h * 16, nm2);
                                }
                                if (!__any_sync(0xffffffffu, follow())) break;
                            }
#pragma unroll
                            for (int h = 0; h < 2; ++h) tmem_st32(s_at + h * 32, *reinterpret_cast<const uint32_t (*)[32]>(&pk[h * 32]));
                        }
                        tmem_wait_st();
                        l += (sum2[0].x + sum2[1].x) + (sum2[0].y + sum2[1].y);
                        tc_fence_before_sync();
                    }
                    mbar_arrive(&p_full[t]);
                }
            }
            if (!ok) break;
            par_at += p->s1 - p->s0;

            // ---- epilogue: row group t's own rows, or (one tile) group 0 for both
            const bool join = !p->two && p->units > 1;
            if (n_units > 0) {
                ok = mbar_wait_bounded(&o_full[t], o_phase, limit, abort_flag);
                o_phase ^= 1;
            }
            if (join && t == 0) {  // group 1 hands its part over once its own O is there
                ok = ok && mbar_wait_bounded(stat_full, stat_phase, limit, abort_flag);
                stat_phase ^= 1;
            }
            ok = __all_sync(0xffffffffu, ok);
            if (!ok) break;
            tc_fence_after_sync();
            if (n_units > kPreDrain && !idle) prefill_drain<DV>(a, lane_base + C::O_COL + t * DV, t, m_ref, true, true);
            if (join && t == 1) {
                stat[row] = make_float2(m_ref, l);
                tc_fence_before_sync();
                mbar_arrive(stat_full);
                ok = __all_sync(0xffffffffu, mbar_wait_bounded(stat_free, stat_phase, limit, abort_flag));
                stat_phase ^= 1;
                if (!ok) break;
            }
            if (p->two || t == 0) {
                float f0 = 1.f, f1 = 0.f;
                if (join) {
                    const float2 other = stat[row];
                    const float m = fmaxf(m_ref, other.x), use = m == -INFINITY ? 0.f : m;
                    f0 = fast_exp2(m_ref - use);
                    f1 = fast_exp2(other.x - use);
                    l = l * f0 + other.y * f1;
                    m_ref = m;
                }
                if (!idle) {
                    // a row that sees no key here is zeros, whatever a scale of NaN made of its masked scores (a sum of NaN is not zero)
                    const bool any = seen > p->s0 * kPreKeys && l != 0.f;
                    const float inv = any ? v_scale / l : 0.f;
                    const float lse2 = any ? m_ref + log2f(l) : -INFINITY;
                    const bool fix = n_units > 0 && p->s1 * kPreKeys > p->first_limit && *bad_v != 0;
                    const long long out_row = (long long)(p->q_row + tok) * a.Hq + p->g * a.G + p->hb * a.g_tile + head_in;
                    const int part_row = (p->slot * 2 + (p->two ? t : 0)) * kPreTile + row;
                    // A row's 64 bytes go out by four lanes (a 16-byte piece each; a lane alone would touch 32 rows an
                    // instruction): lanes of a quad exchange pieces, and lane q writes piece q of the quad's rows in turn.
                    const long long mine = p->slot < 0 ? out_row * DV * 2 : (long long)part_row * DV * 4;
                    char *rows[4];
                    const unsigned there = __ballot_sync(0xffffffffu, real) >> (lane & ~3);
#pragma unroll
                    for (int r = 0; r < 4; ++r) {
                        rows[r] = (p->slot < 0 ? reinterpret_cast<char *>(a.out) : reinterpret_cast<char *>(a.o_part)) +
                                  __shfl_sync(0xffffffffu, mine, (lane & ~3) + r) + (lane & 3) * 16;
                    }
#pragma unroll 1
                    for (int c = 0; c < DV / 32; ++c) {
                        float o[32];
                        if (n_units > 0) {
                            uint32_t ov[32];
                            tmem_ld32(lane_base + C::O_COL + t * DV + c * 32, ov);
                            if (join) {
                                uint32_t ow[32];
                                tmem_ld32(lane_base + C::O_COL + DV + c * 32, ow);
                                tmem_wait_ld();
#pragma unroll
                                for (int e = 0; e < 32; ++e)
                                    o[e] = (__uint_as_float(ov[e]) * f0 + __uint_as_float(ow[e]) * f1) * inv;
                            } else {
                                tmem_wait_ld();
#pragma unroll
                                for (int e = 0; e < 32; ++e) o[e] = __uint_as_float(ov[e]) * inv;
                            }
                        }
                        if (!any) {
#pragma unroll
                            for (int e = 0; e < 32; ++e) o[e] = 0.f;
                        }
                        if constexpr (SRC == kPreInt4) {  // back from the order that 4-bit codes come in
#pragma unroll
                            for (int e = 0; e < 32; e += 8) {
                                const float x1 = o[e + 1], x2 = o[e + 2], x3 = o[e + 3], x4 = o[e + 4], x5 = o[e + 5], x6 = o[e + 6];
                                o[e + 1] = x2, o[e + 2] = x4, o[e + 3] = x6, o[e + 4] = x1, o[e + 5] = x3, o[e + 6] = x5;
                            }
                        }
                        if (p->slot < 0) {
                            uint32_t x[16];
#pragma unroll
                            for (int e = 0; e < 16; ++e) x[e] = pack_bf16x2(o[2 * e], o[2 * e + 1]);
                            quad_transpose(x, lane);
#pragma unroll
                            for (int r = 0; r < 4; ++r)
                                if (there >> r & 1)
                                    *reinterpret_cast<uint4 *>(rows[r] + c * 64) = make_uint4(x[4 * r], x[4 * r + 1], x[4 * r + 2], x[4 * r + 3]);
                        } else {
#pragma unroll
                            for (int half = 0; half < 2; ++half) {
                                uint32_t x[16];
#pragma unroll
                                for (int e = 0; e < 16; ++e) x[e] = __float_as_uint(o[half * 16 + e]);
                                quad_transpose(x, lane);
#pragma unroll
                                for (int r = 0; r < 4; ++r)
                                    if (there >> r & 1)
                                        *reinterpret_cast<uint4 *>(rows[r] + c * 128 + half * 64) =
                                            make_uint4(x[4 * r], x[4 * r + 1], x[4 * r + 2], x[4 * r + 3]);
                            }
                        }
                    }
                    __syncwarp();  // a row's elements were written by its quad
                    if (fix && any) {
                        const int key0 = max(p->first_limit, p->s0 * kPreKeys), key1 = min(seen, p->s1 * kPreKeys);
                        if (p->slot < 0)
                            prefill_add_not_finite<DV, SRC>(a, p->req, p->k_row, p->g, key0, key1, a.out + out_row * DV);
                        else
                            prefill_add_not_finite<DV, SRC>(a, p->req, p->k_row, p->g, key0, key1,
                                                            a.o_part + (long long)part_row * DV);
                    }
                    if (real) {
                        if (p->slot >= 0) a.lse_part[part_row] = lse2;
                        else if (a.lse != nullptr) a.lse[out_row] = lse2 * 0.69314718055994530942f;
                    }
                }
                if (join) {
                    tc_fence_before_sync();
                    mbar_arrive(stat_free);
                }
            }
            tc_fence_before_sync();  // O is read before the next piece's first weights are handed over
            __syncwarp();
            if (lane == 0) feed.done();
            feed.step();
        }
        if (!ok) {
            flag_error(a.err, kErrTimeout);
            *abort_flag = 1;
        }
        __syncwarp();
    }

    // every product is done (the issuer waited for it) and every TMEM access made
    tc_fence_before_sync();
    __syncthreads();
    if (warp == 8) {
        tc_fence_after_sync();
        tmem_dealloc(tbase, C::TMEM_COLS);
    }
}

// Joins the partial results of items whose steps several workers hold: CTA (j, b) rows 32 b .. of the j-th of them.  The
// weights of all its rows and parts first, then the rows' pieces, 16 bytes a thread, in the parts' order.
constexpr int kPreMergeRows = 32, kPreMergeThreads = 256, kPreMergeParts = 64;  // parts whose weights are held at a time

template <int DV>
__global__ void __launch_bounds__(kPreMergeThreads) gqa_prefill_merge_kernel(const __grid_constant__ PrefillArgs a) {
    __shared__ float weight[kPreMergeParts][kPreMergeRows];
    __shared__ float top_s[kPreMergeRows];
    pdl_wait_primary();
    if (int(blockIdx.x) >= a.plan->n_joins) return;
    const int4 join = a.joins[blockIdx.x];
    const int number = join.x;
    const PrefillItem it = a.items[number / a.head_blocks];
    const int r0 = blockIdx.y * kPreMergeRows;
    if (r0 >= kPreTile && it.n_tok <= a.tok_tile) return;
    const int h = number % a.head_blocks, per = a.head_blocks / a.Hkv;
    // part x: what worker first + x did of the item -- the last thing of its share for the first of them, the first for the others
    const int first = join.y, parts = join.z - first + 1;
    auto place_of = [&](int x) { return (x == 0 ? 2 * first + 1 : 2 * (first + x)) * 2 * kPreTile + r0; };
    const int row = threadIdx.x & (kPreMergeRows - 1), lane_part = threadIdx.x / kPreMergeRows;
    constexpr int LANES = kPreMergeThreads / kPreMergeRows;  // parts looked at side by side
    // largest LSE of each row
    float top = -INFINITY;
    for (int x = lane_part; x < parts; x += LANES) {
        top = fmaxf(top, a.lse_part[place_of(x) + row]);
    }
    weight[lane_part][row] = top;
    __syncthreads();
    if (threadIdx.x < kPreMergeRows) {
        for (int x = 1; x < LANES; ++x) top = fmaxf(top, weight[x][row]);
        top_s[row] = top == -INFINITY ? 0.f : top;
    }
    __syncthreads();
    constexpr int COLS = DV / 4, PASS = kPreMergeThreads / COLS, N = kPreMergeRows / PASS;  // rows at a time, rows of a thread
    const int d = threadIdx.x % COLS * 4, sub = threadIdx.x / COLS;
    float4 o[N] = {};
    float total[N] = {};
    for (int x0 = 0; x0 < parts; x0 += kPreMergeParts) {
        const int here = min(kPreMergeParts, parts - x0);
        for (int x = lane_part; x < here; x += LANES)
            weight[x][row] = exp2f(a.lse_part[place_of(x0 + x) + row] - top_s[row]);
        __syncthreads();
#pragma unroll 2
        for (int x = 0; x < here; ++x) {
            const int at = place_of(x0 + x);
#pragma unroll
            for (int n = 0; n < N; ++n) {
                const int r = n * PASS + sub;
                const float f = weight[x][r];
                const float4 y = *reinterpret_cast<const float4 *>(a.o_part + (long long)(at + r) * DV + d);
                total[n] += f;
                if (f != 0.f) {  // a part without a key for the row has no share, whatever it holds
                    o[n].x = fmaf(f, y.x, o[n].x), o[n].y = fmaf(f, y.y, o[n].y);
                    o[n].z = fmaf(f, y.z, o[n].z), o[n].w = fmaf(f, y.w, o[n].w);
                }
            }
        }
        __syncthreads();
    }
#pragma unroll
    for (int n = 0; n < N; ++n) {
        const int r = r0 + n * PASS + sub, tile = r / kPreTile, in = r % kPreTile;
        const int tok_in = in / a.g_tile, tok = tile * a.tok_tile + tok_in, head = h % per * a.g_tile + in % a.g_tile;
        if (tok_in >= a.tok_tile || tok >= it.n_tok || head >= a.G) continue;
        const float inv = total[n] == 0.f ? 0.f : 1.f / total[n];
        const long long to = (long long)(it.q_row + tok) * a.Hq + h / per * a.G + head;
        *reinterpret_cast<uint2 *>(a.out + to * DV + d) =
            make_uint2(pack_bf16x2(o[n].x * inv, o[n].y * inv), pack_bf16x2(o[n].z * inv, o[n].w * inv));
        if (a.lse != nullptr && d == 0)
            a.lse[to] = total[n] == 0.f ? -INFINITY : (top_s[r - r0] + log2f(total[n])) * 0.69314718055994530942f;
    }
}

}  // namespace gqa
