// gqa_prefill_load.cuh -- layout of the prompt attention's shared memory, and the loads of K and V that go through
// registers: pools of codes, converted to fp16, and bf16 pools whose pages are no multiple of 8 tokens.
#pragma once

#include <type_traits>

#include "gqa_prefill_plan.cuh"

namespace gqa {

// 4-bit values may pass fp16's largest (15 scales and a zero: up to 2^20).  32 keys one of whose values may enter the product
// divided by 2^kPreLargeV, and their weights times that.
constexpr int kPreLargeV = 4;

template <int DQK, int DV, int SRC>
struct PrefillCfg {
    static constexpr bool F16 = SRC >= kPreFp8;  // operands: fp16 (codes), else bf16
    static constexpr bool TMA = SRC == kPreDense || SRC == kPrePages;
    static constexpr bool K_PARAMS = SRC == kPreInt4;  // scores take a scale and a zero of each key
    static constexpr int QC = DQK / 64, VC = DV / 64;  // 64-element chunks (one 128-byte swizzle row each)
    static constexpr int Q_BYTES = QC * kPreTile * 128;
    static constexpr int K_BYTES = QC * kPreKeys * 128;
    static constexpr int V_BYTES = VC * kPreKeys * 128;
    static constexpr int KST = DQK == 192 || (DQK == 128 && F16) ? 2 : DQK == 128 ? 3 : F16 ? 4 : 5;
    static constexpr int VST = DQK == 192 ? 1 : DQK == 128 ? 2 : F16 ? 4 : 5;
    // A key's parameters are read until its step's weights are out: when a stage of K is free for the KST-th step after it,
    // the weights of the second step before that one are (one tile an item; of the first with two).
    static constexpr int PST = KST + 2;
    static constexpr int PAR_BYTES = kPreKeys * 8 + 16;  // scales of two keys and their zeros, 64 times; a byte for each 32 keys: values divided
    static constexpr int Q_OFF = 0;
    static constexpr int K_OFF = 2 * Q_BYTES;
    static constexpr int V_OFF = K_OFF + KST * K_BYTES;
    static constexpr int STAT_OFF = V_OFF + VST * V_BYTES;  // [128] float2: what row group 1 hands over
    static constexpr int PIECE_OFF = STAT_OFF + 1024;       // pieces that are known ahead
    static constexpr int PAR_OFF = PIECE_OFF + kPrePieces * 64;  // [PST] parameters of a step
    static constexpr int RAW_OFF = PAR_OFF + (K_PARAMS ? PST * PAR_BYTES : 0);  // codes of K and of V on their way
    static constexpr int RAW_BYTES = !F16 ? 0 : kPreKeys * DV / (SRC == kPreInt4 ? 2 : 1);
    static constexpr int BAR_OFF = RAW_OFF + 2 * RAW_BYTES;
    static constexpr int SMEM = BAR_OFF + 512 + 1024;
    static_assert(SMEM <= 227 * 1024, "shared memory");
    // Registers by warp group, shared out anew from the launch's 168 or 128 a thread (softmax, the group of warp 8, loaders).
    static constexpr int THREADS = TMA ? 384 : 512;
    static constexpr int SOFT_REGS = TMA ? 224 : 192, OTHER_REGS = TMA ? 56 : 48, LOAD_REGS = 80;
    static constexpr int REGS = 256 * SOFT_REGS + 128 * OTHER_REGS + (TMA ? 0 : 128 * LOAD_REGS);
    static constexpr int LAUNCH_REGS = 65536 / THREADS / 8 * 8;
    static_assert(REGS <= LAUNCH_REGS * THREADS, "registers");
    static constexpr uint32_t S_COL = 0, O_COL = 2 * kPreKeys;
    static constexpr uint32_t TMEM_COLS = 512;
    static_assert(O_COL + 2 * DV <= TMEM_COLS, "TMEM");
};

// The warp group's registers a thread from here on; FROM is what it was launched with.  (Giving registers back with a
// number above the present one, or asking for more with one below, is undefined.)
template <int FROM, int N>
__device__ __forceinline__ void set_registers() {
    static_assert(N % 8 == 0 && N >= 24 && N <= 256, "registers");
    if constexpr (N > FROM) asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(N));
    if constexpr (N < FROM) asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(N));
}

// Any of the two 16-bit halves infinite or NaN.
template <bool F16>
__device__ __forceinline__ bool not_finite2(uint32_t x) {
    const uint32_t e = F16 ? 0x7c00u : 0x7f80u;
    return (x & e) == e || (x >> 16 & e) == e;
}

// Zeros in the place of halves that are infinite or NaN.
template <bool F16>
__device__ __forceinline__ uint32_t finite2(uint32_t x) {
    const uint32_t e = F16 ? 0x7c00u : 0x7f80u;
    if ((x & e) == e) x &= 0xffff0000u;
    if ((x >> 16 & e) == e) x &= 0x0000ffffu;
    return x;
}

// key / page_size by a product (exact below 2^31).
__device__ __forceinline__ int prefill_page(const PrefillArgs &a, int key) {
    return int((unsigned long long)unsigned(key) * a.page_mul >> a.page_shift);
}

// Pool row of a request's key, or -1 (flagged) where its page is out of range.
__device__ __forceinline__ int prefill_pool_row(const PrefillArgs &a, int req, int key) {
    const int in_req = prefill_page(a, key);
    const int page = a.page_table[(long long)req * a.pages_per_req + in_req];
    if (page < 0 || page >= a.num_pages) {
        flag_error(a.err, kErrIndex);
        return -1;
    }
    return page * a.page_size + key - in_req * a.page_size;
}

// Four fp16 pairs of eight 8-bit or 4-bit codes.
template <int SRC>
__device__ __forceinline__ uint32_t widen_pair(uint32_t word, int pair) {
    if constexpr (SRC == kPreFp8) {
        return e4m3x2_to_f16x2(uint16_t(pair == 0 ? word : word >> 16));
    } else {  // int8: the code in the mantissa of 1024 + 128 + c
        uint32_t x;
        asm("prmt.b32 %0, %1, %2, %3;" : "=r"(x) : "r"(word ^ 0x80808080u), "r"(0x64646464u), "r"(pair == 0 ? 0x4140u : 0x4342u));
        const __half2 y = __hsub2(*reinterpret_cast<const __half2 *>(&x), __half2(__half_raw{0x6480}, __half_raw{0x6480}));
        return *reinterpret_cast<const uint32_t *>(&y);
    }
}

// Codes i and i + 4 of eight 4-bit codes (element 2 k in the low half of byte k) as an fp16 pair.
__device__ __forceinline__ __half2 widen_int4(uint32_t word, int i) {
    const uint32_t x = (word >> (4 * i) & 0x000f000fu) | 0x64006400u;  // 1024 + code
    return __hsub2(*reinterpret_cast<const __half2 *>(&x), __half2(__half_raw{0x6400}, __half_raw{0x6400}));
}

__device__ __forceinline__ void cp_async16_or_zero(uint32_t smem_dst, const void *src, bool there) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(smem_dst), "l"(src), "r"(there ? 16 : 0) : "memory");
}

// Four warps, each 32 keys of every step: a lane looks up its key's pool row, the row's 16-byte pieces go to the lanes so
// that reads are whole sectors and the writes of a quarter warp cover all banks.  Returns false after a wait that ran out.
template <int DQK, int DV, int SRC>
__device__ __forceinline__ bool prefill_load(const PrefillArgs &a, uint8_t *smem, uint64_t *k_full, uint64_t *k_empty,
                                             uint64_t *v_full, uint64_t *v_empty, PieceFeed feed, volatile int *abort_flag,
                                             volatile int *bad_v) {
    using C = PrefillCfg<DQK, DV, SRC>;
    static_assert(DQK == DV, "pools");
    const int lane = threadIdx.x & 31, lw = (threadIdx.x >> 5) & 3;
    const uint64_t limit = a.wait_limit_ns;
    constexpr int CHUNK = kPreKeys * 128;  // bytes
    bool ok = true;
    struct { int req, L, g, s0, s1, first_limit; } p = {};  // of the piece
    auto masked = [&](int step) { return (step + 1) * kPreKeys > p.first_limit; };
    // The next piece with steps.  before_wait() runs where it is not there yet: the pieces ahead are published as the softmax
    // is done with those behind, so nothing that the softmax waits for may be held back during this wait.
    auto next = [&](auto before_wait) {
        const volatile PrefillPiece *x;
        do {
            if (!__all_sync(0xffffffffu, feed.ready())) before_wait();
            x = feed.next(limit, abort_flag, &ok);
            ok = __all_sync(0xffffffffu, ok);
            if (!ok || x == nullptr) return false;
            p = {x->req, x->L, x->g, x->s0, x->s1, x->first_limit};
            const bool some = x->units > 0;
            __syncwarp();
            if (lane == 0) feed.done();
            feed.step();
            if (some) return true;
        } while (true);
    };
    int at = 0;  // steps so far

    if constexpr (SRC == kPreCopy) {
        // 16-byte asynchronous copies.  K and V of a step are handed on once the copies after them are under way, or before a
        // wait that may depend on them: for a free stage, and for the next piece (behind the last step of a piece, items
        // without steps may fill the ring of pieces, whose first place is only free once that step's V has been used).
        constexpr int PIECES = DV / 8, ROWS = 32 / 8;  // of a row; rows of a warp's copy (8 pieces of one chunk each)
        struct { uint64_t *bar; uint8_t *clean; int from; } pend[2] = {};
        int n_pend = 0;
        auto hand_on = [&](int keep) {  // all but the newest `keep` copies
            if (n_pend <= keep) return;
            if (keep == 1) asm volatile("cp.async.wait_group 1;" ::: "memory");
            else asm volatile("cp.async.wait_group 0;" ::: "memory");
            const int n = n_pend - keep;
            for (int i = 0; i < n; ++i) {
                if (pend[i].clean != nullptr) {  // a step past what some row sees: this lane's own pieces
                    bool found = false;
                    for (int x = 0; x < 32 / ROWS; ++x) {
                        const int key = lw * 32 + x * ROWS + (lane >> 3);
                        if (key < pend[i].from) continue;
                        for (int c = 0; c < C::VC; ++c) {
                            uint4 *y = reinterpret_cast<uint4 *>(pend[i].clean + c * CHUNK + key * 128 + (((lane & 7) ^ (key & 7)) << 4));
                            const uint4 v = *y;
                            if (not_finite2<false>(v.x) || not_finite2<false>(v.y) || not_finite2<false>(v.z) || not_finite2<false>(v.w)) {
                                found = true;
                                *y = make_uint4(finite2<false>(v.x), finite2<false>(v.y), finite2<false>(v.z), finite2<false>(v.w));
                            }
                        }
                    }
                    if (found) *bad_v = 1;
                }
                fence_proxy_async_shared();
                __threadfence_block();
                if (pend[i].bar != nullptr) mbar_arrive(pend[i].bar);
            }
            pend[0] = pend[1];
            n_pend = keep;
        };
        while (ok && next([&]() { hand_on(0); })) {
            for (int step = p.s0; ok && step < p.s1; ++step, ++at) {
                const int key = step * kPreKeys + lw * 32 + lane;
                const int row = key < p.L ? prefill_pool_row(a, p.req, key) : -1;
#pragma unroll 1
                for (int v = 0; v < 2; ++v) {
                    const int stages = v ? C::VST : C::KST, st = at % stages;
                    if (at >= stages) {
                        uint64_t *empty = v ? &v_empty[st] : &k_empty[st];
                        const uint32_t parity = (at / stages - 1) & 1;
                        if (!__all_sync(0xffffffffu, mbar_try_wait(empty, parity))) {
                            hand_on(0);
                            ok = __all_sync(0xffffffffu, mbar_wait_bounded(empty, parity, limit, abort_flag));
                            if (!ok) break;
                        }
                    }
                    uint8_t *dst = smem + (v ? C::V_OFF + st * C::V_BYTES : C::K_OFF + st * C::K_BYTES);
                    const uint8_t *pool = v ? a.v_pool : a.k_pool;
#pragma unroll
                    for (int x = 0; x < 32 / ROWS; ++x) {
                        const int in = x * ROWS + (lane >> 3), k = lw * 32 + in;
                        const int r = __shfl_sync(0xffffffffu, row, in);
                        const uint8_t *src = pool + (((long long)max(r, 0) * a.Hkv + p.g) * PIECES + (lane & 7)) * 16;
#pragma unroll
                        for (int c = 0; c < C::VC; ++c)
                            cp_async16_or_zero(smem_u32(dst + c * CHUNK + k * 128 + (((lane & 7) ^ (k & 7)) << 4)), src + c * 128, r >= 0);
                    }
                    asm volatile("cp.async.commit_group;" ::: "memory");
                    const bool withheld = a.fault_mode == 1 && !v && at == 0;  // test hook: this stage never fills
                    pend[n_pend] = {withheld ? nullptr : v ? &v_full[st] : &k_full[st], v && masked(step) ? dst : nullptr,
                                    p.first_limit - step * kPreKeys};
                    ++n_pend;
                    hand_on(1);
                }
            }
        }
        hand_on(0);
        cp_async_wait_all();
    } else {
        // Codes: a step's pieces of K are on their way while V's are converted and the other way round.  They wait in shared
        // memory, each thread's where nobody else looks, so that a thread only waits for its own copies.  (In registers they
        // came through L1, which beside this much shared memory is smaller than what should be on its way: a mixed step of 32
        // requests over an FP8 cache took 2836 us against 2473.)
        constexpr int PER = SRC == kPreInt4 ? 2 : 4;        // pieces of a 64-element chunk
        constexpr int ROWS = 32 / PER;                      // rows of a warp's load
        constexpr int N = 32 / ROWS * C::VC;                // loads of a lane
        constexpr int ROW_BYTES = SRC == kPreInt4 ? DV / 2 : DV;
        const int in_chunk = lane & (PER - 1), in_rows = lane / PER;
        const uint32_t raw = smem_u32(smem + C::RAW_OFF) + (threadIdx.x & 127) * 16;
        const int row_bytes = a.Hkv * ROW_BYTES;
        uint2 par = {}, next_par = {};
        int row = -1, next_row = -1;
        // Page ids two steps ahead, rows one step ahead: nothing waits for a load that it has just asked for.
        int page = 0;
        const int *table = nullptr;
        auto look_ahead = [&](int step) {
            const int key = step * kPreKeys + lw * 32 + lane;
            if (key < p.L) page = table[prefill_page(a, key)];
        };
        auto look_up = [&](int step) {
            const int key = step * kPreKeys + lw * 32 + lane;
            next_row = -1;
            if (key < p.L && step < p.s1) {
                if (page < 0 || page >= a.num_pages) flag_error(a.err, kErrIndex);
                else next_row = (page - prefill_page(a, key)) * a.page_size + key;
            }
            if constexpr (SRC == kPreInt4) {
                next_par = make_uint2(0, 0);
                if (next_row >= 0) next_par = __ldg(reinterpret_cast<const uint2 *>(a.params) + (long long)next_row * a.Hkv + p.g);
            }
        };
        // `some` is false behind a piece's last step: nothing is copied, but the group counts for the waits.  (Zeros copied
        // there could land after the next piece's codes: copies to one place are ordered by a wait alone, and store() waits
        // for them only where it reads.)
        auto load = [&](bool is_v, const uint8_t *pool, int r, bool some) {
#pragma unroll
            for (int i = 0; i < N; i += C::VC) {
                if (!some) break;
                const int from = __shfl_sync(0xffffffffu, r, i / C::VC * ROWS + in_rows);
                const uint8_t *src = pool + (long long)max(from, 0) * row_bytes;
#pragma unroll
                for (int x = 0; x < C::VC; ++x)
                    cp_async16_or_zero(raw + (is_v ? C::RAW_BYTES : 0) + (i + x) * 2048, src + x * PER * 16, from >= 0);
            }
            asm volatile("cp.async.commit_group;" ::: "memory");
        };
        // first_clean: keys of the step from here on may hold what some row must not see
        auto store = [&](auto is_v_t, auto clean_t, uint8_t *tile, int first_clean) {
            constexpr bool is_v = decltype(is_v_t)::value, careful = decltype(clean_t)::value;
            bool found = false;
            asm volatile("cp.async.wait_group 1;" ::: "memory");  // all but the other one's newest copies
            constexpr int BATCH = N < 4 ? N : 4;  // pieces read before the first is converted
            uint32_t raw_w[BATCH][4];
#pragma unroll
            for (int i = 0; i < N; ++i) {
                const int in = i / C::VC * ROWS + in_rows, k = lw * 32 + in;
                uint8_t *dst = tile + i % C::VC * CHUNK + k * 128;
                if (i % BATCH == 0) {
#pragma unroll
                    for (int x = 0; x < BATCH; ++x)
                        asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];"
                                     : "=r"(raw_w[x][0]), "=r"(raw_w[x][1]), "=r"(raw_w[x][2]), "=r"(raw_w[x][3])
                                     : "r"(raw + (is_v ? C::RAW_BYTES : 0) + (i + x) * 2048));
                }
                const uint32_t (&w)[4] = raw_w[i % BATCH];
                [[maybe_unused]] __half2 vs = {}, vz = {};
                if constexpr (SRC == kPreInt4) {
                    if constexpr (is_v) {
                        const uint32_t x = __shfl_sync(0xffffffffu, par.y, in);
                        const __half2 y = *reinterpret_cast<const __half2 *>(&x);
                        vs = __low2half2(y), vz = __high2half2(y);
                    }
                }
#pragma unroll
                for (int u = 0; u < 8 / PER; ++u) {
                    uint32_t o[4];
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        if constexpr (SRC == kPreInt4) {
                            __half2 x = widen_int4(w[u], e);
                            if constexpr (is_v) x = __hfma2(x, vs, vz);
                            o[e] = *reinterpret_cast<const uint32_t *>(&x);
                        } else {
                            o[e] = widen_pair<SRC>(w[2 * u + (e >> 1)], e & 1);
                        }
                    }
                    if constexpr (careful && SRC != kPreInt8) {
                        if (k >= first_clean) {
#pragma unroll
                            for (int e = 0; e < 4; ++e) {
                                found |= not_finite2<true>(o[e]);
                                o[e] = finite2<true>(o[e]);
                            }
                        }
                    }
                    *reinterpret_cast<uint4 *>(dst + (((in_chunk * (8 / PER) + u) ^ (k & 7)) << 4)) = make_uint4(o[0], o[1], o[2], o[3]);
                }
            }
            if (found) *bad_v = 1;
        };
        while (ok && next([]() {})) {  // (each step hands its own K and V on)
            const uint8_t *k_pool = a.k_pool + p.g * ROW_BYTES + in_chunk * 16, *v_pool = a.v_pool + p.g * ROW_BYTES + in_chunk * 16;
            table = a.page_table + (long long)p.req * a.pages_per_req;
            look_ahead(p.s0);
            look_up(p.s0);
            row = next_row, par = next_par;
            look_ahead(p.s0 + 1);
            load(false, k_pool, row, true);
            load(true, v_pool, row, true);
            for (int step = p.s0; step < p.s1; ++step, ++at) {
                look_up(step + 1);
                look_ahead(step + 2);
                if constexpr (SRC == kPreInt4) {
                    if ((par.x & 0x7c00u) == 0x7c00u || (par.x & 0x7c000000u) == 0x7c000000u) par.x = 0x7fff7fffu;
                    if ((par.y & 0x7c00u) == 0x7c00u || (par.y & 0x7c000000u) == 0x7c000000u) par.y = 0x7fff7fffu;
                    const float2 f = __half22float2(*reinterpret_cast<const __half2 *>(&par.x));
                    const float scale1 = __shfl_down_sync(0xffffffffu, f.x, 1), zero1 = __shfl_down_sync(0xffffffffu, f.y, 1);
                    const float2 v = __half22float2(*reinterpret_cast<const __half2 *>(&par.y));
                    const bool large = __any_sync(0xffffffffu, fabsf(v.x) * 15.f + fabsf(v.y) > 65504.f);  // (not for NaN)
                    if (large) {  // times 2^-4
                        const __half2 less = __hmul2(*reinterpret_cast<const __half2 *>(&par.y), __half2(__half_raw{0x2c00}, __half_raw{0x2c00}));
                        par.y = *reinterpret_cast<const uint32_t *>(&less);
                    }
                    // (the ring of parameters is free when the stage of K is, see PST)
                    ok = at < C::KST || mbar_wait_bounded(&k_empty[at % C::KST], (at / C::KST - 1) & 1, limit, abort_flag);
                    ok = __all_sync(0xffffffffu, ok);
                    if (!ok) break;
                    uint8_t *par_at = smem + C::PAR_OFF + at % C::PST * C::PAR_BYTES;
                    if ((lane & 1) == 0) reinterpret_cast<float4 *>(par_at)[(lw * 32 + lane) / 2] = make_float4(f.x, scale1, f.y, zero1);
                    if (lane == 0) par_at[kPreKeys * 8 + lw] = large;
                } else {
                    ok = at < C::KST || mbar_wait_bounded(&k_empty[at % C::KST], (at / C::KST - 1) & 1, limit, abort_flag);
                    ok = __all_sync(0xffffffffu, ok);
                    if (!ok) break;
                }
                store(std::false_type(), std::false_type(), smem + C::K_OFF + at % C::KST * C::K_BYTES, 0);
                fence_proxy_async_shared();
                if (!(a.fault_mode == 1 && at == 0)) mbar_arrive(&k_full[at % C::KST]);  // test hook: the first stage never fills
                load(false, k_pool, next_row, step + 1 < p.s1);
                ok = at < C::VST || mbar_wait_bounded(&v_empty[at % C::VST], (at / C::VST - 1) & 1, limit, abort_flag);
                ok = __all_sync(0xffffffffu, ok);
                if (!ok) break;
                if (SRC != kPreInt8 && masked(step))
                    store(std::true_type(), std::true_type(), smem + C::V_OFF + at % C::VST * C::V_BYTES, p.first_limit - step * kPreKeys);
                else
                    store(std::true_type(), std::false_type(), smem + C::V_OFF + at % C::VST * C::V_BYTES, 0);
                fence_proxy_async_shared();
                __threadfence_block();
                mbar_arrive(&v_full[at % C::VST]);
                load(true, v_pool, next_row, step + 1 < p.s1);
                row = next_row, par = next_par;
            }
        }
        cp_async_wait_all();
    }
    return ok;
}

}  // namespace gqa
