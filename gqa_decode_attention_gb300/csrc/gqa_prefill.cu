// gqa_prefill.cu -- attention over packed prompts and of new tokens over the
// paged cache: launches, and the C entry points.
#include <algorithm>
#include <cmath>
#include <mutex>

#include "gqa_common.cuh"
#include "gqa_host.h"
#include "gqa_prefill_kernel.cuh"

namespace gqa {
namespace {

constexpr int kMaxDevices = 64;
constexpr int kMaxWorkers = kPlanThreads;
constexpr unsigned long long kPreWaitStepNs = 32000;

// Tiles of a shape: query heads of a KV head side by side, as many tokens as fit.
void prefill_tiles(PrefillArgs *a) {
    const int blocks = (a->G + kPreTile - 1) / kPreTile;
    a->g_tile = (a->G + blocks - 1) / blocks;
    a->tok_tile = kPreTile / a->g_tile;
    a->head_blocks = a->Hkv * blocks;
    a->max_items = a->Tq / (2 * a->tok_tile) + a->B;
}

// Lays the plan and the partial results out in `base` (null: only counts); returns the bytes.
size_t prefill_workspace(PrefillArgs *a, int Dv, bool parts, char *base) {
    size_t at = 0;
    auto take = [&](auto **p, size_t n) {
        *p = reinterpret_cast<std::remove_reference_t<decltype(*p)>>(base + at);
        at += host_align256(n * sizeof(**p));
    };
    take(&a->plan, 1);
    take(&a->items, size_t(a->max_items));
    take(&a->unsorted, size_t(a->max_items));
    take(&a->tile_prefix, size_t(a->B) + 1);
    take(&a->cost_prefix, size_t(a->max_items) + 1);
    take(&a->joins, size_t(a->workers));
    take(&a->cuts, size_t(a->workers) + 1);
    if (parts) {
        take(&a->o_part, size_t(2) * a->workers * 2 * kPreTile * Dv);
        take(&a->lse_part, size_t(2) * a->workers * 2 * kPreTile);
    }
    return at;
}

int prefill_workers(int dev) { return std::max(1, std::min(host_sm_count(dev), kMaxWorkers)); }

cudaError_t launch_after(const void *kern, dim3 grid, int threads, int smem, void **args, cudaStream_t stream) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = dim3(threads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    // Programmatic dependent launch: starts while the kernel before it ends, and waits for it before it reads.
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelExC(&cfg, kern, args);
}

template <int DQK, int DV, int SRC>
gqa_status launch_prefill(PrefillArgs a, long long keys, void *workspace, size_t workspace_bytes, int dev, cudaStream_t cs) {
    using C = PrefillCfg<DQK, DV, SRC>;
    const void *kern = reinterpret_cast<const void *>(gqa_prefill_kernel<DQK, DV, SRC>);
    static std::mutex mu;
    static bool raised[kMaxDevices];
    {
        std::lock_guard<std::mutex> lk(mu);
        if (!raised[dev]) {
            // The kernel's warps share its registers out anew, which goes wrong if they are not as many as counted on.
            cudaFuncAttributes at;
            if (cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, C::SMEM) != cudaSuccess ||
                cudaFuncGetAttributes(&at, kern) != cudaSuccess || at.numRegs != C::LAUNCH_REGS) {
                cudaGetLastError();
                return GQA_ERR_CUDA;
            }
            raised[dev] = true;
        }
    }
    a.workers = prefill_workers(dev);
    // Items of fewer steps than a part of one has at least are not divided, and need neither partial results nor a merge.
    a.may_split = (keys + kPreKeys - 1) / kPreKeys >= kPreMinSplit + kPreSnap;
    // Short keys and no more items than SMs: nothing to share out, each CTA finds its own item (a replayed call on one prompt of
    // 17 tokens 5.9 us, with the plan's launch 9.6; 5 rows over 1K keys 16.8 against 20.4).
    const long long numbers = (long long)a.max_items * a.head_blocks;
    a.direct = !a.may_split && numbers <= a.workers;
    // Some waits last for the items under way: the next rows of Q wait for the last scores of those before, V's cleaner for an
    // item's last steps.  What the limit allows grows with them, at some ten times a step's 1.1 to 1.4 us for three items.
    a.wait_limit_ns += (unsigned long long)((keys + kPreKeys - 1) / kPreKeys) * kPreWaitStepNs;
    CUtensorMap q_map, k_map, v_map;
    bool maps = host_rows_tensor_map(&q_map, a.q, a.Tq, a.Hq, DQK, a.q_stride, a.tok_tile, a.g_tile);
    if (SRC == kPreDense) {
        // (without keys nothing is loaded through the maps)
        const bool none = a.Tk == 0;
        maps = maps && host_rows_tensor_map(&k_map, none ? a.q : a.k, none ? 1 : a.Tk, a.Hkv, DQK, a.k_stride, kPreKeys, 1) &&
               host_rows_tensor_map(&v_map, none ? a.q : a.v, none ? 1 : a.Tk, a.Hkv, DV, a.v_stride, kPreKeys, 1);
    } else if (SRC == kPrePages) {
        const long long rows = (long long)a.num_pages * a.page_size;
        maps = maps && host_rows_tensor_map(&k_map, a.k_pool, rows, a.Hkv, DQK, (long long)a.Hkv * DQK, a.box_rows, 1) &&
               host_rows_tensor_map(&v_map, a.v_pool, rows, a.Hkv, DV, (long long)a.Hkv * DV, a.box_rows, 1);
    }
    if (!maps) return GQA_ERR_CUDA;
    const size_t need = a.direct ? 0 : prefill_workspace(&a, DV, a.may_split, nullptr);
    void *ws = workspace;
    bool owned = false;
    if (ws != nullptr) {
        if (workspace_bytes < prefill_workspace(&a, DV, true, nullptr)) return GQA_ERR_NO_MEMORY;
        if (!host_aligned(ws, 256)) return GQA_ERR_ALIGNMENT;
    } else if (need > 0) {
        if (host_pool_alloc(&ws, need, dev, cs) != cudaSuccess) {
            cudaGetLastError();
            return GQA_ERR_NO_MEMORY;
        }
        owned = true;
    }
    if (need > 0) prefill_workspace(&a, DV, a.may_split, static_cast<char *>(ws));
    constexpr bool paged = SRC != kPreDense;
    // As few threads as hold the sequences, items and workers (us of the plan: one request 5.2 with 256, 9.0 with 1024), all in
    // shared memory up to 2048 items (16 prompts of up to 4K tokens 17.0, with 64-bit sums through the workspace 19.5).
    const long long most_cost = a.max_items * (kPreCostItem + kPreCostTwo * ((keys + kPreKeys - 1) / kPreKeys));
    const int seqs = std::max(a.B, a.workers);
    if (a.direct) {
        // no plan
    } else if (seqs <= 256 && a.max_items <= 256 && most_cost < (1LL << 31)) {
        gqa_prefill_plan_small_kernel<paged, 256, 1><<<1, 256, 0, cs>>>(a);
    } else if (seqs <= 512 && a.max_items <= 2048 && most_cost < (1LL << 31)) {
        gqa_prefill_plan_small_kernel<paged, 512, 4><<<1, 512, 0, cs>>>(a);
    } else {
        gqa_prefill_plan_kernel<paged><<<1, kPlanThreads, 0, cs>>>(a);
    }
    cudaError_t e = cudaGetLastError();
    if (e == cudaSuccess) {
        cudaEvent_t before, after;
        host_kernel_events(&before, &after);
        const bool timed = before != nullptr && after != nullptr;
        if (timed) cudaEventRecord(before, cs);
        void *args[] = {&q_map, &k_map, &v_map, &a};
        e = launch_after(kern, dim3(unsigned(a.direct ? numbers : a.workers)), C::THREADS, C::SMEM, args, cs);
        if (timed) cudaEventRecord(after, cs);
    }
    if (e == cudaSuccess && a.may_split && a.workers > 1) {
        void *args[] = {&a};
        e = launch_after(reinterpret_cast<const void *>(gqa_prefill_merge_kernel<DV>),
                         dim3(unsigned(a.workers - 1), 2 * kPreTile / kPreMergeRows), kPreMergeThreads, 0, args, cs);
    }
    if (owned) cudaFreeAsync(ws, cs);
    if (e != cudaSuccess) {
        cudaGetLastError();
        return GQA_ERR_CUDA;
    }
    return GQA_OK;
}

// What both entry points check alike.
gqa_status check_prefill(int Tq, int B, int Hq, int Hkv, int Dqk, int Dv) {
    if (Tq < 0 || B < 1 || Hkv < 1 || Hq < 1 || Hq % Hkv != 0) return GQA_ERR_INVALID_ARG;
    if (!((Dqk == 64 && Dv == 64) || (Dqk == 128 && Dv == 128) || (Dqk == 192 && Dv == 128))) return GQA_ERR_UNSUPPORTED;
    if (B > 65535 || Hq / Hkv > 4096 || (long long)Tq * Hq >= (1LL << 31)) return GQA_ERR_UNSUPPORTED;
    PrefillArgs a = {};
    a.Tq = Tq, a.B = B, a.Hkv = Hkv, a.G = Hq / Hkv;
    prefill_tiles(&a);
    if ((long long)a.max_items * a.head_blocks >= (1LL << 31) - kMaxWorkers) return GQA_ERR_UNSUPPORTED;  // pieces count in 32 bits
    return GQA_OK;
}

}  // namespace
}  // namespace gqa

using namespace gqa;

extern "C" size_t gqa_prefill_workspace_bytes(int Tq, int B, int Hq, int Hkv, int Dqk, int Dv) {
    int dev = 0;
    if (check_prefill(Tq, B, Hq, Hkv, Dqk, Dv) != GQA_OK || !host_current_device(&dev)) return 0;
    PrefillArgs a = {};
    a.Tq = Tq, a.B = B, a.Hkv = Hkv, a.G = Hq / Hkv;
    prefill_tiles(&a);
    a.workers = prefill_workers(dev);
    return prefill_workspace(&a, Dv, true, nullptr);
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
    if (Tk > (1LL << 31) - 256) return GQA_ERR_UNSUPPORTED;  // key indexes step past the end
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
    prefill_tiles(&a);
    if (Dqk == 64) return launch_prefill<64, 64, kPreDense>(a, Tk, workspace, workspace_bytes, dev, cs);
    if (Dqk == 128) return launch_prefill<128, 128, kPreDense>(a, Tk, workspace, workspace_bytes, dev, cs);
    return launch_prefill<192, 128, kPreDense>(a, Tk, workspace, workspace_bytes, dev, cs);
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
    int lg = 0;
    while ((1LL << lg) < page_size) ++lg;
    a.page_mul = unsigned((1ull << (31 + lg)) / unsigned(page_size) + 1);
    a.page_shift = 31 + lg;
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
    prefill_tiles(&a);
    const long long keys = (long long)pages_per_req * page_size;
    a.box_rows = kPreKeys;
    while (page_size % a.box_rows != 0) a.box_rows /= 2;
#define GQA_PREFILL_SOURCE(SRC)                                                                     \
    (D == 64 ? launch_prefill<64, 64, SRC>(a, keys, workspace, workspace_bytes, dev, cs)            \
             : launch_prefill<128, 128, SRC>(a, keys, workspace, workspace_bytes, dev, cs))
    switch (kv_dtype) {
        case GQA_KV_BF16: return a.box_rows >= 8 ? GQA_PREFILL_SOURCE(kPrePages) : GQA_PREFILL_SOURCE(kPreCopy);
        case GQA_KV_FP8_E4M3FN: return GQA_PREFILL_SOURCE(kPreFp8);
        case GQA_KV_INT8: return GQA_PREFILL_SOURCE(kPreInt8);
        default: return GQA_PREFILL_SOURCE(kPreInt4);
    }
#undef GQA_PREFILL_SOURCE
}
