// gqa_paged_int4.cu -- paged decode over whole requests from a 4-bit cache:
// host side of gqa_paged_int4.cuh and its C entry points.
#include "gqa_paged_int4.cuh"

#include <cmath>
#include <mutex>

#include "gqa_host.h"

namespace gqa {
namespace {

constexpr int kInt4MaxRows = 128;  // query rows per KV head
constexpr int kMaxDevices = 64;

constexpr int kInt4MaxLanes = 8;
constexpr int kInt4MaxShortRows = 32;  // of a KV head, with 8 rows a warp in short requests

// What a shape runs as, before the number of workers is known.
struct Int4Plan {
    int B, Sq, Hq, Hkv, D, G, Mq, page_size;
    int NT;      // tiles of 8 query rows a consumer warp holds
    int RG, HB;  // consumer warps per head, heads per CTA
    int rings, lanes;  // most rings of a CTA; groups of HB x RG warps on each
    int R;       // tokens of a TMA box: the largest power of two, at most a step, that divides the page size
    bool row_copies;  // no TMA for K and V: below R = 4 the boxes are too many (96 a step with pages of 5: 2.7 us)
    int pitch, par_pitch, stage_bytes, nhb;
    bool param_tma;
    int param_rows;  // of a box of the parameters' map if its rows are 32 bytes, 0 if tokens
    int param_heads;
    long long max_steps;
    int change;  // places that a change of request takes in the schedule
};

// The plan's layout with NT tiles of 8 query rows a warp.
void int4_layout(Int4Plan *p, int nt) {
    const int Hkv = p->Hkv, page_size = p->page_size;
    p->NT = nt;
    // Measured (us a call): 256 requests of up to 1K tokens, 8 rows a warp, 47.6 with 1, 46.5 with 2, 48.6 with 4; 16
    // requests of up to 8K tokens, 16 rows a warp, 41.9 with 1, 35.3 with 4, 33.9 with 6, 34.6 with 12.
    p->change = nt == 1 ? 2 : 6;
    p->RG = (p->Mq + 8 * nt - 1) / (8 * nt);
    int hb = 1;
    while (hb < Hkv && 2 * hb * p->RG <= 8) hb *= 2;
    p->HB = hb;
    p->nhb = (Hkv + hb - 1) / hb;
    const int groups = int4_consumers(p->NT) / (hb * p->RG);
    p->rings = groups < kInt4MaxRings ? groups : kInt4MaxRings;
    while (groups % p->rings != 0) --p->rings;
    p->lanes = groups / p->rings;
    // A warp takes 110 to 130 cycles to start a box, which bounds large caches of one small head (126 requests, 79838
    // steps of one head of 64: 112 us with boxes of 16 and parameters by cp.async, 108 with parameters by TMA, 91 with 32).
    p->R = kInt4Step;
    while (page_size % p->R != 0) p->R /= 2;
    p->row_copies = p->R < 4;
    if (p->row_copies) p->R = 16;  // the places of whole boxes
    const int row = p->D / 2;
    p->pitch = (hb * p->R * row + 127) / 128 * 128;  // TMA writes to 128-byte boundaries
    // Parameters by TMA where a token's are whole 16 bytes, or where a CTA has all heads, so that a box's are one
    // piece, seen as rows of 32 bytes (R * Hkv * 8 bytes, R a multiple of 4).
    const bool even = Hkv % 2 == 0 && hb > 1;
    p->param_tma = !p->row_copies && (even || p->nhb == 1);
    p->param_rows = p->param_tma && !even ? p->R * Hkv / 4 : 0;
    p->param_heads = p->param_rows > 0 ? Hkv : hb;
    p->par_pitch = p->param_tma ? (p->param_heads * p->R * 8 + 127) / 128 * 128 : hb * p->R * 8;
    // 512: the period of the swizzle
    p->stage_bytes = ((kInt4Step / p->R) * (2 * p->pitch + p->par_pitch) + 511) / 512 * 512;
}

gqa_status plan_int4(int B, int Sq, int Hq, int Hkv, int D, int page_size, int pages_per_req, int num_pages, Int4Plan *p) {
    gqa_status st = host_check_pages(B, Hkv, D, page_size, pages_per_req, num_pages);
    if (st != GQA_OK) return st;
    if (Sq < 1 || Hq < 1 || Hq % Hkv != 0) return GQA_ERR_INVALID_ARG;
    if ((long long)(Hq / Hkv) * Sq > kInt4MaxRows) return GQA_ERR_UNSUPPORTED;
    if ((long long)pages_per_req * page_size > (1LL << 31) - 256) return GQA_ERR_UNSUPPORTED;  // token indexes step past the end
    p->B = B, p->Sq = Sq, p->Hq = Hq, p->Hkv = Hkv, p->D = D, p->page_size = page_size;
    p->G = Hq / Hkv;
    p->Mq = p->G * Sq;
    p->max_steps = (long long)B * (((long long)pages_per_req * page_size + kInt4Step - 1) / kInt4Step);
    int4_layout(p, p->Mq > 8 ? 2 : 1);
    if (p->max_steps + (long long)B * p->change >= (1LL << 31)) return GQA_ERR_UNSUPPORTED;  // the schedule counts steps in 32 bits
    return GQA_OK;
}

template <int D, int NT>
const void *kernel_for(bool copies) {
    return copies ? reinterpret_cast<const void *>(gqa_paged_int4_kernel<D, NT, true>)
                  : reinterpret_cast<const void *>(gqa_paged_int4_kernel<D, NT, false>);
}
const void *kernel_of(const Int4Plan &p) {
    if (p.D == 64) return p.NT == 1 ? kernel_for<64, 1>(p.row_copies) : kernel_for<64, 2>(p.row_copies);
    return p.NT == 1 ? kernel_for<128, 1>(p.row_copies) : kernel_for<128, 2>(p.row_copies);
}

// Shared memory a CTA may have on `dev`, the current device; the first call
// there raises the kernel's limit to it.  0 on an error.
int int4_smem(int dev, const Int4Plan &p) {
    static std::mutex mu;
    static int most[kMaxDevices][2][2][2];
    std::lock_guard<std::mutex> lk(mu);
    int &m = most[dev][p.D == 128][p.NT - 1][p.row_copies];
    if (m == 0) {
        int n = 0;
        if (cudaDeviceGetAttribute(&n, cudaDevAttrMaxSharedMemoryPerBlockOptin, dev) != cudaSuccess ||
            cudaFuncSetAttribute(kernel_of(p), cudaFuncAttributeMaxDynamicSharedMemorySize, n) != cudaSuccess)
            return 0;
        m = n;
    }
    return m;
}

// CTAs of one wave per head block (a CTA's registers fill an SM).
int int4_ctas(const Int4Plan &p, int dev) {
    const int n = host_sm_count(dev) / p.nhb;
    return n < 1 ? 1 : n;
}

// How the requests' steps are shared out.
struct Int4Split {
    int workers;  // per head block
    bool whole;   // a worker takes whole requests: one launch, no workspace
    int rings, lanes;  // as in the plan; whole requests may take other ones
};

// The automatic choice (requested = 0).  Equal shares of all steps, for every
// ring of one wave and no more than the requests can have steps, keep every SM
// busy whatever the lengths are, but cost a second launch for the merge and the
// workspace.  Short requests are better off whole: one launch, no workspace, all
// warps of a CTA on one request's steps in turns (measured, us a call without /
// with the host's part, shares against whole: one request of 512 tokens, 8 heads
// over 2 of 64, 9.8 / 34 against 8.9 / 30; 40 of 256 tokens, 32 heads over 8 of
// 128, 15.3 / 39 against 13.9 / 35, of 512 17.1 / 39.7 against 20.6 / 40.9).  The
// estimates below are fitted to such measurements; a request's length is known
// only as the page table's width, taken as filled to 0.7 on average where the
// lengths even out; past 40 us uneven lengths cost more than a merge (64 requests
// of up to 6K tokens, 32 rows a head of 64: 196 against 103 us).  A requested
// number is a number of shares, unless it is that of the automatic choice: the
// same number gives the same bits.
Int4Split int4_auto(const Int4Plan &p, int dev, double *us) {
    const long long ctas = int4_ctas(p, dev);
    long long W = ctas * p.rings;
    if (W > p.max_steps) W = p.max_steps;
    if (W > 65535) W = 65535;
    if (W < 1) W = 1;
    const int groups = int4_consumers(p.NT) / (p.HB * p.RG);
    const long long steps = p.max_steps / p.B;  // of a request, at most
    // whole requests: as many rings as requests come to a CTA, the other groups in turns on each
    const long long each = (p.B + ctas - 1) / ctas;
    int rings = 1, lanes = 1;
    while (rings < each && 2 * rings <= groups && rings < kInt4MaxRings) rings *= 2;
    while (lanes < steps && 2 * lanes * rings <= groups && lanes < kInt4MaxLanes) lanes *= 2;
    double turns = double((steps + lanes - 1) / lanes) * (p.D == 64 ? 1.3 : 1.7);
    if (p.row_copies && turns < 0.7 * steps) turns = 0.7 * steps;  // what its producers take
    const double whole = (p.NT == 1 ? 5 : 8) + double((each + rings - 1) / rings) * (turns + 0.2 * (lanes - 1) + 1);
    const double shares = 11.5 + 0.7 * 2.3 / groups * double(p.max_steps + (long long)p.B * p.change) / double(ctas);
    *us = whole < shares ? whole : shares;
    if ((whole < shares && whole < 40) || W == 1) return {int(p.B < ctas * rings ? p.B : ctas * rings), true, rings, lanes};
    return {int(W), false, p.rings, p.lanes};
}

// More than 8 rows a head: 16 of them a warp turn a step's codes into operands
// once for all, 8 of them start and end a request sooner.  Long walks are 8 to
// 10 % faster with 16, short whole requests 6 to 21 % with 8 (22 requests of 11
// tokens, 15 rows a head of 128, 6.7 against 5.3 us).  Shares of up to three steps
// an SM, measured both ways on 112 shapes: most are 3 to 14 % faster with 8 (one
// request of 1K tokens, 16 rows for each of 8 heads of 128, 14.2 against 12.3 us);
// up to 3 % slower are 16 rows for each of 4 heads of 128, four requests of 2K
// tokens and 8 heads, and one request with 24 rows on one head (at 8K tokens, d 64,
// 7 %: 11.7 against 12.5).
Int4Split int4_split(Int4Plan *p, int requested, int dev) {
    Int4Plan best = *p;
    double us;
    Int4Split s = int4_auto(best, dev, &us);
    if (p->NT == 2 && p->Mq <= kInt4MaxShortRows) {
        Int4Plan p1 = *p;
        int4_layout(&p1, 1);
        double us1;
        const Int4Split s1 = int4_auto(p1, dev, &us1);
        if (s1.whole ? us1 < us : !s.whole && p->max_steps < 3LL * int4_ctas(*p, dev)) best = p1, s = s1;
    }
    if (requested == 0 || requested == s.workers) {
        *p = best;
        return s;
    }
    return {requested < 65535 ? requested : 65535, false, p->rings, p->lanes};
}

size_t int4_part_rows(const Int4Plan &p, const Int4Split &s) {
    return s.whole || s.workers <= 1 ? 0 : size_t(p.nhb) * s.workers * 2 * p.HB * p.Mq;
}

size_t int4_workspace(const Int4Plan &p, const Int4Split &s) {
    const size_t rows = int4_part_rows(p, s);
    if (rows == 0) return 0;
    return host_align256(rows * p.D * sizeof(float)) + host_align256(rows * sizeof(float)) +
           host_align256((size_t(p.B) + 2) * sizeof(int));
}

cudaError_t launch(const void *kern, dim3 grid, int threads, int smem, void **args, cudaStream_t stream) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = dim3(threads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    // Programmatic dependent launch: the CTAs may be scheduled while the
    // previous kernel drains; they wait for it before reading.
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelExC(&cfg, kern, args);
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
    Int4Plan p;
    gqa_status st = plan_int4(B, Sq, Hq, Hkv, D, page_size, pages_per_req, num_pages, &p);
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
    const Int4Split split = int4_split(&p, num_splits, dev);
    const int workers = split.workers;
    CUtensorMap k_map = {}, v_map = {}, p_map = {};
    const long long rows = (long long)num_pages * page_size;
    const int smem = int4_smem(dev, p);
    if (smem == 0 ||
        (!p.row_copies && (!host_int4_tensor_map(&k_map, k_pool, rows, Hkv, D / 2, p.R, p.HB) ||
                           !host_int4_tensor_map(&v_map, v_pool, rows, Hkv, D / 2, p.R, p.HB))) ||
        (p.param_tma && !(p.param_rows > 0 ? host_int4_param_map(&p_map, kv_params, rows / 4 * Hkv, 4, p.param_rows, 4)
                                         : host_int4_param_map(&p_map, kv_params, rows, Hkv, p.R, p.HB)))) {
        cudaGetLastError();
        return GQA_ERR_CUDA;
    }
    cudaStream_t cs = reinterpret_cast<cudaStream_t>(stream);
    const size_t need = int4_workspace(p, split);
    void *ws = workspace;
    bool owned = false;
    if (need > 0) {
        if (ws != nullptr) {
            if (workspace_bytes < need) return GQA_ERR_NO_MEMORY;
            if (!host_aligned(ws, 256)) return GQA_ERR_ALIGNMENT;
        } else {
            if (host_pool_alloc(&ws, need, dev, cs) != cudaSuccess) {
                cudaGetLastError();
                return GQA_ERR_NO_MEMORY;
            }
            owned = true;
        }
    }
    Int4Args a = {};
    a.q = static_cast<const __nv_bfloat16 *>(q);
    a.params = static_cast<const __half *>(kv_params);
    a.page_table = page_table;
    a.seq_lens = seq_lens;
    a.out = static_cast<__nv_bfloat16 *>(out);
    a.lse = lse;
    if (need > 0) {
        const size_t part_rows = int4_part_rows(p, split);
        char *w = static_cast<char *>(ws);
        a.o_part = reinterpret_cast<float *>(w);
        w += host_align256(part_rows * D * sizeof(float));
        a.lse_part = reinterpret_cast<float *>(w);
        a.step_prefix = reinterpret_cast<int *>(w + host_align256(part_rows * sizeof(float)));
    }
    a.B = B;
    a.Sq = Sq;
    a.Hq = Hq;
    a.Hkv = Hkv;
    a.G = p.G;
    a.Mq = p.Mq;
    a.g_inv = (65536u + p.G - 1) / p.G;
    a.page_size = page_size;
    a.pages_per_req = pages_per_req;
    a.num_pages = num_pages;
    a.workers = workers;
    a.change = p.change;
    a.whole = split.whole;
    a.next_b = split.whole ? workers : 1;
    int lg = 0;
    while ((1LL << lg) < page_size) ++lg;
    a.by_page.m = (1ull << (31 + lg)) / unsigned(page_size) + 1;
    a.by_page.shift = 31 + lg;
    a.HB = p.HB;
    a.RG = p.RG;
    // One ring a CTA while the workers are fewer than the SMs; the rings share
    // the CTA's memory.
    const int ctas = int4_ctas(p, dev);
    a.rings = workers >= ctas * split.rings ? split.rings : (workers + ctas - 1) / ctas;
    a.rings_max = split.rings;
    a.lanes = split.lanes;
    const int boxes = (a.lanes - 1) * p.HB * p.RG * p.NT * (D / 4 + 6) * 128;  // what the lanes of a ring hand over
    a.stages = ((smem - kInt4HeadBytes) / a.rings - boxes) / p.stage_bytes;
    if (a.stages > kInt4MaxStages) a.stages = kInt4MaxStages;
    a.stages -= a.stages % a.lanes;  // a stage serves one lane only
    a.producers = kInt4MaxRings / a.rings;
    // 16-byte copies: a warp's turn is 32 pieces, 32 / (HB * D / 32) tokens, of its part of the step's 32
    while (p.row_copies && a.producers > p.HB * (D / 32)) a.producers /= 2;
    // TMA: a stage has one producer, and one keeps up with a lane, which takes longer than 0.65 us a step
    while (!p.row_copies && (a.stages % a.producers != 0 || a.producers > a.lanes)) a.producers /= 2;
    const int grid_y = (workers + a.rings - 1) / a.rings;
    a.box_rows = p.R;
    a.box_pitch = p.pitch;
    a.stage_bytes = p.stage_bytes;
    a.tok8 = p.R >= 16 ? 8 * (D / 2) : (8 / p.R) * p.pitch;
    a.tok16 = p.R == 32 ? 16 * (D / 2) : p.R == 16 ? p.pitch : (16 / p.R) * p.pitch;
    a.param_tma = p.param_tma;
    a.param_shift = p.param_rows > 0 ? 2 : 0;
    a.param_mul = p.param_rows > 0 ? Hkv : 1;
    a.param_heads = p.param_heads;
    a.k_pool = static_cast<const uint8_t *>(k_pool);
    a.v_pool = static_cast<const uint8_t *>(v_pool);
    a.param_pitch = p.par_pitch;
    a.par8 = p.R >= 16 ? 8 * p.param_heads * 8 : (8 / p.R) * p.par_pitch;
    a.par16 = p.R == 32 ? 16 * p.param_heads * 8 : p.R == 16 ? p.par_pitch : (16 / p.R) * p.par_pitch;
    a.alpha = host_resolve_scale(scale, D) * 1.4426950408889634f;
    a.wait_limit_ns = host_wait_limit_ns();
    a.fault_mode = host_fault_mode();
    a.err = host_error_word(dev);
    cudaEvent_t before, after;
    host_kernel_events(&before, &after);
    const bool timed = before != nullptr && after != nullptr;
    if (timed) cudaEventRecord(before, cs);
    void *args[] = {&k_map, &v_map, &p_map, &a};
    cudaError_t e = launch(kernel_of(p), dim3(unsigned(p.nhb), unsigned(grid_y)), int4_threads(p.NT),
                           kInt4HeadBytes + a.rings * (a.stages * p.stage_bytes + boxes), args, cs);
    if (timed) cudaEventRecord(after, cs);
    if (e == cudaSuccess && need > 0) {
        // many partials a row: all warps of a CTA on one row
        const bool wide = workers > 16LL * B;
        const int rows = Hkv * p.Mq, per = wide ? 1 : int4_merge_warps(false);
        const void *merge = wide ? (D == 64 ? reinterpret_cast<const void *>(gqa_paged_int4_merge_kernel<64, true>)
                                             : reinterpret_cast<const void *>(gqa_paged_int4_merge_kernel<128, true>))
                                  : (D == 64 ? reinterpret_cast<const void *>(gqa_paged_int4_merge_kernel<64, false>)
                                             : reinterpret_cast<const void *>(gqa_paged_int4_merge_kernel<128, false>));
        void *margs[] = {&a};
        e = launch(merge, dim3(unsigned((rows + per - 1) / per), unsigned(B)), 32 * int4_merge_warps(wide), 0, margs, cs);
    }
    if (owned) cudaFreeAsync(ws, cs);
    if (e != cudaSuccess) {
        cudaGetLastError();
        return GQA_ERR_CUDA;
    }
    return GQA_OK;
}

extern "C" int gqa_decode_paged_int4_num_splits(int B, int Sq, int Hq, int Hkv, int D, int page_size,
                                                int pages_per_req) {
    Int4Plan p;
    const gqa_status st = plan_int4(B, Sq, Hq, Hkv, D, page_size, pages_per_req, 1, &p);
    if (st != GQA_OK) return -int(st);
    int dev = 0;
    if (!host_current_device(&dev)) return -int(GQA_ERR_CUDA);
    return int4_split(&p, 0, dev).workers;
}

extern "C" size_t gqa_decode_paged_int4_workspace_bytes(int B, int Sq, int Hq, int Hkv, int D, int page_size,
                                                        int pages_per_req, int num_splits) {
    Int4Plan p;
    if (plan_int4(B, Sq, Hq, Hkv, D, page_size, pages_per_req, 1, &p) != GQA_OK || num_splits < 0) return 0;
    int dev = 0;
    if (!host_current_device(&dev)) return 0;
    const Int4Split split = int4_split(&p, num_splits, dev);
    return int4_workspace(p, split);
}
