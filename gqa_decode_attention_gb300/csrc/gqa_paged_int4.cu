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

// What a shape runs as.
struct Int4Plan {
    int B, Sq, Hq, Hkv, D, G, Mq;
    int NT;      // tiles of 8 query rows a consumer warp holds
    int RG, HB;  // consumer warps per head, heads per CTA
    int R;       // tokens of a TMA box: the largest power of two, at most 16, that divides the page size
    int pitch, par_pitch, stage_bytes, stages, smem, threads, nhb;
    bool param_tma;
    long long max_steps;
};

gqa_status plan_int4(int B, int Sq, int Hq, int Hkv, int D, int page_size, int pages_per_req, int num_pages, Int4Plan *p) {
    gqa_status st = host_check_pages(B, Hkv, D, page_size, pages_per_req, num_pages);
    if (st != GQA_OK) return st;
    if (Sq < 1 || Hq < 1 || Hq % Hkv != 0) return GQA_ERR_INVALID_ARG;
    if ((long long)(Hq / Hkv) * Sq > kInt4MaxRows) return GQA_ERR_UNSUPPORTED;
    if ((long long)pages_per_req * page_size > (1LL << 31) - 64) return GQA_ERR_UNSUPPORTED;  // token indexes step past the end
    p->B = B, p->Sq = Sq, p->Hq = Hq, p->Hkv = Hkv, p->D = D;
    p->G = Hq / Hkv;
    p->Mq = p->G * Sq;
    p->NT = p->Mq > 8 ? 2 : 1;
    p->RG = (p->Mq + 8 * p->NT - 1) / (8 * p->NT);
    const int cap = p->NT == 1 ? kInt4MaxWarps : 4;
    int hb = 1;
    while (hb < Hkv && 2 * hb * p->RG <= cap) hb *= 2;
    p->HB = hb;
    p->nhb = (Hkv + hb - 1) / hb;
    p->R = 16;
    while (page_size % p->R != 0) p->R /= 2;
    const int row = D / 2;
    p->pitch = (hb * p->R * row + 127) / 128 * 128;  // TMA writes to 128-byte boundaries
    p->par_pitch = (hb * p->R * 8 + 127) / 128 * 128;
    p->param_tma = Hkv % 2 == 0 && hb > 1;           // a box's rows, and their stride, in whole 16 bytes
    const int align = D == 128 ? 512 : 128;          // the swizzle repeats every 512 bytes
    p->stage_bytes = ((kInt4Step / p->R) * (2 * p->pitch + p->par_pitch) + align - 1) / align * align;
    // shared memory of an SM over the CTAs that registers allow (16 warps of 8
    // rows, 12 of 16), less what the system keeps
    const int warps = hb * p->RG, ctas = p->NT == 1 ? 16 / warps : warps <= 4 ? 12 / warps : 1;
    p->stages = (228 * 1024 / ctas - 1024 - kInt4HeadBytes) / p->stage_bytes;
    if (p->stages > kInt4MaxStages) p->stages = kInt4MaxStages;
    if (p->stages < 2) p->stages = 2;
    p->smem = p->stages * p->stage_bytes + kInt4HeadBytes;
    p->threads = 32 * (hb * p->RG + 1);
    p->max_steps = (long long)B * (((long long)pages_per_req * page_size + kInt4Step - 1) / kInt4Step);
    if (p->max_steps >= (1LL << 31)) return GQA_ERR_UNSUPPORTED;  // the schedule counts steps in 32 bits
    return GQA_OK;
}

// Instances: 8 query rows a warp and up to 8 warps; 16 rows a warp and up to 4
// warps (three CTAs an SM); 16 rows and 5 to 8 warps (65 to 128 rows a head).
int instance_of(const Int4Plan &p) { return p.NT == 1 ? 0 : p.HB * p.RG <= 4 ? 1 : 2; }

const void *kernel_of(const Int4Plan &p) {
    static const void *const kernels[2][3] = {
        {reinterpret_cast<const void *>(gqa_paged_int4_kernel<64, 1, 8>), reinterpret_cast<const void *>(gqa_paged_int4_kernel<64, 2, 4>),
         reinterpret_cast<const void *>(gqa_paged_int4_kernel<64, 2, 8>)},
        {reinterpret_cast<const void *>(gqa_paged_int4_kernel<128, 1, 8>), reinterpret_cast<const void *>(gqa_paged_int4_kernel<128, 2, 4>),
         reinterpret_cast<const void *>(gqa_paged_int4_kernel<128, 2, 8>)}};
    return kernels[p.D == 128][instance_of(p)];
}

// Resident CTAs per SM of the plan's instance on `dev`, the current device;
// the first query of an instance also raises its shared-memory limit there.
int int4_occupancy(int dev, const Int4Plan &p) {
    struct Entry {
        int smem, threads, ctas;
    };
    static std::mutex mu;
    static Entry table[kMaxDevices][2][3][64];
    static int used[kMaxDevices][2][3];
    static bool raised[kMaxDevices][2][3];
    std::lock_guard<std::mutex> lk(mu);
    const int d = p.D == 128, n = instance_of(p);
    Entry *t = table[dev][d][n];
    for (int i = 0; i < used[dev][d][n]; ++i)
        if (t[i].smem == p.smem && t[i].threads == p.threads) return t[i].ctas;
    const void *kern = kernel_of(p);
    if (!raised[dev][d][n]) {
        int most = 0;
        if (cudaDeviceGetAttribute(&most, cudaDevAttrMaxSharedMemoryPerBlockOptin, dev) != cudaSuccess ||
            cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, most) != cudaSuccess)
            return 0;
        raised[dev][d][n] = true;
    }
    int ctas = 0;
    if (cudaOccupancyMaxActiveBlocksPerMultiprocessor(&ctas, kern, p.threads, p.smem) != cudaSuccess) return 0;
    if (used[dev][d][n] < 64) t[used[dev][d][n]++] = {p.smem, p.threads, ctas};
    return ctas;
}

// Workers per head block: one resident CTA slot each, and no more than the
// requests can have steps.
int int4_workers(const Int4Plan &p, int requested, int dev) {
    long long W = requested;
    if (requested == 0) {
        const long long occ = int4_occupancy(dev, p);
        W = host_sm_count(dev) * (occ > 0 ? occ : 1) / p.nhb;
        if (W > p.max_steps) W = p.max_steps;
    }
    if (W > 65535) W = 65535;
    return W < 1 ? 1 : int(W);
}

size_t int4_workspace(const Int4Plan &p, int workers) {
    if (workers <= 1) return 0;
    const size_t rows = size_t(p.nhb) * workers * 2 * p.HB * p.Mq;
    return host_align256(rows * p.D * sizeof(float)) + host_align256(rows * sizeof(float)) +
           host_align256((size_t(p.B) + 1) * sizeof(int));
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
    CUtensorMap k_map, v_map, p_map = {};
    const long long rows = (long long)num_pages * page_size;
    if (int4_occupancy(dev, p) < 1 || !host_int4_tensor_map(&k_map, k_pool, rows, Hkv, D / 2, p.R, p.HB) ||
        !host_int4_tensor_map(&v_map, v_pool, rows, Hkv, D / 2, p.R, p.HB) ||
        (p.param_tma && !host_int4_param_map(&p_map, kv_params, rows, Hkv, p.R, p.HB))) {
        cudaGetLastError();
        return GQA_ERR_CUDA;
    }
    const int workers = int4_workers(p, num_splits, dev);
    cudaStream_t cs = reinterpret_cast<cudaStream_t>(stream);
    const size_t need = int4_workspace(p, workers);
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
        const size_t part_rows = size_t(p.nhb) * workers * 2 * p.HB * p.Mq;
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
    a.page_size = page_size;
    a.pages_per_req = pages_per_req;
    a.num_pages = num_pages;
    a.workers = workers;
    a.HB = p.HB;
    a.RG = p.RG;
    a.stages = p.stages;
    a.box_rows = p.R;
    a.box_pitch = p.pitch;
    a.stage_bytes = p.stage_bytes;
    a.tok8 = p.R == 16 ? 8 * (D / 2) : (8 / p.R) * p.pitch;
    a.tok16 = p.R == 16 ? p.pitch : (16 / p.R) * p.pitch;
    a.param_tma = p.param_tma;
    a.param_pitch = p.par_pitch;
    a.par8 = p.R == 16 ? 8 * p.HB * 8 : (8 / p.R) * p.par_pitch;
    a.par16 = p.R == 16 ? p.par_pitch : (16 / p.R) * p.par_pitch;
    a.alpha = host_resolve_scale(scale, D) * 1.4426950408889634f;
    a.wait_limit_ns = host_wait_limit_ns();
    a.fault_mode = host_fault_mode();
    a.err = host_error_word(dev);
    cudaEvent_t before, after;
    host_kernel_events(&before, &after);
    const bool timed = before != nullptr && after != nullptr;
    if (timed) cudaEventRecord(before, cs);
    void *args[] = {&k_map, &v_map, &p_map, &a};
    cudaError_t e = launch(kernel_of(p), dim3(unsigned(p.nhb), unsigned(workers)), p.threads, p.smem, args, cs);
    if (timed) cudaEventRecord(after, cs);
    if (e == cudaSuccess && workers > 1) {
        void *margs[] = {&a};
        const void *merge = D == 64 ? reinterpret_cast<const void *>(gqa_paged_int4_merge_kernel<64>)
                                    : reinterpret_cast<const void *>(gqa_paged_int4_merge_kernel<128>);
        e = launch(merge, dim3(unsigned(Hkv * p.Mq), unsigned(B)), 32 * kInt4MergeWarps, 0, margs, cs);
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
    return int4_workers(p, 0, dev);
}

extern "C" size_t gqa_decode_paged_int4_workspace_bytes(int B, int Sq, int Hq, int Hkv, int D, int page_size,
                                                        int pages_per_req, int num_splits) {
    Int4Plan p;
    if (plan_int4(B, Sq, Hq, Hkv, D, page_size, pages_per_req, 1, &p) != GQA_OK || num_splits < 0) return 0;
    int dev = 0;
    if (num_splits == 0 && !host_current_device(&dev)) return 0;
    return int4_workspace(p, int4_workers(p, num_splits, dev));
}
