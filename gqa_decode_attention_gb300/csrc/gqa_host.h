// gqa_host.h -- what the front end (gqa_api.cu) shares with the other
// translation units that hold C entry points.
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>
#include <stddef.h>
#include <stdint.h>

#include "../../include/gqa_decode.h"

namespace gqa {

// Current device, false when it cannot be had or is past the library's table.
bool host_current_device(int *dev);
int host_sm_count(int dev);
// Device address of the sticky error word on `dev`, the current device.
unsigned *host_error_word(int dev);
// Stream-ordered allocation from the library's own pool of `dev`.
cudaError_t host_pool_alloc(void **p, size_t bytes, int dev, cudaStream_t stream);
uint64_t host_wait_limit_ns();
int host_fault_mode();
// The measurement hook's events (null when off).
void host_kernel_events(cudaEvent_t *before, cudaEvent_t *after);
// scale, or 1 / sqrt(D) where scale is not a positive finite number.
float host_resolve_scale(float scale, int D);

// TMA descriptor of one 4-bit pool: bytes [rows, heads, row_bytes] seen as
// (byte, row, head), boxes of (row_bytes, box_rows, box_heads), the 64-byte
// swizzle for rows of 64 bytes.  Rows and heads past the end read as zeros.
bool host_int4_tensor_map(CUtensorMap *map, const void *base, long long rows, int heads, int row_bytes, int box_rows,
                          int box_heads);

// TMA descriptor of the 4-bit cache's parameters: fp16 [rows, heads, 4] seen as
// rows of heads * 4, boxes of (box_heads * 4, box_rows).
bool host_int4_param_map(CUtensorMap *map, const void *base, long long rows, int heads, int box_rows, int box_heads);

inline bool host_aligned(const void *p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }
inline size_t host_align256(size_t x) { return (x + 255) & ~size_t(255); }

// Sizes every paged entry point checks alike.
inline gqa_status host_check_pages(int B, int Hkv, int D, int page_size, int pages_per_req, int num_pages) {
    if (B < 1 || Hkv < 1 || page_size < 1 || pages_per_req < 1 || num_pages < 1) return GQA_ERR_INVALID_ARG;
    if (D != 64 && D != 128) return GQA_ERR_UNSUPPORTED;
    if ((long long)pages_per_req * page_size >= (1LL << 31) || (long long)num_pages * page_size >= (1LL << 31))
        return GQA_ERR_UNSUPPORTED;
    if (B > 65535) return GQA_ERR_UNSUPPORTED;
    return GQA_OK;
}

}  // namespace gqa
