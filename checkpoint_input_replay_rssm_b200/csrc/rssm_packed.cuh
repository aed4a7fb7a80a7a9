// rssm_packed.cuh -- helpers shared by the operators on packed requests
// (block tables, the 4-bit key/value cache, the packed delta-rule prefill).
#pragma once

#include "rssm_device.cuh"

namespace rssm {

enum PackedErr : int { DEV_BAD_LENGTHS = 4, DEV_NO_PAGES = 5, DEV_BAD_PAGE = 6 };

// Out of line: it is off every kernel's path, and its code would lie between what is on it.
static __device__ __noinline__ void report_opt(int32_t *err, int code, int b, int h, int value) {
    if (err) report(err, code, b, h, value);
}

// Rows [r0, r1) of request b, false when the offsets are out of order or past `rows`.
__device__ __forceinline__ bool packed_rows(const int32_t *cu, int b, int rows, int &r0, int &r1) {
    r0 = cu[b];
    r1 = cu[b + 1];
    return r0 >= 0 && r0 <= r1 && r1 <= rows;
}

// 16-byte global -> shared copy, or 16 zeros (src is then not read).
__device__ __forceinline__ void cp_async16_or_zero(void *dst, const void *src, bool live) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"((uint32_t)__cvta_generic_to_shared(dst)), "l"(src),
                 "r"(live ? 16 : 0)
                 : "memory");
}

static inline bool aligned16(const void *p) { return ((uintptr_t)p & 15) == 0; }

}  // namespace rssm
