// rssm_kv4_attend.cuh -- what the two kernels of the attention over the 4-bit cache share.
#pragma once

#include <cuda_bf16.h>

#include "rssm_kv4.cuh"

namespace rssm {

struct AttendArgs {
    Kv4Args kv;
    int B, Hq, G, tokens, max_pages, max_q, max_seq;
    int tiles, splits, L;  // row tiles a request, splits, cached tokens a split
    int few;               // where both kernels run: requests of up to this many rows are the split one's (0: one kernel has all)
    int packed;            // the 128-row tiles of all requests are numbered through (at most so many), 0: a grid row a request
    float scale;           // sm_scale * k_scale * log2(e)
    const __nv_bfloat16 *q;
    const uint8_t *cache;
    const int32_t *table, *seq_len, *cu;
    __nv_bfloat16 *out;
    float *part;  // [B][Hk][tiles][splits][rows][D], then (m, l) [...][rows][2]
    int32_t *err;
};


constexpr float kLag = 6.f;  // log2 by which the running maximum may trail

// The rows and length of request b; false (and reported) where they do not fit the call.
__device__ __forceinline__ bool attend_request(const AttendArgs &a, int b, int &r0, int &n, int &len) {
    int r1;
    const bool ok = packed_rows(a.cu, b, a.tokens, r0, r1);
    n = r1 - r0;
    len = a.seq_len[b];
    return ok && n <= a.max_q && len >= 0 && len <= a.max_seq && len <= (int64_t)a.max_pages * a.kv.ps;
}

// Whether this kernel of the two is to serve a request of so many rows.
__device__ __forceinline__ bool attend_mine(const AttendArgs &a, int rows, bool tiles) { return a.few == 0 || (rows > a.few) == tiles; }

__device__ __forceinline__ uint32_t f16x2(float lo, float hi) {
    uint32_t r;
    asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
}
__device__ __forceinline__ uint32_t mul2(uint32_t a, uint32_t b) {
    uint32_t r;
    asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    return r;
}
// The four bytes of w, two e2m1 codes each, as fp16 pairs.
__device__ __forceinline__ void widen(uint32_t w, uint32_t (&h)[4]) {
    asm("{\n .reg .b8 a, b, c, d;\n mov.b32 {a, b, c, d}, %4;\n cvt.rn.f16x2.e2m1x2 %0, a;\n"
        " cvt.rn.f16x2.e2m1x2 %1, b;\n cvt.rn.f16x2.e2m1x2 %2, c;\n cvt.rn.f16x2.e2m1x2 %3, d;\n}\n"
        : "=r"(h[0]), "=r"(h[1]), "=r"(h[2]), "=r"(h[3])
        : "r"(w));
}
// Two e4m3 bytes (low 16 bits of w) as an fp16 pair.
__device__ __forceinline__ uint32_t scales2(uint32_t w) {
    uint32_t r;
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(r) : "h"((uint16_t)w));
    return r;
}
// A row's power-of-two scale: the largest magnitude goes to [2^9, 2^10).
__device__ __forceinline__ int row_exponent(float top) {
    const int e = (int)(__float_as_uint(top) >> 23);  // top >= 0
    return e == 0 || e == 255 ? 0 : e - 126 - 10;
}

// 2^e for e in -126 .. 127.
__device__ __forceinline__ float pow2f(int e) { return __uint_as_float((uint32_t)(e + 127) << 23); }

// The factor of a row's raw scores: `scale` and the row's power of two, above 0 so that the largest raw score is the largest
// score and a masked one stays -inf (the sign of `scale` goes to the query, a zero scale becomes a zero query).  A query with an
// infinity makes every visible score NaN, as inf - inf in the softmax does: left as -inf they would be as if masked.
__device__ __forceinline__ float row_factor(float scale, int ex, float top, bool sees) {
    if (top == INFINITY && sees) return NAN;
    return fmaxf(fabsf(scale) * pow2f(ex / 2) * pow2f(ex - ex / 2), 1.2e-38f);
}

// The kernel for tiles of 128 rows (rssm_kv4_attend_tiles.cu).
cudaError_t attend_tiles_launch(const AttendArgs &a, cudaStream_t st);

}  // namespace rssm
