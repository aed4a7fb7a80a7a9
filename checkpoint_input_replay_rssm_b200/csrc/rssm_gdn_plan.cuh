// rssm_gdn_plan.cuh -- where the chunks of packed prompts keep their operands: first[b] = chunks of the requests before b.
//
// The offsets come from the caller and may be wrong.  A request whose own offsets do not fit has no chunks, whatever
// they hold, so that first[] ascends and every other request's slots are its own.
#pragma once

#include "rssm_gdn_prefill.h"
#include "rssm_packed.cuh"

namespace rssm {

constexpr int kGdnChunk = 64;

// Chunks of request b's rows [r0, r1).
__device__ __forceinline__ int gdn_chunks(const GdnPreArgs &a, int b, int &r0, int &r1) {
    return packed_rows(a.cu, b, a.tokens, r0, r1) ? (int)(((int64_t)r1 - r0 + kGdnChunk - 1) / kGdnChunk) : 0;
}

// By one CTA of THR threads: each sums a run of requests, and writes the run again with what lies before it.  A few
// bytes a request, two dependent reads: a call of 8 short prompts takes 1.5 us more than with slots that need no sum
// (32.7 -> 34.3), one of 64 ragged prompts the same.
template <int THR> __device__ void gdn_plan(const GdnPreArgs &a) {
    __shared__ long long wsum[THR / 32];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int per = (a.B + THR - 1) / THR, b0 = min(a.B, tid * per), b1 = min(a.B, b0 + per);
    int r0, r1;
    long long mine = 0;
    for (int b = b0; b < b1; ++b) mine += gdn_chunks(a, b, r0, r1);
    long long x = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const long long u = __shfl_up_sync(0xffffffffu, x, o);
        if (lane >= o) x += u;
    }
    if (lane == 31) wsum[warp] = x;
    __syncthreads();
    x -= mine;
    for (int w = 0; w < warp; ++w) x += wsum[w];
    for (int b = b0; b < b1; ++b) {
        a.first[b] = (int)min(x, 0x7fffffffLL);
        x += gdn_chunks(a, b, r0, r1);
    }
}

}  // namespace rssm
