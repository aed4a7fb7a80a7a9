// rssm_gdn_plan.cuh -- where the chunks of packed prompts keep their operands: first[b] = chunks of the requests before b.
//
// The offsets come from the caller and may be wrong.  A request whose own offsets do not fit has no chunks, whatever
// they hold, so that first[] ascends and every other request's slots are its own.
//
// Which form serves a request goes by its own length, so that its result and its time do not hang on what it is packed
// with.
#pragma once

#include "rssm_gdn_prefill.h"
#include "rssm_packed.cuh"

namespace rssm {

// Chunks of request b's rows [r0, r1): none where its offsets are bad or it is left to the recurrence.
__device__ __forceinline__ int gdn_chunks(const GdnPreArgs &a, int b, int &r0, int &r1) {
    if (!packed_rows(a.cu, b, a.tokens, r0, r1) || r1 - r0 <= kGdnShort) return 0;
    return (int)(((int64_t)r1 - r0 + kGdnChunk - 1) / kGdnChunk);
}

// The plan: chunks in all, requests that have some; then, for each request with chunks in order, itself, its first slot
// and its rows; then first[B].
enum GdnPlanAt { kPlanChunks, kPlanRequests, kPlanOrder = 4 };
__device__ __forceinline__ int4 *gdn_order(const GdnPreArgs &a) { return reinterpret_cast<int4 *>(a.plan + kPlanOrder); }
__device__ __forceinline__ int32_t *gdn_first(const GdnPreArgs &a) { return a.plan + kPlanOrder + 4 * (int64_t)a.B; }

// By one CTA of THR threads: each sums a run of requests, and writes the run again with what lies before it.  A few
// bytes a request, two dependent reads.
template <int THR> __device__ void gdn_plan(const GdnPreArgs &a) {
    __shared__ long long wsum[THR / 32];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int per = (a.B + THR - 1) / THR, b0 = min(a.B, tid * per), b1 = min(a.B, b0 + per);
    // chunks in the low 44 bits (65535 requests of at most 2^25), requests above
    int r0, r1;
    auto count = [&](int b) {
        const long long n = gdn_chunks(a, b, r0, r1);
        return n ? n + (1ll << 44) : 0;
    };
    long long mine = 0;
    for (int b = b0; b < b1; ++b) mine += count(b);
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
    auto chunks = [](long long v) { return (int)min(v & ((1ll << 44) - 1), 0x7fffffffll); };
    for (int b = b0; b < b1; ++b) {
        const long long n = count(b);
        gdn_first(a)[b] = chunks(x);
        if (n) gdn_order(a)[x >> 44] = make_int4(b, chunks(x), r0, r1);
        x += n;
    }
    if (tid == THR - 1) {
        a.plan[kPlanChunks] = chunks(x);
        a.plan[kPlanRequests] = (int)(x >> 44);
    }
}

}  // namespace rssm
