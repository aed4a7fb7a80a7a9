// rssm_tables.cu -- block table, slot map and packed offsets of one step, built on
// the device from the requests' lengths (rssm_build_tables).
//
//   cu_new[b] = sum_{c < b} new_len[c]
//   fresh[b]  = ceil((cached + new) / ps) - ceil(cached / ps), first[b] = sum_{c < b} fresh[c]
//   table[b][held_b + i] = free_pages[head + first[b] + i],  i < fresh[b], held_b = ceil(cached_b / ps)
//   slot(token t of request b at position p) = table[b][p / ps] * ps + p % ps
//
// Whole-number work of a few bytes per request and 8 bytes per token, so a call is
// bound by its launch and by the chain load lengths -> scan -> write.  One launch:
// every CTA scans all the lengths by itself (4 bytes x 2 per request from L2,
// cheaper than a second launch or a grid barrier), keeps the sums in shared
// memory, and then serves its share of the new pages and of the tokens, finding a
// page's or token's request by bisection in the sums.  A fresh page's id comes
// from the free list directly, so no CTA waits for another's table entries.  The
// step is refused as a whole, which every CTA decides from the same scan.
//
// 256 decoding requests take 6.5 us on the device, 96 prompts of up to 4096 tokens 9 us (1.5 MB
// written, 0.23 us at the rate of a copy): launch, three dependent accesses and the scan's
// barriers.  A call from Python takes about 15 us of either, on the host.
#include "rssm_internal.h"
#include "rssm_packed.cuh"

namespace rssm {

namespace {

constexpr int kTabThreads = 512;
constexpr int kTabTokens = 4;        // tokens per thread before another CTA is added
constexpr int kMaxRequests = 16384;  // two int32 sums per request in shared memory (128 KiB)

constexpr int kMaxCount = 1 << 30;   // tokens and free pages: int32 strides over them do not overflow

struct TablesArgs {
    int B, ps, max_pages, num_free, max_tokens;
    const int32_t *cached, *fresh_len, *free_pages, *free_head;
    int32_t *table, *cu, *seq_len, *slot, *pos, *next_free, *err;
};

// Largest b with sums[b] <= v, for sums[0] = 0 <= v < sums[B].
__device__ __forceinline__ int request_of(const int *sums, int B, int v) {
    int lo = 0, hi = B;
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (sums[mid] <= v) lo = mid;
        else hi = mid;
    }
    return lo;
}

__global__ void __launch_bounds__(kTabThreads) tables_kernel(const TablesArgs a) {
    extern __shared__ int sh[];
    int *cu = sh, *first = sh + a.B + 1;
    __shared__ long long wsum[2][kTabThreads / 32];
    __shared__ int bad_b;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, nw = kTabThreads / 32;
    const int B = a.B, ps = a.ps;
    if (tid == 0) bad_b = 0x7fffffff;
    __syncthreads();

    // This thread's run of requests: 64-bit sums, so that lengths that do not fit show as such.
    const int per = (B + kTabThreads - 1) / kTabThreads;
    const int b0 = min(B, tid * per), b1 = min(B, b0 + per);
    long long st = 0, sp = 0;
    for (int b = b0; b < b1; ++b) {
        const long long c = a.cached[b], n = a.fresh_len[b];
        if (c < 0 || n < 0 || c + n > (long long)a.max_pages * ps) {
            atomicMin(&bad_b, b);
        } else {
            st += n;
            sp += (c + n + ps - 1) / ps - (c + ps - 1) / ps;
        }
    }
    long long xt = st, xp = sp;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const long long ut = __shfl_up_sync(0xffffffffu, xt, o), up = __shfl_up_sync(0xffffffffu, xp, o);
        if (lane >= o) {
            xt += ut;
            xp += up;
        }
    }
    if (lane == 31) {
        wsum[0][warp] = xt;
        wsum[1][warp] = xp;
    }
    __syncthreads();
    long long ct = 0, cp = 0, tokens = 0, pages = 0;
    for (int w = 0; w < nw; ++w) {
        if (w < warp) {
            ct += wsum[0][w];
            cp += wsum[1][w];
        }
        tokens += wsum[0][w];
        pages += wsum[1][w];
    }
    const int head = *a.free_head;
    const bool bad_len = bad_b != 0x7fffffff || tokens > a.max_tokens;
    const bool no_pages = !bad_len && (head < 0 || head + pages > a.num_free);
    const bool lead = blockIdx.x == 0;
    const int gid = blockIdx.x * kTabThreads + tid, gsize = gridDim.x * kTabThreads;
    if (bad_len || no_pages) {  // the same in every CTA
        if (lead) {
            for (int b = tid; b < B; b += kTabThreads) {
                a.cu[b + 1] = 0;
                a.seq_len[b] = a.cached[b];
            }
            if (tid == 0) {
                a.cu[0] = 0;
                *a.next_free = head;
                const bool one = bad_b != 0x7fffffff;
                report_opt(a.err, bad_len ? DEV_BAD_LENGTHS : DEV_NO_PAGES, one ? bad_b : -1, 0,
                           (int)min(bad_len ? tokens : pages, 0x7fffffffLL));
            }
        }
        for (int t = gid; t < a.max_tokens; t += gsize) {
            a.slot[t] = -1;
            a.pos[t] = -1;
        }
        return;
    }
    int rt = (int)(ct + xt - st), rp = (int)(cp + xp - sp);
    for (int b = b0; b < b1; ++b) {
        const int c = a.cached[b], n = a.fresh_len[b];
        cu[b] = rt;
        first[b] = rp;
        if (lead) {
            a.cu[b] = rt;
            a.seq_len[b] = c + n;
        }
        rt += n;
        rp += (int)(((long long)c + n + ps - 1) / ps - ((long long)c + ps - 1) / ps);
    }
    if (tid == 0) {
        cu[B] = (int)tokens;
        first[B] = (int)pages;
        if (lead) {
            a.cu[B] = (int)tokens;
            *a.next_free = head + (int)pages;
        }
    }
    __syncthreads();

    for (int i = gid; i < (int)pages; i += gsize) {
        const int b = request_of(first, B, i);
        const int held = (int)(((long long)a.cached[b] + ps - 1) / ps);
        a.table[(int64_t)b * a.max_pages + held + (i - first[b])] = a.free_pages[head + i];
    }
    for (int t = gid; t < a.max_tokens; t += gsize) {
        int slot = -1, p = -1;
        if (t < (int)tokens) {
            const int b = request_of(cu, B, t);
            const int c = a.cached[b];
            p = c + (t - cu[b]);
            const int at = p / ps, held = (int)(((long long)c + ps - 1) / ps);
            const int page = at < held ? a.table[(int64_t)b * a.max_pages + at]
                                       : a.free_pages[head + first[b] + at - held];
            const long long s = (long long)page * ps + (p - at * ps);
            slot = page < 0 || s > 0x7fffffffLL ? -1 : (int)s;
        }
        a.slot[t] = slot;
        a.pos[t] = p;
    }
}

}  // namespace

}  // namespace rssm

extern "C" RSSM_API rssm_status rssm_build_tables(const rssm_tables_config *cfg, const int32_t *cached_len,
                                                  const int32_t *new_len, const int32_t *free_pages,
                                                  const int32_t *free_head, int32_t *block_table, int32_t *cu_new,
                                                  int32_t *seq_len, int32_t *slot_map, int32_t *position,
                                                  int32_t *next_free, int32_t *dev_error, void *stream) {
    using namespace rssm;
    if (!cfg || !cached_len || !new_len || !free_head || !block_table || !cu_new || !seq_len || !slot_map ||
        !position || !next_free || next_free == free_head || seq_len == cached_len || seq_len == new_len)
        return RSSM_EINVAL;
    const rssm_tables_config &c = *cfg;
    if (c.batch < 1 || c.batch > kMaxRequests || c.page_size < 1 || c.page_size > 65536 || c.max_pages < 1 ||
        c.num_free < 0 || c.num_free > kMaxCount || c.max_tokens < 1 || c.max_tokens > kMaxCount ||
        (c.num_free > 0 && !free_pages))
        return RSSM_EINVAL;
    // positions and lengths are int32
    if ((int64_t)c.max_pages * c.page_size > 0x7fffffffLL) return RSSM_EINVAL;
    TablesArgs a{c.batch, c.page_size, c.max_pages, c.num_free, c.max_tokens, cached_len, new_len, free_pages,
                 free_head, block_table, cu_new, seq_len, slot_map, position, next_free, dev_error};
    const size_t smem = (size_t)(2 * (c.batch + 1)) * sizeof(int);
    // What needs no permission is 48 KiB of the sums and the kernel's own arrays together (less than 1 KiB of them).
    if (smem > 47 * 1024 && cudaFuncSetAttribute(tables_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                                 2 * (kMaxRequests + 1) * (int)sizeof(int)) != cudaSuccess)
        return RSSM_ECUDA;
    const int64_t work = c.max_tokens > c.batch ? c.max_tokens : c.batch;
    const int64_t per = kTabThreads * kTabTokens;
    const int64_t grid = (work + per - 1) / per;
    tables_kernel<<<(unsigned)(grid < 1184 ? grid : 1184), kTabThreads, smem, (cudaStream_t)stream>>>(a);
    return cudaGetLastError() == cudaSuccess ? RSSM_OK : RSSM_ECUDA;
}
