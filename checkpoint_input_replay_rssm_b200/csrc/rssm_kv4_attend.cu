// rssm_kv4_attend.cu -- causal grouped-query attention over the paged 4-bit cache
// (rssm_kv4_attend).
//
//   out = sum_j p_j V_j / sum_j p_j,  p_j = exp(sm_scale q . K_j - m),  m the running maximum
//
// One CTA per (query row, query head); its warps take the cached tokens in turn, a
// lane holding D / 32 channels, and join their (m, sum, O) at the end.
#include <cuda_bf16.h>

#include <math.h>

#include "rssm_internal.h"
#include "rssm_kv4.cuh"

namespace rssm {

namespace {

struct AttendArgs {
    Kv4Args kv;
    int B, Hq, tokens, max_pages, max_q, max_seq;
    float scale;
    const __nv_bfloat16 *q;
    const uint8_t *cache;
    const int32_t *table, *seq_len, *cu;
    __nv_bfloat16 *out;
    int32_t *err;
};

// The rows and length of request b; false (and reported) where they do not fit the call.
__device__ __forceinline__ bool attend_request(const AttendArgs &a, int b, int &r0, int &n, int &len) {
    int r1;
    const bool ok = packed_rows(a.cu, b, a.tokens, r0, r1);
    n = r1 - r0;
    len = a.seq_len[b];
    return ok && n <= a.max_q && len >= 0 && len <= a.max_seq && len <= (int64_t)a.max_pages * a.kv.ps;
}

constexpr int kAttWarps = 4;

__device__ __forceinline__ float e2m1_value(uint32_t c) {
    const float m = (c & 6) == 0 ? 0.5f * (c & 1) : ldexpf(1.f + 0.5f * (c & 1), (int)((c >> 1) & 3) - 1);
    return (c & 8) ? -m : m;
}
__device__ __forceinline__ float e4m3_f(uint32_t b) {
    return __half2float(__half(__nv_cvt_fp8_to_halfraw((__nv_fp8_storage_t)b, __NV_E4M3)));
}

template <int D>
__global__ void __launch_bounds__(32 * kAttWarps) attend_rows_kernel(const AttendArgs a) {
    constexpr int E = D / 32;
    __shared__ float so[kAttWarps][D], sm[kAttWarps], sl[kAttWarps];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int i = blockIdx.x, hq = blockIdx.y, b = blockIdx.z;
    int r0, n, len;
    if (!attend_request(a, b, r0, n, len)) {
        if (threadIdx.x == 0) report_opt(a.err, DEV_BAD_LENGTHS, b, 0, len);
        return;
    }
    if (i >= n) return;
    const int seen = len - n + i + 1, h = hq / (a.Hq / a.kv.Hk), ps = a.kv.ps;
    const int64_t at = ((int64_t)(r0 + i) * a.Hq + hq) * D + lane * E;
    float q[E], o[E] = {}, m = -INFINITY, l = 0.f;
#pragma unroll
    for (int e = 0; e < E; ++e) q[e] = __bfloat162float(a.q[at + e]) * a.scale;
    for (int t = warp; t < seen; t += kAttWarps) {
        const int page = a.table[(int64_t)b * a.max_pages + t / ps], off = t % ps;
        if (page < 0 || page >= a.kv.pages) {
            if (lane == 0) report_opt(a.err, DEV_BAD_PAGE, b, h, page);
            continue;
        }
        const uint8_t *kb = a.cache + ((int64_t)page * a.kv.Hk + h) * kv4_head_bytes(ps, D), *vb = kb + ps * (D * 9 / 16);
        const float ks = e4m3_f(kb[ps * (D / 2) + off * (D / 16) + lane * E / 16]) * a.kv.k_scale;
        const float vs = e4m3_f(vb[ps * (D / 2) + off * (D / 16) + lane * E / 16]) * a.kv.v_scale;
        float s = 0.f, v[E];
#pragma unroll
        for (int e = 0; e < E; ++e) {
            const int byte = off * (D / 2) + (lane * E + e) / 2, sh = 4 * (e & 1);
            s = fmaf(q[e], e2m1_value((kb[byte] >> sh) & 15) * ks, s);
            v[e] = e2m1_value((vb[byte] >> sh) & 15) * vs;
        }
#pragma unroll
        for (int d = 16; d; d >>= 1) s += __shfl_xor_sync(0xffffffffu, s, d);
        const float mn = fmaxf(m, s), c = expf(m - mn), p = expf(s - mn);
        l = l * c + p;
#pragma unroll
        for (int e = 0; e < E; ++e) o[e] = o[e] * c + p * v[e];
        m = mn;
    }
#pragma unroll
    for (int e = 0; e < E; ++e) so[warp][lane * E + e] = o[e];
    if (lane == 0) {
        sm[warp] = m;
        sl[warp] = l;
    }
    __syncthreads();
    if (warp) return;
    float mm = -INFINITY, ll = 0.f;
    for (int w = 0; w < kAttWarps; ++w) mm = fmaxf(mm, sm[w]);
#pragma unroll
    for (int e = 0; e < E; ++e) o[e] = 0.f;
    for (int w = 0; w < kAttWarps; ++w) {
        const float c = sm[w] == -INFINITY ? 0.f : expf(sm[w] - mm);
        ll += c * sl[w];
#pragma unroll
        for (int e = 0; e < E; ++e) o[e] += c * so[w][lane * E + e];
    }
#pragma unroll
    for (int e = 0; e < E; ++e) a.out[at + e] = __float2bfloat16_rn(ll > 0.f || ll != ll ? o[e] / ll : 0.f);
}

bool attend_valid(const rssm_kv4_config *c, const rssm_attend_config *t, Kv4Args *kv) {
    if (!kv4_args(c, kv) || !t) return false;
    if (t->batch < 1 || t->batch > 65535 || t->n_q_heads < 1 || t->n_q_heads > 65535 || t->n_q_heads % kv->Hk != 0)
        return false;
    if (t->tokens < 1 || t->max_pages < 1 || t->max_q < 1 || t->max_seq < 1 || !isfinite(t->sm_scale)) return false;
    return true;
}

}  // namespace

}  // namespace rssm

extern "C" {

RSSM_API size_t rssm_kv4_attend_workspace_bytes(const rssm_kv4_config *cfg, const rssm_attend_config *att) {
    return 0;
}

RSSM_API rssm_status rssm_kv4_attend(const rssm_kv4_config *cfg, const rssm_attend_config *att, const void *q,
                                     const void *cache, const int32_t *block_table, const int32_t *seq_len,
                                     const int32_t *cu_q, void *out, void *workspace, size_t workspace_bytes,
                                     int32_t *dev_error, void *stream) {
    using namespace rssm;
    AttendArgs a{};
    if (!attend_valid(cfg, att, &a.kv) || !q || !cache || !block_table || !seq_len || !cu_q || !out) return RSSM_EINVAL;
    if (!aligned16(q) || !aligned16(cache) || !aligned16(out)) return RSSM_EINVAL;
    a.B = att->batch; a.Hq = att->n_q_heads; a.tokens = att->tokens; a.max_pages = att->max_pages;
    a.max_q = att->max_q; a.max_seq = att->max_seq; a.scale = att->sm_scale;
    a.q = (const __nv_bfloat16 *)q; a.cache = (const uint8_t *)cache;
    a.table = block_table; a.seq_len = seq_len; a.cu = cu_q; a.out = (__nv_bfloat16 *)out; a.err = dev_error;
    auto k = a.kv.D == 64 ? attend_rows_kernel<64> : attend_rows_kernel<128>;
    k<<<dim3(a.max_q, a.Hq, a.B), 32 * kAttWarps, 0, (cudaStream_t)stream>>>(a);
    return cudaGetLastError() == cudaSuccess ? RSSM_OK : RSSM_ECUDA;
}

}  // extern "C"
