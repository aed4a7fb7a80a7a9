// rssm_gdn_prefill.cu -- the gated delta rule over packed prompts (rssm_gdn_prefill):
// every token's output and the fp32 state after each prompt, which a replay decode
// starts from (rssm_import_state).
//
// Recurrent form, for any supported shape and input type, all arithmetic fp32.  The
// state's rows are independent (row p meets only v[p]), so a warp owns 8 of them and
// keeps them in registers over the whole prompt.  Per token and row s:
//   a = alpha s,  c = beta (v[p] - a . k),  o[p] = a . q + c (k . q),  s = a + c k
// The output is written from the decayed old state, so that the dot products a.k and a.q
// are one reduction (8 lanes, 3 shuffles) instead of two in sequence, and k.q is formed
// once per token for all rows: the issue of a token's instructions and the chain through
// the reduction bound this kernel, not HBM.  A row's columns lie over 8 lanes in pieces
// of 16 bytes, 4 lane groups of 2 rows each; products take two columns an instruction
// (fp32 pairs).  Tokens are staged 16 at a time in shared memory (fp32), the next 16 in
// flight meanwhile.
//
// 16 prompts of 1 to 200 tokens, 16 heads, P = N = 64, fp32: 66 us of 6 at the rate of a copy.  The longest prompt
// decides: about a third of a us a token, most of it the chain products -> shuffles -> state.
#include "rssm_gdn_plan.cuh"
#include "rssm_internal.h"
#include "rssm_pair.cuh"

namespace rssm {

namespace {

constexpr int kRecWarps = 4;             // 8 state rows each
constexpr int kRecRows = 8 * kRecWarps;  // rows of one CTA
constexpr int kRecTok = 16;              // tokens staged at a time

template <typename IN> __device__ __forceinline__ float in_value(const void *p, int64_t i);
template <> __device__ __forceinline__ float in_value<float>(const void *p, int64_t i) { return ((const float *)p)[i]; }
template <> __device__ __forceinline__ float in_value<__nv_bfloat16>(const void *p, int64_t i) {
    return __bfloat162float(((const __nv_bfloat16 *)p)[i]);
}

template <typename IN, int N>
__global__ void __launch_bounds__(32 * kRecWarps) gdn_recurrent_kernel(const GdnPreArgs a) {
    constexpr int kThr = 32 * kRecWarps;
    constexpr int V = N >= 32 ? 4 : 2;  // columns per piece
    constexpr int J = N / (8 * V);      // pieces per lane
    constexpr int U = J * V / 2;        // pairs per lane and row
    constexpr int NQ = kRecTok * N / kThr, NV = kRecTok * kRecRows / kThr;
    typedef unsigned long long u64;
    __shared__ __align__(16) float sk[2][kRecTok][N], sq[2][kRecTok][N];
    __shared__ float sv[2][kRecTok][kRecRows], sa[2][kRecTok], sb[2][kRecTok], skq[kRecTok];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int l8 = lane & 7, g4 = lane >> 3;
    // Beside the chunked form (plan is set) this kernel has the short requests.
    const bool beside = N == 128 && sizeof(IN) == 2 && a.plan;
    // It does not end before the kernels that it was started beside: its first CTA waits for them.
    auto end = [&] {
        if (beside && (blockIdx.x | blockIdx.y | blockIdx.z) == 0) pdl_wait();
    };
    const int h = blockIdx.y, b = blockIdx.z, p0 = blockIdx.x * kRecRows;
    const int rows = min(kRecRows, a.P - p0);
    int r0, r1;
    if (!packed_rows(a.cu, b, a.tokens, r0, r1)) {
        if (tid == 0) report_opt(a.err, DEV_BAD_LENGTHS, b, h, r1);
        return end();
    }
    if (beside && r1 - r0 > kGdnShort) return end();
    const int64_t head = (int64_t)b * a.H + h;
    const int row0 = 8 * warp + 2 * g4;  // this lane group's rows: row0, row0 + 1 (P is a multiple of 8)
    const bool on = row0 < rows;
    // This lane's pairs of a row of N values: V consecutive ones of every 8 V.
    auto pairs = [&](const float *row, u64 (&x)[U]) {
#pragma unroll
        for (int j = 0; j < J; ++j) {
            const float *at = row + j * 8 * V + l8 * V;
            if constexpr (V == 4) {
                const ulonglong2 v = *reinterpret_cast<const ulonglong2 *>(at);
                x[2 * j] = v.x;
                x[2 * j + 1] = v.y;
            } else {
                x[j] = *reinterpret_cast<const u64 *>(at);
            }
        }
    };
    u64 s[2][U];
#pragma unroll
    for (int r = 0; r < 2; ++r) {
#pragma unroll
        for (int u = 0; u < U; ++u) s[r][u] = 0;
        if (on && a.S0) pairs(a.S0 + (head * a.P + p0 + row0 + r) * N, s[r]);
    }

    float rk[NQ], rq[NQ], rv[NV], ra = 0.f, rb = 0.f;
    auto fetch = [&](int t0) {
#pragma unroll
        for (int i = 0; i < NQ; ++i) {
            const int e = tid + i * kThr, t = e / N, n = e % N;
            const int64_t at = ((int64_t)(t0 + t) * a.H + h) * N + n;
            const bool live = t0 + t < r1;
            rk[i] = live ? in_value<IN>(a.k, at) : 0.f;
            rq[i] = live ? in_value<IN>(a.q, at) : 0.f;
        }
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int e = tid + i * kThr, t = e / kRecRows, p = e % kRecRows;
            rv[i] = t0 + t < r1 && p < rows ? in_value<IN>(a.v, ((int64_t)(t0 + t) * a.H + h) * a.P + p0 + p) : 0.f;
        }
        if (tid < kRecTok) {
            const bool live = t0 + tid < r1;
            ra = live ? a.alpha[(int64_t)(t0 + tid) * a.H + h] : 0.f;
            rb = live ? a.beta[(int64_t)(t0 + tid) * a.H + h] : 0.f;
        }
    };
    auto put = [&](int buf) {
#pragma unroll
        for (int i = 0; i < NQ; ++i) {
            const int e = tid + i * kThr;
            sk[buf][e / N][e % N] = rk[i];
            sq[buf][e / N][e % N] = rq[i];
        }
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int e = tid + i * kThr;
            sv[buf][e / kRecRows][e % kRecRows] = rv[i];
        }
        if (tid < kRecTok) {
            sa[buf][tid] = ra;
            sb[buf][tid] = rb;
        }
    };

    int buf = 0;
    if (r0 < r1) fetch(r0);
    for (int t0 = r0; t0 < r1; t0 += kRecTok, buf ^= 1) {
        put(buf);  // the other buffer's readers passed the barrier of the step before
        __syncthreads();
        if (t0 + kRecTok < r1) fetch(t0 + kRecTok);
        const int nt = min(kRecTok, r1 - t0);
        // k . q of every token, 8 lanes a token: once for all of the CTA's rows
        {
            const int t = 4 * warp + g4;
            u64 kk[U], qq[U], d2 = 0;
            pairs(sk[buf][t], kk);
            pairs(sq[buf][t], qq);
#pragma unroll
            for (int u = 0; u < U; ++u) d2 = f2_fma(kk[u], qq[u], d2);
            float lo, hi;
            f2_unpack(d2, lo, hi);
            lo += hi;
#pragma unroll
            for (int o = 1; o < 8; o <<= 1) lo += __shfl_xor_sync(0xffffffffu, lo, o);
            if (l8 == 0) skq[t] = lo;
        }
        __syncthreads();
#pragma unroll 2
        for (int t = 0; t < nt; ++t) {
            const float al = sa[buf][t], be = sb[buf][t], kq = skq[t];
            const u64 al2 = f2_pack(al, al);
            u64 kk[U], qq[U], dk2[2] = {0, 0}, dq2[2] = {0, 0};
            pairs(sk[buf][t], kk);
            pairs(sq[buf][t], qq);
#pragma unroll
            for (int u = 0; u < U; ++u)
#pragma unroll
                for (int r = 0; r < 2; ++r) {
                    s[r][u] = f2_mul(s[r][u], al2);
                    dk2[r] = f2_fma(s[r][u], kk[u], dk2[r]);
                    dq2[r] = f2_fma(s[r][u], qq[u], dq2[r]);
                }
            float dk[2], dq[2];
#pragma unroll
            for (int r = 0; r < 2; ++r) {
                float lo, hi;
                f2_unpack(dk2[r], lo, hi);
                dk[r] = lo + hi;
                f2_unpack(dq2[r], lo, hi);
                dq[r] = lo + hi;
            }
#pragma unroll
            for (int o = 1; o < 8; o <<= 1)
#pragma unroll
                for (int r = 0; r < 2; ++r) {
                    dk[r] += __shfl_xor_sync(0xffffffffu, dk[r], o);
                    dq[r] += __shfl_xor_sync(0xffffffffu, dq[r], o);
                }
            float o[2];
#pragma unroll
            for (int r = 0; r < 2; ++r) {
                const float c = be * (sv[buf][t][row0 + r] - dk[r]);
                const u64 c2 = f2_pack(c, c);
                o[r] = fmaf(c, kq, dq[r]);
#pragma unroll
                for (int u = 0; u < U; ++u) s[r][u] = f2_fma(c2, kk[u], s[r][u]);
            }
            if (l8 == 0 && on)
                *reinterpret_cast<float2 *>(a.y + ((int64_t)(t0 + t) * a.H + h) * a.P + p0 + row0) =
                    make_float2(o[0], o[1]);
        }
    }
    if (on)
#pragma unroll
        for (int r = 0; r < 2; ++r)
#pragma unroll
            for (int u = 0; u < U; ++u) {
                const int at = V == 4 ? (u >> 1) * 32 + l8 * 4 + 2 * (u & 1) : u * 16 + l8 * 2;
                *reinterpret_cast<u64 *>(a.S_out + (head * a.P + p0 + row0 + r) * N + at) = s[r][u];
            }
    end();
}

}  // namespace

template <typename IN>
cudaError_t gdn_recurrent_launch(const GdnPreArgs &a, int N, cudaStream_t st) {
    auto k = N == 16 ? gdn_recurrent_kernel<IN, 16>
                     : N == 32 ? gdn_recurrent_kernel<IN, 32>
                               : N == 64 ? gdn_recurrent_kernel<IN, 64> : gdn_recurrent_kernel<IN, 128>;
    const dim3 grid((a.P + kRecRows - 1) / kRecRows, a.H, a.B);
    if (a.plan) return launch_early(k, grid, 32 * kRecWarps, 0, a, st);
    k<<<grid, 32 * kRecWarps, 0, st>>>(a);
    return cudaGetLastError();
}
template cudaError_t gdn_recurrent_launch<__nv_bfloat16>(const GdnPreArgs &, int, cudaStream_t);

namespace {

int gdn_dtype(const rssm_gdn_prefill_config &c) { return c.input_dtype & ~RSSM_GDN_FP32; }

bool gdn_prefill_valid(const rssm_gdn_prefill_config *c) {
    return c && c->batch >= 1 && c->batch <= 65535 && c->nheads >= 1 && c->nheads <= 65535 && c->headdim >= 8 &&
           c->headdim <= 256 && c->headdim % 8 == 0 &&
           (c->dstate == 16 || c->dstate == 32 || c->dstate == 64 || c->dstate == 128) &&
           (gdn_dtype(*c) == RSSM_F32 || gdn_dtype(*c) == RSSM_BF16) && c->tokens >= 1;
}

// Whether the call may have requests for the chunked form: what its tiles are made for, and rows for a longer one.
bool gdn_chunked(const rssm_gdn_prefill_config &c) {
    return c.dstate == 128 && c.input_dtype == RSSM_BF16 && c.tokens > kGdnShort;  // (and not by the recurrence on request)
}

}  // namespace

}  // namespace rssm

extern "C" {

RSSM_API size_t rssm_gdn_prefill_workspace_bytes(const rssm_gdn_prefill_config *cfg) {
    using namespace rssm;
    return gdn_prefill_valid(cfg) && gdn_chunked(*cfg) ? gdn_chunk_bytes(cfg->batch, cfg->nheads, cfg->tokens) : 0;
}

RSSM_API rssm_status rssm_gdn_prefill(const rssm_gdn_prefill_config *cfg, const float *S0, const rssm_inputs *in,
                                      const int32_t *cu, float *y, float *S_out, void *workspace,
                                      size_t workspace_bytes, int32_t *dev_error, void *stream) {
    using namespace rssm;
    if (!gdn_prefill_valid(cfg) || !in || !in->q || !in->k || !in->v || !in->alpha || !in->beta || !cu || !y || !S_out)
        return RSSM_EINVAL;
    if (S0 && S0 == S_out) return RSSM_EINVAL;
    if (!aligned16(in->q) || !aligned16(in->k) || !aligned16(in->v) || !aligned16(y) || !aligned16(S_out) ||
        !aligned16(S0))
        return RSSM_EINVAL;
    const size_t need = rssm_gdn_prefill_workspace_bytes(cfg);
    if (need && (!workspace || workspace_bytes < need || ((uintptr_t)workspace & 255))) return RSSM_EINVAL;
    const rssm_gdn_prefill_config &c = *cfg;
    const GdnPreArgs a{c.batch, c.nheads, c.headdim, c.tokens, in->q, in->k, in->v, in->alpha, in->beta,
                       cu, S0, y, S_out, 0, nullptr, nullptr, dev_error};
    const cudaError_t e = gdn_chunked(c) ? gdn_chunk_launch(a, (uint8_t *)workspace, (cudaStream_t)stream)
                          : gdn_dtype(c) == RSSM_BF16 ? gdn_recurrent_launch<__nv_bfloat16>(a, c.dstate, (cudaStream_t)stream)
                                                      : gdn_recurrent_launch<float>(a, c.dstate, (cudaStream_t)stream);
    return e == cudaSuccess ? RSSM_OK : RSSM_ECUDA;
}

}  // extern "C"
