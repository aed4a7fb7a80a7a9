// rssm_gdn_chunk.cu -- the gated delta rule over packed prompts in chunks of 64
// tokens on the 5th-generation tensor cores (N = 128, bf16 inputs).
//
// With Lam_i = sum_{j <= i} log2 alpha_j over the chunk, S the state (P x N) at its start,
// K, Q, V the chunk's rows, and u_i = beta_i (v_i - alpha_i S_{i-1} k_i) the write of token i:
//   A_ij = beta_i 2^{Lam_i - Lam_j} k_i.k_j (j < i),   T = (I + A)^{-1}
//   R = V - diag(2^Lam) K S^T,   U = (T diag(beta)) R
//   O = diag(2^Lam) Q S^T + (M T diag(beta)) R,   M_ij = 2^{Lam_i - Lam_j} q_i.k_j (j <= i)
//   S <- 2^{Lam_C} S + sum_j 2^{Lam_C - Lam_j} u_j k_j^T
// What does not meet the state is one kernel over all chunks at once: it leaves the 128 x 64
// matrix [T diag(beta); M T diag(beta)] for the other, which walks the chunks of one
// (request, head, 128 rows of the state) with three products a chunk:
//   S [K; Q]^T       (128 x 128 x 128: the K columns give R, the Q columns the first part of O)
//   R^T [T b; M T b]^T  (128 x 128 x 64: the K columns give U, the Q columns the second part of O)
//   (w U)^T K        (128 x 128 x 64 onto the state, which stays in tensor memory)
// q, k and v are bf16 and enter exactly; fp32 operands enter as a (hi, lo) bf16 pair, which
// leaves 2^-18 of the value, and the lo lo product is dropped (2^-18): near-fp32 accuracy at
// two or three bf16 products, where one tf32 product would leave 2^-11.
//
// T comes from forward substitution in fp32, in blocks: the 16 x 16 diagonal blocks
// column by column, then T_21 = -T_22 A_21 T_11 twice.  (The product of I + (-A)^{2^i} is shorter
// and fails where keys repeat: the powers of A grow to 10^17 and cancel.)  Lam is summed in 64
// bits and kept as two fp32, so that a difference between neighbours is exact to fp32 however far
// down the chunk they are.
//
// Values that are not finite.  A product over a chunk's tokens meets every token with every other, the later ones with a
// factor of zero, and zero times an infinity or a NaN is NaN: a token that brings one would reach outputs before it.
// So the factors are kept finite.  The chunk kernel puts zeros in A and T and hands on the first token that is lost (by k, alpha,
// beta, or a system that grows past fp32); the scan puts zeros in R from that token on, and from the first such value of v
// on in its state row.  Outputs of the row from there on and its last state are then NaN, whatever was computed for
// them.  An infinity or a NaN in q has only its own row of M and column of Y; in S, all that follows in its row is lost.
//
// Request b's chunk c has slot first[b] + c, first[] a prefix sum that a kernel before makes (rssm_gdn_plan.cuh).
// It takes nothing from the offsets on trust; slots at r0 / 64 + b + c, which need no sum, are distinct only where
// every request's offsets are in order.
//
// 64 prompts of 1 to 1024 tokens (34500 in all), 32 heads, P = 128: 412 us for the chunk kernel and 500 for the
// scan, of 259 at the rate of a copy for both (together 1.9 TB/s of what a call has to move).  The chunk kernel is
// bound by its short fp32 steps out of shared memory: warps wait at the barriers between them, and that pipe is 67% busy (four
// CTAs an SM, which its shared memory and registers allow).  The scan is a chain: 2.7 us a chunk of a prompt, three products that wait
// for each other and the conversions between them, with one CTA an SM, and about 13 us to start and end a CTA.  One
// prompt of 8191 tokens: 98 and 355 us.
#include <cuda_bf16.h>

#include "rssm_gdn_plan.cuh"
#include "rssm_umma.cuh"

namespace rssm {

namespace {

constexpr int kC = kGdnChunk;           // 64 tokens
constexpr int kDk = 128;                // state columns (N)
constexpr int kTile = 128 * kC * 2;     // [128 x 64] bf16
constexpr int kSlot = 2 * kTile + 528;  // hi, lo, then 2^Lam_i and 2^{Lam_C - Lam_i} fp32, then the first lost token

// Eight fp32 values as 16-byte chunks of their (hi, lo) parts.  The conversions are the two-value ones: the
// one-value form runs at an eighth of their rate.
__device__ __forceinline__ uint32_t bf16x2(float lo, float hi) {
    uint32_t r;
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
}
__device__ __forceinline__ void split8(const float *v, uint4 &hi, uint4 &lo) {
    uint32_t *ph = &hi.x, *pl = &lo.x;
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        const uint32_t h = bf16x2(v[2 * e], v[2 * e + 1]);
        ph[e] = h;
        pl[e] = bf16x2(v[2 * e] - __uint_as_float(h << 16), v[2 * e + 1] - __uint_as_float(h & 0xffff0000u));
    }
}
// Whether all n values are finite: one multiply-add a value.
template <int n> __device__ __forceinline__ bool all_finite(const float *v) {
    float z[2] = {0.f, 0.f};
#pragma unroll
    for (int j = 0; j < n; ++j) z[j & 1] = fmaf(v[j], 0.f, z[j & 1]);
    return z[0] + z[1] == 0.f;
}
// n values of row i of a factor as a product may have them, *first the first row that was not finite.
template <int n> __device__ __forceinline__ void keep_finite(float *v, int i, int *first) {
    if (all_finite<n>(v)) return;
    atomicMin(first, i);
#pragma unroll
    for (int j = 0; j < n; ++j)
        if (!isfinite(v[j])) v[j] = 0.f;
}
__device__ __forceinline__ void bulk_s2g(void *dst, const void *src, uint32_t bytes) {
    asm volatile("cp.async.bulk.global.shared::cta.bulk_group [%0], [%1], %2;" ::"l"(dst), "r"(smem_u32(src)), "r"(bytes)
                 : "memory");
}

// ---------------------------------------------------------------- chunk operands
constexpr int kLd = 68;  // fp32 row of A and T: 16-byte aligned, rows 4 banks apart
constexpr int kChunkThreads = 256;
struct ChunkSmem {
    static constexpr int kKQ = 0;  // [K; Q] 128 x 128 bf16 in two column blocks; the operand's hi and lo afterwards
    static constexpr int kHi = kKQ, kLo = kHi + kTile;
    static constexpr int kA = kLo + kTile;  // A, and T in its place
    static constexpr int kLam = kA + kC * kLd * 4;  // Lam hi, Lam lo, beta, 2^{Lam_ref - Lam}
    static constexpr int kBar = kLam + 4 * kC * 4;
    static constexpr int kBytes = kBar + 32;
};

// One chunk and head.  The barrier is in its first phase before and after; true where a wait gave up.
__device__ __forceinline__ bool chunk_unit(const GdnPreArgs &a, uint8_t *sm, uint64_t *bar, int *sfound, uint32_t tmem, int slot, int h) {
    using L = ChunkSmem;
    uint8_t *sKQ = sm + L::kKQ, *sHi = sm + L::kHi, *sLo = sm + L::kLo;
    float *sA = reinterpret_cast<float *>(sm + L::kA);
    float *lamh = reinterpret_cast<float *>(sm + L::kLam), *laml = lamh + kC, *sbeta = laml + kC, *sg = sbeta + kC;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, H = a.H;
    // The request of this slot: the last b with first[b] <= slot, 32 candidates a round.
    if (warp == 0) {
        const int32_t *first = gdn_first(a);
        int lo = 0, n = a.B;  // b is in [lo, lo + n)
        while (n > 1) {
            const int step = (n + 31) / 32, at = lo + lane * step;
            const bool le = lane * step < n && (lane == 0 || first[at] <= slot);
            const int last = 31 - __clz(__ballot_sync(0xffffffffu, le));
            n = min(step, n - last * step);
            lo += last * step;
        }
        if (lane == 0) {
            sfound[0] = lo;
            sfound[1] = slot - first[lo];
            sfound[2] = kC;
        }
    }
    __syncthreads();
    const int b = sfound[0], c = sfound[1];
    int *slost = sfound + 2;
    int r0, r1;
    const bool work = c < gdn_chunks(a, b, r0, r1);
    const int t0 = work ? r0 + c * kC : 0;
    bool failed = false;
    if (work) {
        const int Lc = min(kC, r1 - t0);
        float al[2] = {1.f, 1.f}, be[2] = {0.f, 0.f};  // gates of tokens 2 lane, 2 lane + 1
        if (warp == 0) {
#pragma unroll
            for (int e = 0; e < 2; ++e)
                if (2 * lane + e < Lc) {
                    al[e] = a.alpha[(int64_t)(t0 + 2 * lane + e) * H + h];
                    be[e] = a.beta[(int64_t)(t0 + 2 * lane + e) * H + h];
                }
        }
        // K and Q rows, 16 lanes a row, 16 rows a round; rows behind the prompt are zero.
        {
            const int r = tid >> 4, ch = tid & 15;
            const int64_t at = ((int64_t)(t0 + r) * H + h) * kDk + 8 * ch, step = 16 * (int64_t)H * kDk;
            const __nv_bfloat16 *k = reinterpret_cast<const __nv_bfloat16 *>(a.k) + at, *q = reinterpret_cast<const __nv_bfloat16 *>(a.q) + at;
            uint8_t *dst = sKQ + sw128_chunk(r, ch, 128);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const bool live = r + 16 * i < Lc;
                cp_async16_or_zero(dst + 2048 * i, live ? k + i * step : a.k, live);
                cp_async16_or_zero(dst + 2048 * (i + 4), live ? q + i * step : a.q, live);
            }
        }
        cp_async_commit();
        if (warp == 0) {
            // Lam.  A gate of 0 counts as 2^-200, which is 0 in every
            // fp32 product that it enters.
            double v[2];
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                const float lg = log2f(al[e]);
                v[e] = (double)(lg < -200.f ? -200.f : lg);
            }
            double x = v[0] + v[1];
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const double u = __shfl_up_sync(0xffffffffu, x, o);
                if (lane >= o) x += u;
            }
            const double ref = __shfl_sync(0xffffffffu, x, lane | 7);  // the last token of this 16-token block
            const double end = __shfl_sync(0xffffffffu, x, 31);
            float *out = reinterpret_cast<float *>(a.ws + ((int64_t)slot * H + h) * kSlot + 2 * kTile);
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                const double s = e ? x : x - v[1];
                const int t = 2 * lane + e;
                lamh[t] = (float)s;
                laml[t] = (float)(s - (double)(float)s);
                sbeta[t] = be[e];
                if (!(s < 128.0)) atomicMin(slost, t);  // not a number, or past fp32
                sg[t] = exp2f((float)(ref - s));
                out[t] = exp2f((float)s);  // decays that the scan wants
                out[kC + t] = exp2f((float)(end - s));
            }
        }
        cp_async_wait_all();
        fence_async_smem();
        __syncthreads();
        // G = [K; Q] K^T
        if (warp == 0 && elect_one()) {
            const uint32_t d = sw128_desc_lo(smem_u32(sKQ));
#pragma unroll
            for (int ks = 0; ks < kDk / 16; ++ks) {
                const uint64_t kd = sw128_desc_of(d + ((ks >> 2) * kTile + (ks & 3) * 32) / 16);
                umma_bf16(tmem, kd, kd, idesc_bf16_f32(128, kC), ks > 0);
            }
            umma_commit(bar);
        }
        __syncwarp();
        failed = !bar_wait(bar, 0);
        failed = __syncthreads_or(failed);
        tc_fence_after();
        if (!failed) {
            // Row i of A (lanes of K rows) or of M (Q rows), 32 columns a thread: its lower triangle with decays.
            // Left of the diagonal's 16-column block the decay is 2^{Lam_i - Lam_ref} 2^{Lam_ref - Lam_j}, ref the
            // last token of j's block, so that neither exponent is positive where gates are at most 1.
            const uint32_t base = tmem + ((uint32_t)(32 * (warp & 3)) << 16);
            const int row = tid & 127, i = row & 63, half = tid >> 7;
            const bool is_k = row < kC;
            const float li = lamh[i], ll = laml[i], bi = is_k ? sbeta[i] : 1.f;
            const int lim = is_k ? i : i + 1;       // columns below lim are kept
            const int last_blk = 2 * (warp & 1) + 1;  // of this warp's rows
#pragma unroll
            for (int q = 0; q < 2; ++q) {
                const int blk = 2 * half + q, j0 = 16 * blk;
                float gv[16];
                if (blk <= last_blk) {  // warp-uniform
                    tmem_ld16(base + j0, gv);
                    if ((i >> 4) == blk) {
                        if (is_k) {  // |k_i|^2 shows what k_i holds
                            float kk = 0.f;
#pragma unroll
                            for (int j = 0; j < 16; ++j) kk = j0 + j == i ? gv[j] : kk;
                            if (!isfinite(kk)) atomicMin(slost, i);
                        }
#pragma unroll
                        for (int j = 0; j < 16; j += 4) {
                            const float4 h4 = *reinterpret_cast<const float4 *>(lamh + j0 + j);
                            const float4 l4 = *reinterpret_cast<const float4 *>(laml + j0 + j);
#pragma unroll
                            for (int e = 0; e < 4; ++e) {
                                const float w = bi * ex2((li - (&h4.x)[e]) + (ll - (&l4.x)[e]));
                                gv[j + e] = j0 + j + e < lim ? w * gv[j + e] : 0.f;
                            }
                        }
                    } else {
                        const bool left = (i >> 4) > blk;
                        const float f = left ? bi * ex2((li - lamh[j0 + 15]) + (ll - laml[j0 + 15])) : 0.f;
#pragma unroll
                        for (int j = 0; j < 16; j += 4) {
                            const float4 g4 = *reinterpret_cast<const float4 *>(sg + j0 + j);
#pragma unroll
                            for (int e = 0; e < 4; ++e) gv[j + e] = left ? f * (&g4.x)[e] * gv[j + e] : 0.f;
                        }
                    }
                } else {
#pragma unroll
                    for (int j = 0; j < 16; ++j) gv[j] = 0.f;
                }
                if (is_k) {
                    keep_finite<16>(gv, i, slost);
#pragma unroll
                    for (int j = 0; j < 16; j += 4)
                        *reinterpret_cast<float4 *>(sA + i * kLd + j0 + j) = make_float4(gv[j], gv[j + 1], gv[j + 2], gv[j + 3]);
                } else {
#pragma unroll
                    for (int k = 0; k < 2; ++k) {
                        uint4 hi, lo;
                        split8(gv + 8 * k, hi, lo);
                        *reinterpret_cast<uint4 *>(sHi + sw128_chunk(row, 2 * blk + k, 128)) = hi;
                        *reinterpret_cast<uint4 *>(sLo + sw128_chunk(row, 2 * blk + k, 128)) = lo;
                    }
                }
            }
            __syncthreads();
            // T, diagonal blocks: thread (block, column).
            {
                const int d0 = tid & 48, j = tid & 15;
                float x[16];
                if (tid < kC) {
#pragma unroll
                    for (int r = 0; r < 16; ++r) {
                        float s = r == j ? 1.f : 0.f;
                        const float4 *ar = reinterpret_cast<const float4 *>(sA + (d0 + r) * kLd + d0);
#pragma unroll
                        for (int k = 0; k < r; k += 4) {
                            const float4 v = ar[k >> 2];
                            s = fmaf(-v.x, x[k], s);
                            if (k + 1 < r) s = fmaf(-v.y, x[k + 1], s);
                            if (k + 2 < r) s = fmaf(-v.z, x[k + 2], s);
                            if (k + 3 < r) s = fmaf(-v.w, x[k + 3], s);
                        }
                        x[r] = s;
                    }
                    __syncwarp();  // the warp's two blocks have been read
#pragma unroll
                    for (int r = 0; r < 16; ++r) sA[(d0 + r) * kLd + d0 + j] = x[r];
                }
            }
            __syncthreads();
            // T_21 = -T_22 (A_21 T_11) in A_21's place, the bracket kept above the diagonal: blocks of 16, then of 32.
            {
                const int d0 = 32 * (tid >> 7), r = (tid & 127) >> 3, c0 = (tid & 7) * 2;
#pragma unroll
                for (int pass = 0; pass < 2; ++pass) {
                    const float *lhs = sA + (d0 + 16 + r) * kLd + d0 + (pass ? 16 : 0);
                    const float *rhs = sA + d0 * kLd + d0 + (pass ? 16 : 0) + c0;
                    float2 s = make_float2(0.f, 0.f);
#pragma unroll
                    for (int k = 0; k < 16; k += 4) {
                        const float4 x = *reinterpret_cast<const float4 *>(lhs + k);
#pragma unroll
                        for (int e = 0; e < 4; ++e) {
                            const float2 y = *reinterpret_cast<const float2 *>(rhs + (k + e) * kLd);
                            s.x = fmaf((&x.x)[e], y.x, s.x);
                            s.y = fmaf((&x.x)[e], y.y, s.y);
                        }
                    }
                    if (pass) {
                        *reinterpret_cast<float2 *>(sA + (d0 + 16 + r) * kLd + d0 + c0) = make_float2(-s.x, -s.y);
                    } else {
                        keep_finite<2>(&s.x, d0 + 16 + r, slost);
                        *reinterpret_cast<float2 *>(sA + (d0 + r) * kLd + d0 + 16 + c0) = s;
                    }
                    __syncthreads();
                }
            }
            {
                // A warp has 4 columns, a lane a row: the right factor is the same address for all lanes.  Where T has
                // zeros above its diagonal blocks the array has brackets: they are passed over (the first product
                // starts at its columns' row, in the second the first 16 rows end at 16).
                const int c0 = 4 * warp;
#pragma unroll
                for (int pass = 0; pass < 2; ++pass) {
                    const float *lhs = sA + (32 + lane) * kLd + (pass ? 32 : 0);
                    const float *rhs = sA + (pass ? 32 : 0) + c0;
                    float4 s = make_float4(0.f, 0.f, 0.f, 0.f);
                    for (int k = pass ? 0 : c0; k < 32; k += 4) {
                        float4 x = *reinterpret_cast<const float4 *>(lhs + k);
                        if (pass && k >= 16 && lane < 16) x = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
                        for (int e = 0; e < 4; ++e) {
                            const float4 y = *reinterpret_cast<const float4 *>(rhs + (k + e) * kLd);
                            const float xe = (&x.x)[e];
                            s.x = fmaf(xe, y.x, s.x); s.y = fmaf(xe, y.y, s.y); s.z = fmaf(xe, y.z, s.z); s.w = fmaf(xe, y.w, s.w);
                        }
                    }
                    if (pass) {
                        *reinterpret_cast<float4 *>(sA + (32 + lane) * kLd + c0) = make_float4(-s.x, -s.y, -s.z, -s.w);
                    } else {
                        keep_finite<4>(&s.x, 32 + lane, slost);
                        *reinterpret_cast<float4 *>(sA + lane * kLd + 32 + c0) = s;
                    }
                    __syncthreads();
                }
            }
            // T diag(beta) as rows 0 .. 63 of the operand.
            {
                const int ti = tid & 63, q0 = (tid >> 6) * 16;
#pragma unroll
                for (int k = 0; k < 2; ++k) {
                    float v[8];
#pragma unroll
                    for (int j = 0; j < 8; j += 4) {
                        const float4 t4 = *reinterpret_cast<const float4 *>(sA + ti * kLd + q0 + 8 * k + j);
                        const float4 b4 = *reinterpret_cast<const float4 *>(sbeta + q0 + 8 * k + j);
#pragma unroll
                        for (int e = 0; e < 4; ++e) v[j + e] = q0 + 8 * k + j + e <= ti ? (&t4.x)[e] * (&b4.x)[e] : 0.f;
                    }
                    keep_finite<8>(v, ti, slost);
                    uint4 hi, lo;
                    split8(v, hi, lo);
                    *reinterpret_cast<uint4 *>(sHi + sw128_chunk(ti, (q0 >> 3) + k, 128)) = hi;
                    *reinterpret_cast<uint4 *>(sLo + sw128_chunk(ti, (q0 >> 3) + k, 128)) = lo;
                }
            }
            fence_async_smem();
            tc_fence_before();
            __syncthreads();
            tc_fence_after();
            // M (T diag(beta)): rows 64 .. 127 of the operand times its rows 0 .. 63, read as K x N.
            if (warp == 0 && elect_one()) {
                const uint32_t hi = sw128_desc_lo(smem_u32(sHi)), lo = hi + kTile / 16;
#pragma unroll
                for (int pr = 0; pr < 3; ++pr)
#pragma unroll
                    for (int ks = 0; ks < kC / 16; ++ks)
                        umma_bf16(tmem + kC, sw128_desc_of((pr == 2 ? lo : hi) + ks * 2), sw128_desc_of((pr == 1 ? lo : hi) + ks * 128),
                                  idesc_bf16_f32_mn(128, kC, false, true), pr > 0 || ks > 0);
                umma_commit(bar);
            }
            __syncwarp();
            failed = !bar_wait(bar, 1);
            failed = __syncthreads_or(failed);
            tc_fence_after();
            if (!failed) {
                if ((warp & 3) >= 2) {
#pragma unroll
                    for (int q = 0; q < 2; ++q) {
                        const int j0 = 32 * half + 16 * q;
                        float v[16];
                        tmem_ld16(base + kC + j0, v);
#pragma unroll
                        for (int k = 0; k < 2; ++k) {
                            uint4 hi, lo;
                            split8(v + 8 * k, hi, lo);
                            *reinterpret_cast<uint4 *>(sHi + sw128_chunk(row, (j0 >> 3) + k, 128)) = hi;
                            *reinterpret_cast<uint4 *>(sLo + sw128_chunk(row, (j0 >> 3) + k, 128)) = lo;
                        }
                    }
                }
                fence_async_smem();
                __syncthreads();
                if (tid == 0) {
                    *reinterpret_cast<int *>(a.ws + ((int64_t)slot * H + h) * kSlot + 2 * kTile + 512) = *slost;
                    bulk_s2g(a.ws + ((int64_t)slot * H + h) * kSlot, sHi, 2 * kTile);
                    asm volatile("cp.async.bulk.commit_group;" ::: "memory");
                    asm volatile("cp.async.bulk.wait_group.read 0;" ::: "memory");
                }
            }
        }
        if (failed && tid == 0) report_opt(a.err, DEV_PIPE_TIMEOUT, b, h, t0);
    }
    return failed;
}

// Between the two products the work is fp32 out of shared memory in short steps with barriers between them: four CTAs
// to an SM fill each other's waits, for which T takes A's place and the operand that of K and Q.  How many chunks there
// are is known on the device only: the CTAs share them out.
__global__ void __launch_bounds__(kChunkThreads, 4) gdn_chunk_kernel(const GdnPreArgs a) {
    using L = ChunkSmem;
    extern __shared__ __align__(1024) uint8_t raw[];
    uint8_t *sm = raw + ((1024 - (smem_u32(raw) & 1023)) & 1023);
    uint64_t *bar = reinterpret_cast<uint64_t *>(sm + L::kBar);
    uint32_t *tslot = reinterpret_cast<uint32_t *>(bar + 1);
    const int warp = threadIdx.x >> 5;
    pdl_wait();
    const int chunks = min(a.plan[kPlanChunks], a.slots), units = chunks * a.H;
    if ((int)blockIdx.x >= units) return;
    if (warp == 1) {
        tmem_alloc(tslot, 128);
        if (elect_one()) {
            mbar_init(bar, 1);
            mbar_init_fence();
        }
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    // The scan's CTAs may start (they read this kernel's results behind their own wait), once this one has its tensor
    // memory: one of them has all of an SM's.
    pdl_trigger();
    const uint32_t tmem = *tslot;
    for (int u = blockIdx.x; u < units; u += gridDim.x) {
        if (chunk_unit(a, sm, bar, reinterpret_cast<int *>(bar + 2), tmem, u % chunks, u / chunks)) break;
        tc_fence_before();
        __syncthreads();
        tc_fence_after();
    }
    tc_fence_before();
    __syncthreads();
    if (warp == 1) tmem_dealloc(tmem, 128);
}

// ---------------------------------------------------------------- scan over the chunks
// Everything is transposed, so that a tensor-memory lane is a state row p and a thread meets one row only: the
// state, the products Y^T = S [K; Q]^T and Z^T = R^T [T b; M T b]^T, and the left operands, which live in tensor
// memory too (bf16 pairs) and never pass through shared memory.  v and o are then read and written along p, whole
// lines at a time.
// Columns: S fp32 (128); Y^T of the K tokens, whose place Z^T of the K tokens and then (w U)^T take (16 tokens of it as
// 8 columns of hi and 8 of lo, which are the columns that the warps writing them have read); Y^T of the Q tokens; S hi
// and lo (128); Z^T of the Q tokens (64); R^T hi and lo (64).
// The chain from state to state is S -> Y_k -> R -> Z_k -> U -> S; what only the outputs need is issued behind it
// and read while the next chunk's first product runs.
constexpr uint32_t kTmS = 0, kTmY = 128, kTmA = 256, kTmZq = 384, kTmR = 448;
//
// Roles, each a set of warps, meeting on barriers in shared memory only:
//  16 chain warps   S, R and U of every chunk as operands: 4 a lane quarter, 32 state columns or 16 tokens each
//   4 output warps  the finished chunk's O
//   3 input warps   the next chunks' rows into shared memory
//   1 issuing warp  the products
struct ScanSmem {
    static constexpr int kKQ = 0;                     // [K; Q] 128 x 128 bf16, two buffers
    static constexpr int kOp = kKQ + 2 * 2 * kTile;   // [T b; M T b] hi, lo and the decays, two buffers
    static constexpr int kOpStep = 2 * kTile + 1024;
    static constexpr int kV = kOp + 2 * kOpStep;      // v [64 tokens][128 p] bf16, two buffers
    static constexpr int kO = kV + 2 * kC * 256;      // o [64 tokens][128 p] fp32
    static constexpr int kBar = kO + kC * 512;
    static constexpr int kLost = kBar + 144;  // first token of each state row that is lost to a value that is not finite
    static constexpr int kBytes = kLost + 512;
};
constexpr int kChainWarps = 16, kOutWarps = 4, kInWarps = 3;
constexpr int kFirstIn = kChainWarps + kOutWarps, kIssuer = kFirstIn + kInWarps;
constexpr int kScanThreads = 32 * (kIssuer + 1);
enum ScanBar {
    kBarYk, kBarZk, kBarS, kBarZq,  // products done (one phase a chunk)
    kBarPutS, kBarPutR, kBarPutU,   // operands in place (every chain warp arrives)
    kBarOut,                        // the output warps meet
    kBarO,                          // Y and Z of the Q tokens and the decays read (every output warp arrives)
    kBarIn,                         // a chunk's K, Q and v rows in shared memory, per buffer (every input warp arrives)
    kBarOp = kBarIn + 2,            // a chunk's matrix and decays, per buffer
    kBarEnd = kBarOp + 2,           // the state's way out (every chain warp arrives)
    kBarDrain,                      // everything issued, after a failure
    kBarN
};

__global__ void __launch_bounds__(kScanThreads, 1) gdn_scan_kernel(const GdnPreArgs a) {
    using L = ScanSmem;
    extern __shared__ __align__(1024) uint8_t raw[];
    uint8_t *sm = raw + ((1024 - (smem_u32(raw) & 1023)) & 1023);
    uint64_t *bar = reinterpret_cast<uint64_t *>(sm + L::kBar);
    uint32_t *tslot = reinterpret_cast<uint32_t *>(bar + kBarN);
    volatile int *sfail = reinterpret_cast<volatile int *>(tslot + 1);
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int slices = (a.P + 127) / 128, h = blockIdx.x / slices, p_base = (blockIdx.x % slices) * 128;
    const int H = a.H, P = a.P;
    const int p_here = min(128, P - p_base);  // state rows of this CTA
    pdl_trigger();  // the recurrence's CTAs, for the short requests, take what SMs this kernel leaves
    // The plan is complete: the chunk kernel lets this one start behind its own wait for it.  (Not through L1, which may
    // hold what the call before had there.)
    const int4 mine = __ldcg(gdn_order(a) + blockIdx.y);  // on its way while it is not known whether there is one
    if ((int)blockIdx.y >= __ldcg(a.plan + kPlanRequests)) {
        if (blockIdx.x == 0 && blockIdx.y == 0) pdl_wait();  // this kernel does not end before the chunk kernel has
        return;
    }
    const int b = mine.x, slot0 = mine.y, r0 = mine.z, r1 = mine.w, nchunks = (r1 - r0 + kC - 1) / kC;
    if ((int64_t)slot0 + nchunks > a.slots) {  // more chunks than these rows have: requests that overlap
        if (tid == 0) report_opt(a.err, DEV_BAD_LENGTHS, b, h, r1);
        return;
    }
    if (warp == 0) tmem_alloc(tslot, 512);
    if (tid == 0) {
        for (int i = 0; i < kBarN; ++i)
            mbar_init(bar + i, (i >= kBarPutS && i <= kBarPutU) || i == kBarEnd ? kChainWarps
                               : i == kBarOut || i == kBarO   ? kOutWarps
                               : i == kBarIn || i == kBarIn + 1 ? kInWarps : 1);
        *sfail = 0;
        mbar_init_fence();
    }
    volatile int *slost = reinterpret_cast<volatile int *>(sm + L::kLost);
    if (tid < 128) slost[tid] = 0x7fffffff;
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *tslot, base = tmem + ((uint32_t)(32 * (warp & 3)) << 16);
    const uint32_t smem0 = smem_u32(sm);
    const int64_t v_row = (int64_t)H * P;

    // Wait for a barrier's phase, a warp at a time; false, for every role, once any wait has run out.
    auto wait_for = [&](int which, int parity) {
        if (!warp_wait(bar + which, parity, sfail)) return false;
        tc_fence_after();
        return true;
    };
    // This warp's share is in place.
    auto arrive = [&](int which) {
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(bar + which);
    };

    if (warp < kChainWarps) {
        const int row = tid & 127, grp = tid >> 7;
        const uint32_t s_tm = base + kTmS + 32 * grp;  // S[p][32 grp ..]
        // The state in and out passes through shared memory: 32 lanes of a row each read whole lines, a lane a row
        // 32 of them for 16 bytes each.  Chunks of 16 bytes are exchanged by row so that neither side has conflicts.
        auto chain_meet = [] { asm volatile("bar.sync 2, %0;" ::"n"(32 * kChainWarps) : "memory"); };
        float *st = reinterpret_cast<float *>(sm + L::kO);  // [128 p][64 n] at a time
#pragma unroll 1
        for (int half = 0; half < 2; ++half) {
#pragma unroll
            for (int r = 0; r < 4; ++r) {
                const int pr = (tid >> 4) + 32 * r, ch = tid & 15;
                const bool live = a.S0 && pr < p_here;
                const float *src = a.S0 + ((((int64_t)b * H + h) * P + p_base + pr) * kDk + 64 * half + 4 * ch);
                cp_async16_or_zero(st + pr * 64 + 4 * (ch ^ (pr & 7)), live ? src : a.y, live);
            }
            cp_async_wait_all();
            chain_meet();
            if ((grp >> 1) == half) {
                float s[32];
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    const float4 x = *reinterpret_cast<const float4 *>(st + row * 64 + 4 * ((8 * (grp & 1) + j) ^ (row & 7)));
                    s[4 * j] = x.x; s[4 * j + 1] = x.y; s[4 * j + 2] = x.z; s[4 * j + 3] = x.w;
                }
                tmem_st32(s_tm, s);
            }
            chain_meet();
        }
        // 16 fp32 as 8 columns of hi and of lo.
        auto put16 = [&](const float *x, uint32_t hi_at, uint32_t lo_at) {
            alignas(16) uint32_t hi[8], lo[8];
            split8(x, *reinterpret_cast<uint4 *>(hi), *reinterpret_cast<uint4 *>(lo));
            split8(x + 8, *reinterpret_cast<uint4 *>(hi + 4), *reinterpret_cast<uint4 *>(lo + 4));
            tmem_st_u32(base + hi_at, hi);
            tmem_st_u32(base + lo_at, lo);
        };
        bool ok = true;
        for (int c = 0; c < nchunks; ++c) {
            const int par = c & 1;
            const float *dec = reinterpret_cast<const float *>(sm + L::kOp + par * L::kOpStep + 2 * kTile);
            // S at the chunk's start as (hi, lo), then 2^{Lam_C} S.
            // (It is read twice: values held over the barrier would be spilled, and what is spilled comes back from
            // L2, so little is left of L1.)
            if (c > 0 && !(ok = wait_for(kBarS, par ^ 1))) break;
            {
                float s[32];
                tmem_ld32(s_tm, s);
                put16(s, kTmA + 16 * grp, kTmA + 64 + 16 * grp);
                put16(s + 16, kTmA + 16 * grp + 8, kTmA + 64 + 16 * grp + 8);
            }
            tmem_st_wait();
            arrive(kBarPutS);
            if (!(ok = wait_for(kBarOp + par, (c >> 1) & 1))) break;
            {
                float s[32];
                const float d = dec[kC - 1];
                tmem_ld32(s_tm, s);
#pragma unroll
                for (int j = 0; j < 32; ++j) s[j] *= d;
                tmem_st32(s_tm, s);
            }
            // R^T = V^T - Y^T 2^Lam (behind the prompt v and K are zero, and so is this).
            if (!(ok = wait_for(kBarIn + par, (c >> 1) & 1))) break;
            float x[16], v[16];
            const uint16_t *vs = reinterpret_cast<const uint16_t *>(sm + L::kV + par * kC * 256) + 16 * grp * 128 + row;
#pragma unroll
            for (int j = 0; j < 16; ++j) v[j] = bf16_bits_to_float(vs[j * 128]);
            const int lost = reinterpret_cast<const int *>(dec)[2 * kC];  // first lost token of the chunk
            const bool losing = __any_sync(0xffffffffu, !all_finite<16>(v) || lost < kC);
            if (!(ok = wait_for(kBarYk, par))) break;
            tmem_ld16(base + kTmY + 16 * grp, x);
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                const float4 e = reinterpret_cast<const float4 *>(dec + 16 * grp)[k];
#pragma unroll
                for (int j = 0; j < 4; ++j) x[4 * k + j] = fmaf(-(&e.x)[j], x[4 * k + j], v[4 * k + j]);
            }
            if (losing) {
                int at = lost < kC ? lost : kC;
#pragma unroll
                for (int j = 15; j >= 0; --j)
                    if (!isfinite(v[j])) at = min(at, 16 * grp + j);
#pragma unroll
                for (int j = 0; j < 16; ++j) x[j] = 16 * grp + j >= at ? 0.f : x[j];
                if (at < kC) atomicMin(const_cast<int *>(slost) + row, kC * c + at);
                __syncwarp();
            }
            put16(x, kTmR + 8 * grp, kTmR + 32 + 8 * grp);
            tmem_st_wait();
            arrive(kBarPutR);
            if (!(ok = wait_for(kBarZk, par))) break;
            tmem_ld16(base + kTmY + 16 * grp, x);
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                const float4 w = reinterpret_cast<const float4 *>(dec + kC + 16 * grp)[k];
#pragma unroll
                for (int j = 0; j < 4; ++j) x[4 * k + j] *= (&w.x)[j];
            }
            put16(x, kTmY + 16 * grp, kTmY + 16 * grp + 8);
            tmem_st_wait();
            arrive(kBarPutU);
        }
        // All products are done, so that K's and Q's place is free.
        if (ok) ok = wait_for(kBarS, (nchunks - 1) & 1) && wait_for(kBarZq, (nchunks - 1) & 1);
        if (ok) {
            float s[32];
            tmem_ld32(s_tm, s);
            if (slost[row] != 0x7fffffff)
#pragma unroll
                for (int j = 0; j < 32; ++j) s[j] = NAN;
            st = reinterpret_cast<float *>(sm + L::kKQ);  // [128 p][128 n]
#pragma unroll
            for (int j = 0; j < 8; ++j)
                *reinterpret_cast<float4 *>(st + row * 128 + 4 * ((8 * grp + j) ^ (row & 7))) = make_float4(s[4 * j], s[4 * j + 1], s[4 * j + 2], s[4 * j + 3]);
            arrive(kBarEnd);
            ok = wait_for(kBarEnd, 0);
        }
        if (ok) {
            float *dst = a.S_out + (((int64_t)b * H + h) * P + p_base) * kDk + 4 * lane;
#pragma unroll
            for (int r = 0; r < 8; ++r) {
                const int pr = warp + 16 * r;
                if (pr < p_here) *reinterpret_cast<float4 *>(dst + pr * kDk) = *reinterpret_cast<const float4 *>(st + pr * 128 + 4 * (lane ^ (pr & 7)));
            }
        }
    } else if (warp < kFirstIn) {
        // v and o meet global memory in runs of 16 bytes a lane along p: a warp's accesses of 2 and 4 bytes a lane
        // took 1600 and 2500 cycles a chunk, a bulk copy a token about as long.
        const int ot = tid - 32 * kChainWarps;  // = tensor-memory lane = state row
        int meets = 0;
        auto meet = [&] {
            arrive(kBarOut);
            return wait_for(kBarOut, meets++ & 1);
        };
        float *so = reinterpret_cast<float *>(sm + L::kO);
        for (int c = 0; c < nchunks; ++c) {
            if (!wait_for(kBarOp + (c & 1), (c >> 1) & 1) || !wait_for(kBarZq, c & 1)) break;
            // O^T = 2^Lam (S q) + Z, to rows of p.
            const float4 *e = reinterpret_cast<const float4 *>(sm + L::kOp + (c & 1) * L::kOpStep + 2 * kTile);
#pragma unroll 1
            for (int i0 = 0; i0 < kC; i0 += 16) {
                float y[16], z[16];
                tmem_ld16(base + kTmY + kC + i0, y);
                tmem_ld16(base + kTmZq + i0, z);
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    const float4 d = e[(i0 >> 2) + k];
#pragma unroll
                    for (int j = 0; j < 4; ++j) so[(i0 + 4 * k + j) * 128 + ot] = fmaf((&d.x)[j], y[4 * k + j], z[4 * k + j]);
                }
            }
            arrive(kBarO);
            for (int t = max(0, slost[ot] - kC * c); t < kC; ++t) so[t * 128 + ot] = NAN;
            if (!meet()) break;
            const int t0 = r0 + c * kC, at = lane * 4;
            float *dst = a.y + (int64_t)t0 * v_row + (int64_t)h * P + p_base + at;
            if (at < p_here)
#pragma unroll 4
                for (int t = warp - kChainWarps; t < min(kC, r1 - t0); t += kOutWarps)
                    *reinterpret_cast<float4 *>(dst + t * v_row) = *reinterpret_cast<const float4 *>(so + t * 128 + at);
            if (!meet()) break;
        }
    } else if (warp < kIssuer) {
        // 64 rows of 256 bytes a chunk for each warp (K, Q or v), 16 lanes a row, two rows a copy.  Rows behind the
        // prompt and state rows behind P are zero.
        const int what = warp - kFirstIn, ch = lane & 15, r = lane >> 4;
        const int64_t step = 2 * (what == 2 ? v_row : (int64_t)H * kDk);
        const __nv_bfloat16 *first = reinterpret_cast<const __nv_bfloat16 *>(what == 2 ? a.v : what ? a.q : a.k) +
                                     (r0 + r) * (step / 2) + (what == 2 ? (int64_t)h * P + p_base : (int64_t)h * kDk) + 8 * ch;
        const bool cols = what < 2 || 8 * ch < p_here;
        // rows 8 apart lie 8 rows' bytes apart in either layout
        uint32_t dst[4];
#pragma unroll
        for (int u = 0; u < 4; ++u)
            dst[u] = what == 2 ? L::kV + 256 * (2 * u + r) + 16 * ch : L::kKQ + what * kC * 128 + sw128_chunk(2 * u + r, ch, 128);
        const uint32_t dst_step = what == 2 ? 2048 : 1024, dst_buf = what == 2 ? kC * 256 : 2 * kTile;
        auto load = [&](int cc) {
            const int n = cols ? r1 - (r0 + cc * kC) - r : 0;
            const __nv_bfloat16 *src = first + cc * (kC / 2) * step;
            uint8_t *to = sm + (cc & 1) * dst_buf;
#pragma unroll
            for (int i = 0; i < kC / 2; ++i) {
                cp_async16_or_zero(to + dst[i & 3] + (i >> 2) * dst_step, 2 * i < n ? src : first, 2 * i < n);
                src += step;
            }
        };
        if (warp == kFirstIn) pdl_wait();  // the chunk kernel's operands are there
        int copies = 0;
        for (int c = 0; c < nchunks; ++c) {
            if (c >= 2 && !wait_for(kBarZq, c & 1)) break;  // chunk c - 2's products are done
            load(c);
            if (c >= 2 && !wait_for(kBarO, c & 1)) break;   // and its decays read
            if (warp == kFirstIn && lane == 0) {
                uint64_t *br = bar + kBarOp + (c & 1);
                mbar_arrive_expect_tx(br, kSlot);
                bulk_g2s(sm + L::kOp + (c & 1) * L::kOpStep, a.ws + ((int64_t)(slot0 + c) * H + h) * kSlot, kSlot, br);
            }
            copies = c + 1;
            cp_async_wait_all();
            fence_async_smem();
            arrive(kBarIn + (c & 1));
        }
        cp_async_wait_all();
        if (warp == kFirstIn && warp_failed(sfail))  // copies that may still be in flight
            for (int c = max(0, copies - 2); c < copies; ++c) bar_wait(bar + kBarOp + (c & 1), (c >> 1) & 1);
    } else {
        const bool lead = elect_one();
        for (int c = 0; c < nchunks; ++c) {
            const int par = c & 1, use = (c >> 1) & 1;
            // descriptors: K (Q's rows lie 8192 bytes on) along its columns, K along its tokens, the matrix
            const uint32_t kq = sw128_desc_lo(smem0 + L::kKQ + par * 2 * kTile), kt = sw128_desc_lo(smem0 + L::kKQ + par * 2 * kTile, kTile);
            const uint32_t op = sw128_desc_lo(smem0 + L::kOp + par * L::kOpStep);
            auto y_products = [&](int q) {  // Y^T = S [K; Q]^T
#pragma unroll
                for (int hl = 0; hl < 2; ++hl)
#pragma unroll
                    for (int ks = 0; ks < kDk / 16; ++ks)
                        umma_ts(tmem + kTmY + q * kC, tmem + kTmA + 64 * hl + 8 * ks,
                                     sw128_desc_of(kq + (q * kC * 128 + (ks >> 2) * kTile + (ks & 3) * 32) / 16),
                                     idesc_bf16_f32(128, kC), hl > 0 || ks > 0);
            };
            auto z_products = [&](uint32_t d, int q) {  // Z^T = R^T [T b; M T b]^T
#pragma unroll
                for (int pr = 0; pr < 3; ++pr)
#pragma unroll
                    for (int ks = 0; ks < kC / 16; ++ks)
                        umma_ts(d, tmem + kTmR + (pr == 2 ? 32 : 0) + 8 * ks,
                                     sw128_desc_of(op + (q * kC * 128 + (pr == 1 ? kTile : 0) + ks * 32) / 16),
                                     idesc_bf16_f32(128, kC), pr > 0 || ks > 0);
            };
            if (!wait_for(kBarIn + par, use) || !wait_for(kBarPutS, par)) break;
            if (lead) {
                y_products(0);
                umma_commit(bar + kBarYk);
            }
            if (!wait_for(kBarOp + par, use) || !wait_for(kBarPutR, par)) break;
            if (lead) {
                z_products(tmem + kTmY, 0);
                umma_commit(bar + kBarZk);
            }
            if (c > 0 && !wait_for(kBarO, par ^ 1)) break;
            if (lead) y_products(1);
            if (!wait_for(kBarPutU, par)) break;
            if (lead) {
#pragma unroll
                for (int hl = 0; hl < 2; ++hl)  // S += (w U)^T K
#pragma unroll
                    for (int ks = 0; ks < kC / 16; ++ks)
                        umma_ts(tmem + kTmS, tmem + kTmY + 16 * ks + 8 * hl, sw128_desc_of(kt + ks * 2048 / 16),
                                     idesc_bf16_f32_mn(128, kDk, false, true), true);
                umma_commit(bar + kBarS);
                z_products(tmem + kTmZq, 1);
            }
            // The next chunk's rows are there, so that every input warp has seen the phase of kBarZq before this
            // one: no phase of it passes while someone waits for the one before.
            if (c + 1 < nchunks && !wait_for(kBarIn + (par ^ 1), ((c + 1) >> 1) & 1)) break;
            if (lead) umma_commit(bar + kBarZq);
        }
        if (warp_failed(sfail)) {  // products that may still run
            if (lead) umma_commit(bar + kBarDrain);
            __syncwarp();
            bar_wait(bar + kBarDrain, 0);
        }
    }
    tc_fence_before();
    __syncthreads();
    if (*sfail && tid == 0) report_opt(a.err, DEV_PIPE_TIMEOUT, b, h, 0);
    if (warp == 0) tmem_dealloc(tmem, 512);
}

constexpr int kChunkCtas = 4 * 148;  // as many as are resident

constexpr int kPlanThreads = 256;
__global__ void __launch_bounds__(kPlanThreads) gdn_plan_kernel(const GdnPreArgs a) {
    pdl_trigger();
    gdn_plan<kPlanThreads>(a);
}

// Chunks of requests that do not overlap: at most one more than their share of the rows for each that is not short.
int most_long(int B, int tokens) { return min(B, tokens / (kGdnShort + 1)); }
int64_t slots_of(int B, int tokens) { return (int64_t)tokens / kC + most_long(B, tokens); }
size_t plan_bytes(int B) { return ((kPlanOrder + 5 * (size_t)B) * sizeof(int32_t) + 255) / 256 * 256; }

}  // namespace

size_t gdn_chunk_bytes(int B, int H, int tokens) { return plan_bytes(B) + (size_t)(slots_of(B, tokens) * H) * kSlot; }

// Which requests are long is known on the device only, so that every kernel is launched and what it has no work for ends at
// once.  255 single tokens and one prompt of 2048: 326 us, of 254 and 125 apart (1249 by the recurrence alone); 64 single
// tokens in arrays of 1000 rows 92 (182 in chunks).  The price is paid where all are short: 64 x 1 token 76 us against 68 by
// the recurrence alone, 64 x 12 195 against 168, most of it the scan's CTAs, 1.1 us of an SM each to start and end.
cudaError_t gdn_chunk_launch(GdnPreArgs a, uint8_t *workspace, cudaStream_t st) {
    const int s1 = ChunkSmem::kBytes + 1024, s2 = ScanSmem::kBytes + 1024;
    cudaError_t e = cudaFuncSetAttribute(gdn_chunk_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, s1);
    if (e == cudaSuccess) e = cudaFuncSetAttribute(gdn_scan_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, s2);
    if (e != cudaSuccess) return e;
    a.slots = (int)slots_of(a.B, a.tokens);
    a.plan = reinterpret_cast<int32_t *>(workspace);
    a.ws = workspace + plan_bytes(a.B);
    const int64_t units = (int64_t)a.slots * a.H;
    gdn_plan_kernel<<<1, kPlanThreads, 0, st>>>(a);
    if ((e = cudaGetLastError()) != cudaSuccess) return e;
    e = launch_early(gdn_chunk_kernel, dim3((unsigned)min(units, (int64_t)kChunkCtas)), kChunkThreads, s1, a, st);
    if (e == cudaSuccess) e = launch_early(gdn_scan_kernel, dim3(a.H * ((a.P + 127) / 128), most_long(a.B, a.tokens)), kScanThreads, s2, a, st);
    return e == cudaSuccess ? gdn_recurrent_launch<__nv_bfloat16>(a, kDk, st) : e;
}

}  // namespace rssm
