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
// (request, head, 64 rows of the state) with three products a chunk, all with 128 rows:
//   [K; Q] S^T        (128 x 128 x 64: the K rows give R, the Q rows the first part of O)
//   [T b; M T b] R    (128 x 64 x 64:  the K rows give U, the Q rows the second part of O)
//   K^T (w U)         (128 x 64 x 64 onto the state, which stays in tensor memory, transposed)
// q, k and v are bf16 and enter exactly; fp32 operands enter as a (hi, lo) bf16 pair, which
// leaves 2^-17 of the value, and the lo lo product is dropped (2^-18): near-fp32 accuracy at
// two or three bf16 products, where one tf32 product would leave 2^-11.
//
// T comes from forward substitution in fp32, in blocks: the 16 x 16 diagonal blocks
// column by column, then T_21 = -T_22 A_21 T_11 twice.  (The product of I + (-A)^{2^i} is shorter
// and fails where keys repeat: the powers of A grow to 10^17 and cancel.)  Lam is summed in 64
// bits and kept as two fp32, so that a difference between neighbours is exact to fp32 however far
// down the chunk they are.
//
// Request b's chunk c has slot r0 / 64 + b + c (r0 its first row): slots do not collide, since
// floor((x + len) / 64) + 1 >= ceil(len / 64), and no prefix sum over the requests is needed.
#include <cuda_bf16.h>

#include "rssm_gdn_prefill.h"
#include "rssm_packed.cuh"
#include "rssm_umma.cuh"

namespace rssm {

namespace {

constexpr int kC = 64;                  // chunk
constexpr int kDk = 128;                // state columns (N)
constexpr int kPs = 64;                 // state rows a scan CTA owns
constexpr int kTile = 128 * kC * 2;     // [128 x 64] bf16
constexpr int kSlot = 2 * kTile + 512;  // hi, lo, then 2^Lam_i and 2^{Lam_C - Lam_i} fp32

__device__ __forceinline__ uint32_t bf2(__nv_bfloat16 a, __nv_bfloat16 b) {
    return (uint32_t)__bfloat16_as_ushort(a) | (uint32_t)__bfloat16_as_ushort(b) << 16;
}
// Eight fp32 values as 16-byte chunks of their (hi, lo) parts.
__device__ __forceinline__ void split8(const float *v, uint4 &hi, uint4 &lo) {
    uint32_t *ph = &hi.x, *pl = &lo.x;
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        __nv_bfloat16 h0, l0, h1, l1;
        split_bf16(v[2 * e], h0, l0);
        split_bf16(v[2 * e + 1], h1, l1);
        ph[e] = bf2(h0, h1);
        pl[e] = bf2(l0, l1);
    }
}
__device__ __forceinline__ void bulk_s2g(void *dst, const void *src, uint32_t bytes) {
    asm volatile("cp.async.bulk.global.shared::cta.bulk_group [%0], [%1], %2;" ::"l"(dst), "r"(smem_u32(src)), "r"(bytes)
                 : "memory");
}

// ---------------------------------------------------------------- chunk operands
constexpr int kLd = 68;  // fp32 row of A and T: 16-byte aligned, rows 4 banks apart
struct ChunkSmem {
    static constexpr int kKQ = 0;  // [K; Q] 128 x 128 bf16 in two column blocks; A and T afterwards
    static constexpr int kT = kKQ + 2 * kC * kLd * 4;
    static constexpr int kHi = (kT + 1023) / 1024 * 1024;
    static constexpr int kLo = kHi + kTile;
    static constexpr int kLam = kLo + kTile;  // Lam hi, Lam lo, beta
    static constexpr int kBar = kLam + 3 * kC * 4;
    static constexpr int kBytes = kBar + 32;
};
static_assert(2 * kC * kLd * 4 >= 2 * 128 * 128, "A and T overlay the K, Q tile");

__global__ void __launch_bounds__(128, 3) gdn_chunk_kernel(const GdnPreArgs a) {
    using L = ChunkSmem;
    extern __shared__ __align__(1024) uint8_t raw[];
    uint8_t *sm = raw + ((1024 - (smem_u32(raw) & 1023)) & 1023);
    uint8_t *sKQ = sm + L::kKQ, *sHi = sm + L::kHi, *sLo = sm + L::kLo;
    float *sA = reinterpret_cast<float *>(sm + L::kKQ), *sT = sA + kC * kLd;
    float *lamh = reinterpret_cast<float *>(sm + L::kLam), *laml = lamh + kC, *sbeta = laml + kC;
    uint64_t *bar = reinterpret_cast<uint64_t *>(sm + L::kBar);
    uint32_t *tslot = reinterpret_cast<uint32_t *>(bar + 1);
    int *sfound = reinterpret_cast<int *>(bar + 2);
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int slot = blockIdx.x, h = blockIdx.y, H = a.H;

    // The request of this slot: the last b with cu[b] / 64 + b <= slot, 32 candidates a round.
    if (warp == 0) {
        int lo = 0, n = a.B;  // b is in [lo, lo + n)
        while (n > 1) {
            const int step = (n + 31) / 32, at = lo + lane * step;
            const bool le = lane * step < n && (lane == 0 || a.cu[at] / kC + at <= slot);
            const int last = 31 - __clz(__ballot_sync(0xffffffffu, le));
            n = min(step, n - last * step);
            lo += last * step;
        }
        if (lane == 0) *sfound = lo;
        tmem_alloc(tslot, 128);
        if (lane == 0) {
            mbar_init(bar, 1);
            mbar_init_fence();
        }
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *tslot;
    const int b = *sfound;
    int r0, r1;
    const bool ok = packed_rows(a.cu, b, a.tokens, r0, r1);
    const int c = slot - (r0 / kC + b), t0 = r0 + c * kC;
    const bool work = ok && c >= 0 && t0 < r1;
    bool failed = false;
    if (work) {
        const int Lc = min(kC, r1 - t0);
        // K and Q rows, 16 lanes a row; rows behind the prompt are zero.
        for (int i = tid; i < 128 * 16; i += 128) {
            const int row = i >> 4, ch = i & 15, t = row & 63;
            uint8_t *dst = sKQ + sw128_chunk(row, ch, 128);
            const uint8_t *src = reinterpret_cast<const uint8_t *>(row < kC ? a.k : a.q) +
                                 (((int64_t)(t0 + t) * H + h) * kDk) * 2 + 16 * ch;
            if (t < Lc) cp_async16(dst, src);
            else *reinterpret_cast<uint4 *>(dst) = make_uint4(0, 0, 0, 0);
        }
        cp_async_commit();
        if (warp == 0) {
            // Lam: lane l has tokens 2l, 2l + 1.  A gate of 0 counts as 2^-200, which is 0 in every
            // fp32 product that it enters.
            double v[2];
            float be[2];
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                const int t = 2 * lane + e;
                const bool live = t < Lc;
                const float al = live ? a.alpha[(int64_t)(t0 + t) * H + h] : 1.f;
                be[e] = live ? a.beta[(int64_t)(t0 + t) * H + h] : 0.f;
                const float lg = log2f(al);
                v[e] = (double)(lg < -200.f ? -200.f : lg);
            }
            double x = v[0] + v[1];
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const double u = __shfl_up_sync(0xffffffffu, x, o);
                if (lane >= o) x += u;
            }
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                const double s = e ? x : x - v[1];
                lamh[2 * lane + e] = (float)s;
                laml[2 * lane + e] = (float)(s - (double)(float)s);
                sbeta[2 * lane + e] = be[e];
            }
        }
        cp_async_wait_all();
        fence_async_smem();
        __syncthreads();
        // G = [K; Q] K^T
        if (tid == 0) {
            const uint32_t at = smem_u32(sKQ);
            for (int ks = 0; ks < kDk / 16; ++ks)
                umma_bf16(tmem, sw128_desc(at, 128, ks), sw128_desc(at, 128, ks), idesc_bf16_f32(128, kC), ks > 0);
            umma_commit(bar);
        }
        const int i = tid & 63;
        const float li = lamh[i], ll = laml[i];
        if (tid < kC) {  // decays that the scan wants
            float *out = reinterpret_cast<float *>(a.ws + ((int64_t)slot * H + h) * kSlot + 2 * kTile);
            out[i] = exp2f(li + ll);
            out[kC + i] = exp2f((lamh[kC - 1] - li) + (laml[kC - 1] - ll));
        }
        __syncwarp();
        failed = !mbar_wait(bar, 0);
        failed = __syncthreads_or(failed);
        tc_fence_after();
        if (!failed) {
            // Row i of A (threads of K rows) or of M (Q rows): its lower triangle with decays.
            const uint32_t base = tmem + ((uint32_t)(32 * warp) << 16);
            const float bi = tid < kC ? sbeta[i] : 1.f;
            const int lim = tid < kC ? i : i + 1;  // columns below lim are kept
            const int warp_lim = 32 * (warp & 1) + 32;
#pragma unroll 1
            for (int j0 = 0; j0 < kC; j0 += 16) {
                float gv[16];
                if (j0 < warp_lim) {  // warp-uniform
                    tmem_ld16(base + j0, gv);
#pragma unroll
                    for (int j = 0; j < 16; ++j)
                        gv[j] = j0 + j < lim ? bi * exp2f((li - lamh[j0 + j]) + (ll - laml[j0 + j])) * gv[j] : 0.f;
                } else {
#pragma unroll
                    for (int j = 0; j < 16; ++j) gv[j] = 0.f;
                }
                if (tid < kC) {
#pragma unroll
                    for (int j = 0; j < 16; j += 4)
                        *reinterpret_cast<float4 *>(sA + i * kLd + j0 + j) = make_float4(gv[j], gv[j + 1], gv[j + 2], gv[j + 3]);
                } else {
#pragma unroll
                    for (int k = 0; k < 2; ++k) {
                        uint4 hi, lo;
                        split8(gv + 8 * k, hi, lo);
                        *reinterpret_cast<uint4 *>(sHi + sw128_chunk(tid, (j0 >> 3) + k, 128)) = hi;
                        *reinterpret_cast<uint4 *>(sLo + sw128_chunk(tid, (j0 >> 3) + k, 128)) = lo;
                    }
                }
            }
            __syncthreads();
            // T, diagonal blocks: thread (block, column).  The other threads clear the blocks above them.
            if (tid < kC) {
                const int d0 = tid & ~15, j = tid & 15;
                float x[16];
#pragma unroll
                for (int r = 0; r < 16; ++r) {
                    float s = r == j ? 1.f : 0.f;
#pragma unroll
                    for (int k = 0; k < r; ++k) s = fmaf(-sA[(d0 + r) * kLd + d0 + k], x[k], s);
                    x[r] = s;
                    sT[(d0 + r) * kLd + d0 + j] = s;
                }
            } else {
                const int r = (tid - kC) >> 1, col = ((tid - kC) & 1) * 8;  // 32 rows: 0-15 and 32-47
                const int row = (r & 15) + 32 * (r >> 4);
#pragma unroll
                for (int e = 0; e < 8; e += 4)
                    *reinterpret_cast<float4 *>(sT + row * kLd + 32 * (r >> 4) + 16 + col + e) = make_float4(0.f, 0.f, 0.f, 0.f);
            }
            __syncthreads();
            // T_21 = -T_22 (A_21 T_11), the bracket kept above A's diagonal: blocks of 16, then of 32.
            {
                const int d0 = 32 * (tid >> 6), r = (tid & 63) >> 2, c0 = (tid & 3) * 4;
#pragma unroll
                for (int pass = 0; pass < 2; ++pass) {
                    const float *lhs = (pass ? sT + (d0 + 16 + r) * kLd + d0 + 16 : sA + (d0 + 16 + r) * kLd + d0);
                    const float *rhs = (pass ? sA + d0 * kLd + d0 + 16 : sT + d0 * kLd + d0) + c0;
                    float4 s = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 4
                    for (int k = 0; k < 16; ++k) {
                        const float x = lhs[k];
                        const float4 y = *reinterpret_cast<const float4 *>(rhs + k * kLd);
                        s.x = fmaf(x, y.x, s.x); s.y = fmaf(x, y.y, s.y); s.z = fmaf(x, y.z, s.z); s.w = fmaf(x, y.w, s.w);
                    }
                    if (pass) *reinterpret_cast<float4 *>(sT + (d0 + 16 + r) * kLd + d0 + c0) = make_float4(-s.x, -s.y, -s.z, -s.w);
                    else *reinterpret_cast<float4 *>(sA + (d0 + r) * kLd + d0 + 16 + c0) = s;
                    __syncthreads();
                }
            }
            {
                const int r = tid >> 2, c0 = (tid & 3) * 8;
#pragma unroll
                for (int pass = 0; pass < 2; ++pass) {
                    const float *lhs = pass ? sT + (32 + r) * kLd + 32 : sA + (32 + r) * kLd;
                    const float *rhs = (pass ? sA + 32 : sT) + c0;
                    float s[8] = {};
#pragma unroll 4
                    for (int k = 0; k < 32; ++k) {
                        const float x = lhs[k];
#pragma unroll
                        for (int e = 0; e < 8; e += 4) {
                            const float4 y = *reinterpret_cast<const float4 *>(rhs + k * kLd + e);
                            s[e] = fmaf(x, y.x, s[e]); s[e + 1] = fmaf(x, y.y, s[e + 1]);
                            s[e + 2] = fmaf(x, y.z, s[e + 2]); s[e + 3] = fmaf(x, y.w, s[e + 3]);
                        }
                    }
                    float *dst = pass ? sT + (32 + r) * kLd + c0 : sA + r * kLd + 32 + c0;
                    const float sg = pass ? -1.f : 1.f;
#pragma unroll
                    for (int e = 0; e < 8; e += 4)
                        *reinterpret_cast<float4 *>(dst + e) = make_float4(sg * s[e], sg * s[e + 1], sg * s[e + 2], sg * s[e + 3]);
                    __syncthreads();
                }
            }
            // T diag(beta) as rows 0 .. 63 of the operand.
            {
                const int half = (tid >> 6) * 32;
#pragma unroll 1
                for (int j0 = half; j0 < half + 32; j0 += 8) {
                    float v[8];
#pragma unroll
                    for (int j = 0; j < 8; ++j) v[j] = j0 + j <= i ? sT[i * kLd + j0 + j] * sbeta[j0 + j] : 0.f;
                    uint4 hi, lo;
                    split8(v, hi, lo);
                    *reinterpret_cast<uint4 *>(sHi + sw128_chunk(i, j0 >> 3, 128)) = hi;
                    *reinterpret_cast<uint4 *>(sLo + sw128_chunk(i, j0 >> 3, 128)) = lo;
                }
            }
            fence_async_smem();
            tc_fence_before();
            __syncthreads();
            tc_fence_after();
            // M (T diag(beta)): rows 64 .. 127 of the operand times its rows 0 .. 63, read as K x N.
            if (tid == 0) {
                const uint32_t hi = smem_u32(sHi), lo = smem_u32(sLo);
                for (int pr = 0; pr < 3; ++pr) {
                    const uint32_t A = pr == 2 ? lo : hi, B = pr == 1 ? lo : hi;
                    for (int ks = 0; ks < kC / 16; ++ks)
                        umma_bf16(tmem + kC, sw128_desc(A, 128, ks), sw128_mn_desc(B, 1024, ks),
                                  idesc_bf16_f32_mn(128, kC, false, true), pr > 0 || ks > 0);
                }
                umma_commit(bar);
            }
            __syncwarp();
            failed = !mbar_wait(bar, 1);
            failed = __syncthreads_or(failed);
            tc_fence_after();
            if (!failed) {
                if (warp >= 2) {
#pragma unroll 1
                    for (int j0 = 0; j0 < kC; j0 += 16) {
                        float v[16];
                        tmem_ld16(base + kC + j0, v);
#pragma unroll
                        for (int k = 0; k < 2; ++k) {
                            uint4 hi, lo;
                            split8(v + 8 * k, hi, lo);
                            *reinterpret_cast<uint4 *>(sHi + sw128_chunk(tid, (j0 >> 3) + k, 128)) = hi;
                            *reinterpret_cast<uint4 *>(sLo + sw128_chunk(tid, (j0 >> 3) + k, 128)) = lo;
                        }
                    }
                }
                fence_async_smem();
                __syncthreads();
                if (tid == 0) {
                    bulk_s2g(a.ws + ((int64_t)slot * H + h) * kSlot, sHi, 2 * kTile);
                    asm volatile("cp.async.bulk.commit_group;" ::: "memory");
                    asm volatile("cp.async.bulk.wait_group 0;" ::: "memory");
                }
            }
        }
        if (failed && tid == 0) report_opt(a.err, DEV_PIPE_TIMEOUT, b, h, t0);
    }
    tc_fence_before();
    __syncthreads();
    if (warp == 0) tmem_dealloc(tmem, 128);
}

// ---------------------------------------------------------------- scan over the chunks
struct ScanSmem {
    static constexpr int kKQ = 0;                 // [K; Q] 128 x 128 bf16
    static constexpr int kOp = kKQ + 2 * kTile;   // [T b; M T b] hi, lo, then the decays
    static constexpr int kDec = kOp + 2 * kTile;
    static constexpr int kS = kDec + 1024;        // S hi, lo [128 n][64 p]; then R hi, lo and w U hi, lo [64 j][64 p]
    static constexpr int kBar = kS + 2 * kTile;
    static constexpr int kBytes = kBar + 32;
};
constexpr int kRTile = kC * kPs * 2;  // one part of R or w U
constexpr int kScanThreads = 256;

__global__ void __launch_bounds__(kScanThreads, 2) gdn_scan_kernel(const GdnPreArgs a) {
    using L = ScanSmem;
    extern __shared__ __align__(1024) uint8_t raw[];
    uint8_t *sm = raw + ((1024 - (smem_u32(raw) & 1023)) & 1023);
    uint8_t *sKQ = sm + L::kKQ, *sOp = sm + L::kOp, *sS = sm + L::kS;
    float *dec = reinterpret_cast<float *>(sm + L::kDec);  // 2^Lam_i, then 2^{Lam_C - Lam_i}
    uint64_t *bar = reinterpret_cast<uint64_t *>(sm + L::kBar);
    uint32_t *tslot = reinterpret_cast<uint32_t *>(bar + 2);
    const int tid = threadIdx.x, warp = tid >> 5;
    const int row = tid & 127;               // tensor-memory lane: token (K rows, Q rows) or state column n
    const int pl = (tid >> 7) * (kPs / 2);   // this thread's 32 of the CTA's 64 state rows
    const int slices = a.P / kPs, h = blockIdx.x / slices, p0 = (blockIdx.x % slices) * kPs, b = blockIdx.y, H = a.H;
    int r0, r1;
    if (!packed_rows(a.cu, b, a.tokens, r0, r1)) {
        if (tid == 0) report_opt(a.err, DEV_BAD_LENGTHS, b, h, r1);
        return;
    }
    const int64_t head = (int64_t)b * H + h;
    if (warp == 0) tmem_alloc(tslot, 256);
    if (tid == 0) {
        mbar_init(bar, 1);
        mbar_init_fence();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *tslot, base = tmem + ((uint32_t)(32 * (warp & 3)) << 16);
    const uint32_t cY = 0, cZ = kPs, cS = 2 * kPs;
    const int nchunks = (r1 - r0 + kC - 1) / kC;
    const uint8_t *ws = a.ws + ((int64_t)(r0 / kC + b) * H + h) * kSlot;
    const int64_t ws_step = (int64_t)H * kSlot;

    // Parts of the next chunk's operands: K rows, Q rows, the matrix and decays.
    auto load_rows = [&](int cc, bool q) {
        const int t0 = r0 + cc * kC, Lc = min(kC, r1 - t0);
        const uint8_t *src = reinterpret_cast<const uint8_t *>(q ? a.q : a.k);
        for (int i = tid; i < kC * 16; i += kScanThreads) {
            const int t = i >> 4, ch = i & 15;
            uint8_t *dst = sKQ + sw128_chunk(q ? kC + t : t, ch, 128);
            if (t < Lc) cp_async16(dst, src + (((int64_t)(t0 + t) * H + h) * kDk) * 2 + 16 * ch);
            else *reinterpret_cast<uint4 *>(dst) = make_uint4(0, 0, 0, 0);
        }
    };
    auto load_op = [&](int cc) {
        const uint8_t *src = ws + cc * ws_step;
        for (int i = tid; i < kSlot / 16; i += kScanThreads) cp_async16(sOp + 16 * i, src + 16 * i);
    };
    uint4 vreg[4];  // v of this thread's token and 32 state rows (threads of K rows)
    auto load_v = [&](int cc) {
        const int t = r0 + cc * kC + row;
        const bool live = row < kC && t < r1;
        const uint4 *src = reinterpret_cast<const uint4 *>(reinterpret_cast<const __nv_bfloat16 *>(a.v) +
                                                           ((int64_t)t * H + h) * a.P + p0 + pl);
#pragma unroll
        for (int k = 0; k < 4; ++k) vreg[k] = live ? src[k] : make_uint4(0, 0, 0, 0);
    };

    float s[32];  // S^T[n = row][pl ..]
#pragma unroll
    for (int j = 0; j < 32; ++j) s[j] = a.S0 ? a.S0[(head * a.P + p0 + pl + j) * kDk + row] : 0.f;
    if (nchunks > 0) {
        load_rows(0, false);
        load_rows(0, true);
        load_op(0);
        load_v(0);
    }
    cp_async_commit();

    uint32_t phase = 0;
    bool failed = false;
    // All of the CTA's writes are visible to the tensor cores; thread 0 then issues.
    auto ready = [&]() {
        fence_async_smem();
        tc_fence_before();
        __syncthreads();
        tc_fence_after();
    };
    auto wait_mma = [&]() {
        __syncwarp();
        if (!mbar_wait(bar, phase & 1)) failed = true;
        ++phase;
        failed = __syncthreads_or(failed);
        tc_fence_after();
        return !failed;
    };
    for (int c = 0; c < nchunks; ++c) {
        const int t0 = r0 + c * kC;
        // S at the chunk's start as (hi, lo), and 2^{Lam_C} S into tensor memory.
        if (c > 0) tmem_ld32(base + cS + pl, s);
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            uint4 hi, lo;
            split8(s + 8 * k, hi, lo);
            const uint32_t off = sw128_chunk(row, (pl >> 3) + k, 128);
            *reinterpret_cast<uint4 *>(sS + off) = hi;
            *reinterpret_cast<uint4 *>(sS + kTile + off) = lo;
        }
        cp_async_wait_all();
        ready();
        if (tid == 0) {
            const uint32_t kq = smem_u32(sKQ);
            for (int hl = 0; hl < 2; ++hl)
                for (int ks = 0; ks < kDk / 16; ++ks)
                    umma_bf16(tmem + cY, sw128_desc(kq, 128, ks), sw128_mn_desc(smem_u32(sS) + hl * kTile, 1024, ks),
                              idesc_bf16_f32_mn(128, kPs, false, true), hl > 0 || ks > 0);
            umma_commit(bar);
        }
        {
            const float d = dec[kC - 1];
#pragma unroll
            for (int j = 0; j < 32; ++j) s[j] *= d;
            tmem_st32(base + cS + pl, s);
        }
        const float di = dec[row & 63];
        if (!wait_mma()) break;
        // R = V - 2^Lam (K S^T), over S's place (its product has completed).
        float yv[32];
        tmem_ld32(base + cY + pl, yv);
        if (row < kC) {
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                float r[8];
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    const uint32_t w = (&vreg[k].x)[e >> 1];
                    r[e] = fmaf(-di, yv[8 * k + e], bf16_bits_to_float((e & 1) ? w >> 16 : w & 0xffff));
                }
                uint4 hi, lo;
                split8(r, hi, lo);
                const uint32_t off = sw128_chunk(row, (pl >> 3) + k, kC);
                *reinterpret_cast<uint4 *>(sS + off) = hi;
                *reinterpret_cast<uint4 *>(sS + kRTile + off) = lo;
            }
        }
        ready();
        if (tid == 0) {
            const uint32_t op = smem_u32(sOp), r = smem_u32(sS);
            for (int pr = 0; pr < 3; ++pr)
                for (int ks = 0; ks < kC / 16; ++ks)
                    umma_bf16(tmem + cZ, sw128_desc(op + (pr == 2 ? kTile : 0), 128, ks),
                              sw128_mn_desc(r + (pr == 1 ? kRTile : 0), 1024, ks),
                              idesc_bf16_f32_mn(128, kPs, false, true), pr > 0 || ks > 0);
            umma_commit(bar);
        }
        if (c + 1 < nchunks) {
            load_rows(c + 1, true);  // Q's rows are done with
            load_v(c + 1);
        }
        const float wi = dec[kC + (row & 63)];
        if (!wait_mma()) break;
        float zv[32];
        tmem_ld32(base + cZ + pl, zv);
        if (row < kC) {  // w U
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                float u[8];
#pragma unroll
                for (int e = 0; e < 8; ++e) u[e] = wi * zv[8 * k + e];
                uint4 hi, lo;
                split8(u, hi, lo);
                const uint32_t off = sw128_chunk(row, (pl >> 3) + k, kC);
                *reinterpret_cast<uint4 *>(sS + kTile + off) = hi;
                *reinterpret_cast<uint4 *>(sS + kTile + kRTile + off) = lo;
            }
        }
        ready();
        if (tid == 0) {
            const uint32_t kq = smem_u32(sKQ), u = smem_u32(sS) + kTile;
            for (int hl = 0; hl < 2; ++hl)
                for (int ks = 0; ks < kC / 16; ++ks)
                    umma_bf16(tmem + cS, sw128_mn_desc(kq, kTile, ks), sw128_mn_desc(u + hl * kRTile, 1024, ks),
                              idesc_bf16_f32_mn(128, kPs, true, true), true);
            umma_commit(bar);
        }
        if (row >= kC) {  // O
            const int t = t0 + row - kC;
            if (t < r1) {
                float4 *dst = reinterpret_cast<float4 *>(a.y + ((int64_t)t * H + h) * a.P + p0 + pl);
#pragma unroll
                for (int k = 0; k < 8; ++k)
                    dst[k] = make_float4(fmaf(di, yv[4 * k], zv[4 * k]), fmaf(di, yv[4 * k + 1], zv[4 * k + 1]),
                                         fmaf(di, yv[4 * k + 2], zv[4 * k + 2]), fmaf(di, yv[4 * k + 3], zv[4 * k + 3]));
            }
        }
        if (c + 1 < nchunks) load_op(c + 1);
        if (!wait_mma()) break;
        if (c + 1 < nchunks) load_rows(c + 1, false);
    }
    cp_async_wait_all();
    if (failed) {
        if (tid == 0) report_opt(a.err, DEV_PIPE_TIMEOUT, b, h, 0);
    } else {
        if (nchunks > 0) tmem_ld32(base + cS + pl, s);
#pragma unroll
        for (int j = 0; j < 32; ++j) a.S_out[(head * a.P + p0 + pl + j) * kDk + row] = s[j];
    }
    tc_fence_before();
    __syncthreads();
    if (warp == 0) tmem_dealloc(tmem, 256);
}

int64_t slots(int B, int tokens) { return (int64_t)tokens / kC + B + 1; }

}  // namespace

size_t gdn_chunk_bytes(int B, int H, int tokens) { return (size_t)(slots(B, tokens) * H) * kSlot; }

cudaError_t gdn_chunk_launch(const GdnPreArgs &a, cudaStream_t st) {
    const int s1 = ChunkSmem::kBytes + 1024, s2 = ScanSmem::kBytes + 1024;
    cudaError_t e = cudaFuncSetAttribute(gdn_chunk_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, s1);
    if (e == cudaSuccess) e = cudaFuncSetAttribute(gdn_scan_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, s2);
    if (e != cudaSuccess) return e;
    gdn_chunk_kernel<<<dim3((unsigned)slots(a.B, a.tokens), a.H), 128, s1, st>>>(a);
    if ((e = cudaGetLastError()) != cudaSuccess) return e;
    gdn_scan_kernel<<<dim3(a.H * (a.P / kPs), a.B), kScanThreads, s2, st>>>(a);
    return cudaGetLastError();
}

}  // namespace rssm
