// rssm_kv4_attend_tiles.cu -- attention over the paged 4-bit cache for many query rows (a prompt chunk, the drafts of
// wide groups): tiles of 128 rows by 128 tokens on the 5th-generation tensor cores.
//
// With few rows what counts is that codes become operands inside a thread (rssm_kv4_attend.cu); with many, a widened
// tile serves 128 rows, and the products decide.  Per tile of 128 tokens:
//   S = Q K^T     128 x 128 x D   Q and K fp16 in shared memory
//   O += P V      128 x D x 128   P fp16 in tensor memory, in S's place; V as stored, read token by token
// One thread has one row, so that its maximum and sum need no exchange; tokens go to two streams by turns, each with S,
// O, maximum and sum of its own, so that one's softmax runs beside the other's products, and the two are joined at the
// end.  The exponentials (16 a cycle and SM) and the products (2 x 512 cycles a tile at D = 128) are both near 1000
// cycles a tile, and the rest of the work is laid beside them on warps of their own.
//
// Roles: 8 softmax warps (4 a stream), 4 widening warps (one token a thread, the next tile's bytes in registers ahead),
// 1 issuing warp.  They meet on barriers in shared memory; every wait is bounded.
#include <math.h>

#include "rssm_internal.h"
#include "rssm_kv4_attend.cuh"
#include "rssm_umma.cuh"

namespace rssm {

namespace {

constexpr int kSoftWarps = 8, kWideWarps = 4;
constexpr int kWide0 = kSoftWarps, kTilesIssuer = kSoftWarps + kWideWarps;
constexpr int kTilesThreads = 32 * (kTilesIssuer + 1);
enum TilesBar {
    kBarK = 0,    // K tile written, per stream (every widening warp)
    kBarVt = 2,   // V tile written
    kBarQ = 4,    // Q written (the four warps that write it)
    kBarSc = 5,   // S done, per stream
    kBarP = 7,    // P written, per stream (its four warps)
    kBarPv = 9,   // O updated, per stream
    kBarMl = 11,  // maxima and sums written (every softmax warp)
    kBarJoin = 12,  // the second stream's O written (its four warps)
    kBarDrain = 13,
    kTilesBars = 14
};

template <int D> struct TilesSmem {
    static constexpr int kTileB = 128 * D * 2;
    static constexpr int kQ = 0, kKt = kTileB, kVt = 3 * kTileB;  // K and V: one tile a stream each
    static constexpr int kOut = kKt;                                // the second stream's O, fp32 rows of D + 4
    static constexpr int kMl = 5 * kTileB;                          // (m, l) [2][128]
    static constexpr int kNan = kMl + 2 * 128 * 8;                  // first token with a NaN value, per block of 16 channels
    static constexpr int kGone = kNan + 8 * 4;                      // tokens whose page is not there, a bit each: [tile mod 4][4]
    static constexpr int kBar = kGone + 4 * 16;
    static constexpr int kBytes = kBar + kTilesBars * 8 + 16;
    static_assert(128 * (D + 4) * 4 <= 4 * kTileB, "O overlays the K and V tiles");
};

template <int D>
__global__ void __launch_bounds__(kTilesThreads, 1) attend_tiles_kernel(const AttendArgs a) {
    using L = TilesSmem<D>;
    constexpr uint32_t kTmO = 256;  // tensor memory: S (then P) of the streams at 0 and 128, O at 256 and 256 + D
    extern __shared__ __align__(1024) uint8_t raw[];
    uint8_t *sm = raw + ((1024 - (smem_u32(raw) & 1023)) & 1023);
    uint64_t *bar = reinterpret_cast<uint64_t *>(sm + L::kBar);
    uint32_t *tslot = reinterpret_cast<uint32_t *>(bar + kTilesBars);
    volatile int *sfail = reinterpret_cast<volatile int *>(tslot + 1);
    float2 *sml = reinterpret_cast<float2 *>(sm + L::kMl);
    int *snan = reinterpret_cast<int *>(sm + L::kNan);
    uint32_t *sgone = reinterpret_cast<uint32_t *>(sm + L::kGone);
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int split = blockIdx.x, tile = blockIdx.y % a.tiles, h = blockIdx.y / a.tiles, b = blockIdx.z;
    const int ps = a.kv.ps, G = a.G;
    if (a.splits > 1) pdl_trigger();  // the joining kernel's CTAs may start, up to their wait
    int r0, n, len;
    if (!attend_request(a, b, r0, n, len)) {
        if (tid == 0) report_opt(a.err, DEV_BAD_LENGTHS, b, 0, len);
        return;
    }
    const int rows = n * G, row0 = tile * 128;
    if (row0 >= rows) return;
    const int last = min(row0 + 128, rows) - 1;
    const int tlen = max(0, len - n + last / G + 1);  // tokens that the tile's last row sees
    const int ns = max(1, (tlen + a.L - 1) / a.L);
    if (split >= ns) return;
    const int t_begin = split * a.L, t_end = min(tlen, t_begin + a.L);
    const int ntiles = (t_end - t_begin + 127) / 128;

    if (warp == 0) tmem_alloc(tslot, 512);
    if (tid == 0) {
        for (int i = 0; i < kTilesBars; ++i)
            mbar_init(bar + i, i < kBarQ ? kWideWarps : i == kBarQ || i == kBarP || i == kBarP + 1 || i == kBarJoin ? 4 : i == kBarMl ? 8 : 1);
        for (int i = 0; i < 8; ++i) snan[i] = 0x7fffffff;
        *sfail = 0;
        mbar_init_fence();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *tslot, base = tmem + ((uint32_t)(32 * (warp & 3)) << 16);
    // Wait for a barrier's phase; false, for every role, once any wait has run out.
    auto wait_for = [&](int which, int parity) {
        if (!bar_try(bar + which, parity)) {
            const long long t0 = clock64();
            while (!bar_try(bar + which, parity))
                if (*sfail || clock64() - t0 > kWaitCycles) {
                    *sfail = 1;
                    return false;
                }
        }
        tc_fence_after();
        return true;
    };
    auto arrive = [&](int which) {
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(bar + which);
    };

    if (warp < kSoftWarps) {
        const int row = tid & 127, st = tid >> 7, grow = row0 + row;
        const bool live = grow < rows;
        const int i = live ? grow / G : 0, hd = live ? grow - i * G : 0;
        const int seen = live ? len - n + i + 1 : 0;
        const int64_t q_at = ((int64_t)(r0 + i) * a.Hq + h * G + hd) * D;
        float f;
        {
            // This row of Q, scaled by a power of two (see rssm_kv4_attend.cu); the first stream's threads write it.
            const uint4 *src = reinterpret_cast<const uint4 *>(a.q + q_at);
            float top = 0.f;
#pragma unroll 4
            for (int k = 0; k < D / 8; ++k) {
                const uint4 v = live ? src[k] : make_uint4(0, 0, 0, 0);
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const uint32_t x = (&v.x)[e];
                    top = fmaxf(top, fmaxf(fabsf(bf16_bits_to_float(x & 0xffff)), fabsf(bf16_bits_to_float(x >> 16))));
                }
            }
            const int ex = row_exponent(top);
            const float s0 = copysignf(pow2f(-(ex / 2)), a.scale);
            const float s1 = a.scale == 0.f ? 0.f : pow2f(-(ex - ex / 2));
            f = fmaxf(fabsf(a.scale) * pow2f(ex / 2) * pow2f(ex - ex / 2), 1.2e-38f);
            if (st == 0) {
#pragma unroll 4
                for (int k = 0; k < D / 8; ++k) {
                    const uint4 v = live ? src[k] : make_uint4(0, 0, 0, 0);
                    uint4 w;
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        const uint32_t x = (&v.x)[e];
                        (&w.x)[e] = f16x2(bf16_bits_to_float(x & 0xffff) * s0 * s1, bf16_bits_to_float(x >> 16) * s0 * s1);
                    }
                    *reinterpret_cast<uint4 *>(sm + L::kQ + sw128_chunk(row, k, 128)) = w;
                }
                fence_async_smem();
                arrive(kBarQ);
            }
        }
        const uint32_t s_tm = base + 128 * st, o_tm = base + kTmO + D * st;
        float m = -INFINITY, l = 0.f;
        bool ok = true;
        for (int j = st; j < ntiles; j += 2) {
            const int k = j >> 1, t0 = t_begin + 128 * j;
            if (!(ok = wait_for(kBarSc + st, k & 1))) break;
            const int lim = min(seen, t_end) - t0;  // columns below lim are seen
            const uint32_t *gone = sgone + 4 * (j & 3);
            const bool edge = __any_sync(0xffffffffu, lim < 128) || (gone[0] | gone[1] | gone[2] | gone[3]);
            float top = -INFINITY;
#pragma unroll 1
            for (int c = 0; c < 128; c += 32) {
                float x[32];
                tmem_ld32(s_tm + c, x);
                if (edge) {
                    const uint32_t gw = gone[c >> 5];
#pragma unroll
                    for (int e = 0; e < 32; ++e)
                        if (c + e >= lim || (gw >> e & 1)) x[e] = -INFINITY;
                }
#pragma unroll
                for (int e = 0; e < 32; ++e) top = fmaxf(top, x[e]);
            }
            top *= f;
            if (__any_sync(0xffffffffu, top > m + kLag)) {
                const float mn = fmaxf(m, top), fac = mn == -INFINITY ? 1.f : ex2(m - mn);
                l *= fac;
                m = mn;
                if (k > 0) {
                    if (!(ok = wait_for(kBarPv + st, (k - 1) & 1))) break;
#pragma unroll 1
                    for (int c = 0; c < D; c += 32) {
                        float x[32];
                        tmem_ld32(o_tm + c, x);
#pragma unroll
                        for (int e = 0; e < 32; ++e) x[e] *= fac;
                        tmem_st32(o_tm + c, x);
                    }
                }
            }
            const float off = m == -INFINITY ? 0.f : m;  // a row that has seen nothing yet keeps p = 2^-inf = 0
#pragma unroll 1
            for (int c = 0; c < 128; c += 32) {
                float x[32];
                uint32_t w[16];
                tmem_ld32(s_tm + c, x);
                if (edge) {
                    const uint32_t gw = gone[c >> 5];
#pragma unroll
                    for (int e = 0; e < 32; ++e)
                        if (c + e >= lim || (gw >> e & 1)) x[e] = -INFINITY;
                }
#pragma unroll
                for (int e = 0; e < 32; ++e) {
                    x[e] = ex2(fmaf(x[e], f, -off));
                    l += x[e];
                }
#pragma unroll
                for (int e = 0; e < 16; ++e) w[e] = f16x2(x[2 * e], x[2 * e + 1]);
                tmem_st_u32(s_tm + c / 2, w);  // over columns that have been read
            }
            tmem_st_wait();
            arrive(kBarP + st);
        }
        // Join the streams: the second's O comes through shared memory, once all products are done.
        if (ok) {
            sml[128 * st + row] = make_float2(m, l);
            arrive(kBarMl);
            ok = wait_for(kBarMl, 0);
        }
        if (ok && ntiles > 0) ok = wait_for(kBarPv, ((ntiles + 1) / 2 - 1) & 1);
        if (ok && ntiles > 1) ok = wait_for(kBarPv + 1, (ntiles / 2 - 1) & 1);
        float fac = 1.f, sum = 0.f, top = m;
        if (ok) {
            const float2 o2 = sml[128 * (st ^ 1) + row];
            top = fmaxf(m, o2.x);
            fac = m == -INFINITY ? 1.f : ex2(m - top);
            sum = l * fac + o2.y * (o2.x == -INFINITY ? 1.f : ex2(o2.x - top));
        }
        float *so = reinterpret_cast<float *>(sm + L::kOut) + row * (D + 4);
        if (st == 1) {
            if (ok && ntiles > 1) {
#pragma unroll 1
                for (int c = 0; c < D; c += 32) {
                    float x[32];
                    tmem_ld32(o_tm + c, x);
#pragma unroll
                    for (int e = 0; e < 32; e += 4)
                        *reinterpret_cast<float4 *>(so + c + e) = make_float4(x[e] * fac, x[e + 1] * fac, x[e + 2] * fac, x[e + 3] * fac);
                }
                arrive(kBarJoin);
            }
        } else if (ok) {
            if (ntiles > 1) ok = wait_for(kBarJoin, 0);
            const int64_t unit = (((int64_t)b * a.kv.Hk + h) * a.tiles + tile) * a.splits + split;
            const float inv = ns > 1 ? 1.f : sum == 0.f ? 0.f : a.kv.v_scale / sum;
            if (ok) {
#pragma unroll 1
                for (int c = 0; c < D; c += 32) {
                    float x[32];
                    if (ntiles > 0) tmem_ld32(o_tm + c, x);
#pragma unroll
                    for (int e = 0; e < 32; e += 4) {
                        float4 y = ntiles > 1 ? *reinterpret_cast<const float4 *>(so + c + e) : make_float4(0.f, 0.f, 0.f, 0.f);
                        if (ntiles > 0) {
                            y.x = fmaf(x[e], fac, y.x); y.y = fmaf(x[e + 1], fac, y.y);
                            y.z = fmaf(x[e + 2], fac, y.z); y.w = fmaf(x[e + 3], fac, y.w);
                        }
                        // a NaN value belongs to the rows that see its token
                        const float w = snan[(c + e) >> 4] < seen ? NAN : inv;
                        x[e] = y.x * w; x[e + 1] = y.y * w; x[e + 2] = y.z * w; x[e + 3] = y.w * w;
                    }
                    if (live && ns > 1) {
                        float4 *dst = reinterpret_cast<float4 *>(a.part + (unit * 128 + row) * D + c);
#pragma unroll
                        for (int e = 0; e < 8; ++e) dst[e] = make_float4(x[4 * e], x[4 * e + 1], x[4 * e + 2], x[4 * e + 3]);
                    } else if (live) {
                        uint4 *dst = reinterpret_cast<uint4 *>(a.out + q_at + c);
#pragma unroll
                        for (int e = 0; e < 4; ++e) {
                            uint32_t w[4];
#pragma unroll
                            for (int u = 0; u < 4; ++u) {
                                const __nv_bfloat162 v = __floats2bfloat162_rn(x[8 * e + 2 * u], x[8 * e + 2 * u + 1]);
                                w[u] = *reinterpret_cast<const uint32_t *>(&v);
                            }
                            dst[e] = make_uint4(w[0], w[1], w[2], w[3]);
                        }
                    }
                    __syncwarp();
                }
                if (live && ns > 1) {
                    float2 *ml = reinterpret_cast<float2 *>(a.part + (int64_t)a.B * a.kv.Hk * a.tiles * a.splits * 128 * D);
                    ml[unit * 128 + row] = make_float2(top, sum);
                }
            }
        }
    } else if (warp < kTilesIssuer) {
        // Thread: a token of a tile.
        const int row = tid - 32 * kWide0;
        const int64_t head_bytes = kv4_head_bytes(ps, D);
        struct Bytes {
            uint4 k[D / 32], v[D / 32];
            uint32_t ks[D / 64], vs[D / 64];
            bool gone;
        };
        auto fetch = [&](int j) {
            Bytes x;
#pragma unroll
            for (int u = 0; u < D / 32; ++u) x.k[u] = x.v[u] = make_uint4(0, 0, 0, 0);
#pragma unroll
            for (int u = 0; u < D / 64; ++u) x.ks[u] = x.vs[u] = 0;
            x.gone = false;
            const int t = t_begin + 128 * j + row;
            if (j < ntiles && t < t_end) {
                const int at = t / ps, off = t - at * ps, page = a.table[(int64_t)b * a.max_pages + at];
                if (page < 0 || page >= a.kv.pages) {
                    report_opt(a.err, DEV_BAD_PAGE, b, h, page);
                    x.gone = true;
                } else {
                    const uint8_t *kp = a.cache + ((int64_t)page * a.kv.Hk + h) * head_bytes, *vp = kp + ps * (D * 9 / 16);
                    const int code = off * (D / 2), sc = ps * (D / 2) + off * (D / 16);
#pragma unroll
                    for (int u = 0; u < D / 32; ++u) {
                        x.k[u] = *reinterpret_cast<const uint4 *>(kp + code + 16 * u);
                        x.v[u] = *reinterpret_cast<const uint4 *>(vp + code + 16 * u);
                    }
#pragma unroll
                    for (int u = 0; u < D / 64; ++u) {
                        x.ks[u] = *reinterpret_cast<const uint32_t *>(kp + sc + 4 * u);
                        x.vs[u] = *reinterpret_cast<const uint32_t *>(vp + sc + 4 * u);
                    }
                }
            }
            return x;
        };
        auto put = [&](uint8_t *to, const uint4 (&codes)[D / 32], const uint32_t (&scales)[D / 64]) {
#pragma unroll
            for (int w = 0; w < D / 8; ++w) {  // words of 8 codes, two to a block
                uint32_t hh[4];
                widen((&codes[w >> 2].x)[w & 3], hh);
                const uint32_t s2 = scales2((scales[w >> 3] >> (8 * ((w >> 1) & 3))) & 0xff), s = __byte_perm(s2, s2, 0x1010);
                *reinterpret_cast<uint4 *>(to + sw128_chunk(row, w, 128)) = make_uint4(mul2(hh[0], s), mul2(hh[1], s), mul2(hh[2], s), mul2(hh[3], s));
            }
        };
        Bytes cur = fetch(0);
        for (int j = 0; j < ntiles; ++j) {
            const int st = j & 1, k = j >> 1, t = t_begin + 128 * j + row;
            const Bytes next = fetch(j + 1);
            // A NaN value leaves the product (0 NaN is NaN); the first token with one is kept for its block.
#pragma unroll
            for (int u = 0; u < D / 16; ++u)
                if (((cur.vs[u >> 2] >> (8 * (u & 3))) & 0x7f) == 0x7f) {
                    atomicMin(snan + u, t);
                    cur.vs[u >> 2] &= ~(0xffu << (8 * (u & 3)));
                }
            if (j >= 2 && !wait_for(kBarSc + st, (k - 1) & 1)) break;
            const uint32_t gone = __ballot_sync(0xffffffffu, cur.gone);
            if (lane == 0) sgone[4 * (j & 3) + warp - kWide0] = gone;
            put(sm + L::kKt + st * L::kTileB, cur.k, cur.ks);
            fence_async_smem();
            arrive(kBarK + st);
            if (j >= 2 && !wait_for(kBarPv + st, (k - 1) & 1)) break;
            put(sm + L::kVt + st * L::kTileB, cur.v, cur.vs);
            fence_async_smem();
            arrive(kBarVt + st);
            cur = next;
        }
    } else {
        const bool lead = elect_one();
        const uint32_t smem0 = smem_u32(sm), q = sw128_desc_lo(smem0 + L::kQ);
        auto scores = [&](int j) {
            const uint32_t kd = sw128_desc_lo(smem0 + L::kKt + (j & 1) * L::kTileB);
#pragma unroll
            for (int ks = 0; ks < D / 16; ++ks) {
                const uint32_t at = ((ks >> 2) * 128 * 128 + (ks & 3) * 32) / 16;
                umma_bf16(tmem + 128 * (j & 1), sw128_desc_of(q + at), sw128_desc_of(kd + at), idesc_f16_f32(128, 128, false), ks > 0);
            }
            umma_commit(bar + kBarSc + (j & 1));
        };
        auto output = [&](int j) {
            const uint32_t vd = sw128_desc_lo(smem0 + L::kVt + (j & 1) * L::kTileB, 128 * 128);
#pragma unroll
            for (int ks = 0; ks < 8; ++ks)
                umma_ts(tmem + kTmO + D * (j & 1), tmem + 128 * (j & 1) + 8 * ks, sw128_desc_of(vd + ks * 2048 / 16),
                        idesc_f16_f32(128, D, true), j > 1 || ks > 0);
            umma_commit(bar + kBarPv + (j & 1));
        };
        bool ok = ntiles == 0 || wait_for(kBarQ, 0);
        for (int j = 0; ok && j < 2 && j < ntiles; ++j) {
            if (!(ok = wait_for(kBarK + j, 0))) break;
            if (lead) scores(j);
        }
        for (int j = 0; ok && j < ntiles; ++j) {
            const int st = j & 1, k = j >> 1;
            if (!(ok = wait_for(kBarVt + st, k & 1) && wait_for(kBarP + st, k & 1))) break;
            if (lead) output(j);
            if (j + 2 < ntiles) {
                if (!(ok = wait_for(kBarK + st, (k + 1) & 1))) break;
                if (lead) scores(j + 2);
            }
        }
        if (*sfail) {  // products that may still run
            if (lead) umma_commit(bar + kBarDrain);
            __syncwarp();
            bar_wait(bar + kBarDrain, 0);
        }
    }
    tc_fence_before();
    __syncthreads();
    if (*sfail && tid == 0) report_opt(a.err, DEV_PIPE_TIMEOUT, b, h, t_begin);
    if (warp == 0) tmem_dealloc(tmem, 512);
}

template <int D> cudaError_t launch(const AttendArgs &a, cudaStream_t st) {
    // One CTA has the SM's tensor memory: a second one (which D = 64 would leave room for) could only wait for it.
    const int need = TilesSmem<D>::kBytes + 1024, smem = need > 116 * 1024 ? need : 116 * 1024;
    const cudaError_t e = cudaFuncSetAttribute(attend_tiles_kernel<D>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    if (e != cudaSuccess) return e;
    attend_tiles_kernel<D><<<dim3(a.splits, a.tiles * a.kv.Hk, a.B), kTilesThreads, smem, st>>>(a);
    return cudaGetLastError();
}

}  // namespace

cudaError_t attend_tiles_launch(const AttendArgs &a, cudaStream_t st) {
    return a.kv.D == 64 ? launch<64>(a, st) : launch<128>(a, st);
}

}  // namespace rssm
