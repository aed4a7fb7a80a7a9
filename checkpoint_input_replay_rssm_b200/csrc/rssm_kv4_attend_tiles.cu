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
// Roles: 8 softmax warps (4 a stream, the first of which issues the stream's products) and 8 widening warps (16 tokens
// each, the next tile's bytes in registers ahead).  They meet on barriers in shared memory; every wait is bounded.
//
// 8 prompts' chunks of 100 to 512 tokens behind up to 4096, 16 query heads a key/value head of 128: 184 us of 41 at
// the rate of a library product.  A tile takes about 1.7 us, not the 0.55 that its products ask for: a stream's score
// read, maximum, exponentials and stores are one chain of which two streams hide a half, and a CTA's start (queries,
// first pages) is 10 us.
#include <math.h>

#include "rssm_internal.h"
#include "rssm_kv4_attend.cuh"
#include "rssm_umma.cuh"

namespace rssm {

namespace {

constexpr int kSoftWarps = 8, kWideWarps = 8, kWide0 = kSoftWarps;
constexpr int kTilesThreads = 32 * (kSoftWarps + kWideWarps);
enum TilesBar {
    kBarK = 0,    // K tile written, per stream (every widening warp)
    kBarVt = 2,   // V tile written
    kBarQ = 4,    // Q written (the four warps that write it)
    kBarSc = 5,   // S done, per stream
    kBarP = 7,    // P written, per stream (its four warps)
    kBarPv = 9,   // O updated, per stream
    kBarMl = 11,  // maxima and sums written (every softmax warp)
    kBarJoin = 12,  // the second stream's O written (its four warps)
    kBarDrain = 13,  // everything issued, per stream, after a failure
    kTilesBars = 15
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

// Request and tile of number u of the requests that are this kernel's, by all threads of a CTA; false past the last one.
__device__ bool find_tile(const AttendArgs &a, int u, int &b, int &tile) {
    __shared__ long long wsum[kTilesThreads / 32];
    __shared__ int found[2];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int per = (a.B + kTilesThreads - 1) / kTilesThreads, b0 = min(a.B, tid * per), b1 = min(a.B, b0 + per);
    auto tiles_of = [&](int i) {
        int r0, n, len;
        const bool ok = attend_request(a, i, r0, n, len) && attend_mine(a, n * a.G, true);
        return ok ? (n * a.G + 127) / 128 : 0;
    };
    long long mine = 0;
    for (int i = b0; i < b1; ++i) mine += tiles_of(i);
    long long x = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const long long v = __shfl_up_sync(0xffffffffu, x, o);
        if (lane >= o) x += v;
    }
    if (lane == 31) wsum[warp] = x;
    __syncthreads();
    x -= mine;
    long long all = 0;
    for (int w = 0; w < kTilesThreads / 32; ++w) {
        if (w < warp) x += wsum[w];
        all += wsum[w];
    }
    // more tiles than the rows have: requests that overlap
    if (all > a.packed && u == 0 && tid == 0) report_opt(a.err, DEV_BAD_LENGTHS, -1, 0, (int)min(all, 0x7fffffffll));
    if (u >= all) return false;
    if (u >= x && u < x + mine)
        for (int i = b0; i < b1; ++i) {
            const int n = tiles_of(i);
            if (u < x + n) {
                found[0] = i;
                found[1] = (int)(u - x);
                break;
            }
            x += n;
        }
    __syncthreads();
    b = found[0];
    tile = found[1];
    return true;
}

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
    const int h = blockIdx.y;
    const int ps = a.kv.ps, G = a.G;
    int tile = blockIdx.x, b = blockIdx.z;
    if (a.few) pdl_trigger();  // the split kernel may start, for the requests that are its own
    if (a.packed && !find_tile(a, blockIdx.x, b, tile)) return;
    int r0, n, len;
    if (!attend_request(a, b, r0, n, len)) {
        if (tid == 0) report_opt(a.err, DEV_BAD_LENGTHS, b, 0, len);
        return;
    }
    const int rows = n * G, row0 = tile * 128;
    if (row0 >= rows || !attend_mine(a, rows, true)) return;
    const int last = min(row0 + 128, rows) - 1;
    const int t_end = max(0, len - n + last / G + 1);  // tokens that the tile's last row sees
    const int ntiles = (t_end + 127) / 128;

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
    // Wait for a barrier's phase, a warp at a time; false, for every role, once any wait has run out.
    auto wait_for = [&](int which, int parity) {
        if (!warp_wait(bar + which, parity, sfail)) return false;
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
            if (!live) src = reinterpret_cast<const uint4 *>(a.q);  // any row: its scores are masked
            uint4 v[D / 8];
#pragma unroll
            for (int k = 0; k < D / 8; ++k) v[k] = src[k];
            float top = 0.f;
#pragma unroll
            for (int k = 0; k < D / 8; ++k) {
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const uint32_t x = (&v[k].x)[e];
                    top = fmaxf(top, fmaxf(fabsf(bf16_bits_to_float(x & 0xffff)), fabsf(bf16_bits_to_float(x >> 16))));
                }
            }
            const int ex = row_exponent(top);
            const float s0 = copysignf(pow2f(-(ex / 2)), a.scale);
            const float s1 = a.scale == 0.f ? 0.f : pow2f(-(ex - ex / 2));
            f = row_factor(a.scale, ex, top, seen > 0);
            if (st == 0) {
#pragma unroll
                for (int k = 0; k < D / 8; ++k) {
                    uint4 w;
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        const uint32_t x = (&v[k].x)[e];
                        (&w.x)[e] = f16x2(bf16_bits_to_float(x & 0xffff) * s0 * s1, bf16_bits_to_float(x >> 16) * s0 * s1);
                    }
                    *reinterpret_cast<uint4 *>(sm + L::kQ + sw128_chunk(row, k, 128)) = w;
                }
                fence_async_smem();
                arrive(kBarQ);
            }
        }
        const uint32_t s_tm = base + 128 * st, o_tm = base + kTmO + D * st;
        // The products of this stream, issued by one thread of its first warp.
        const bool issues = (warp & 3) == 0, lead = issues && elect_one();
        const uint32_t smem0 = smem_u32(sm), q = sw128_desc_lo(smem0 + L::kQ);
        const uint32_t kd = sw128_desc_lo(smem0 + L::kKt + st * L::kTileB), vd = sw128_desc_lo(smem0 + L::kVt + st * L::kTileB, 128 * 128);
        auto scores = [&] {
            if (lead) {
#pragma unroll
                for (int ks = 0; ks < D / 16; ++ks) {
                    const uint32_t at = ((ks >> 2) * 128 * 128 + (ks & 3) * 32) / 16;
                    umma_bf16(tmem + 128 * st, sw128_desc_of(q + at), sw128_desc_of(kd + at), idesc_f16_f32(128, 128, false), ks > 0);
                }
                umma_commit(bar + kBarSc + st);
            }
            __syncwarp();
        };
        auto output = [&](bool more) {
            if (lead) {
#pragma unroll
                for (int ks = 0; ks < 8; ++ks)
                    umma_ts(tmem + kTmO + D * st, tmem + 128 * st + 8 * ks, sw128_desc_of(vd + ks * 2048 / 16),
                            idesc_f16_f32(128, D, true), more || ks > 0);
                umma_commit(bar + kBarPv + st);
            }
            __syncwarp();
        };
        float m = -INFINITY, l = 0.f;
        bool ok = true;
        if (issues && st < ntiles) {
            ok = wait_for(kBarQ, 0) && wait_for(kBarK + st, 0);
            if (ok) scores();
        }
        for (int j = st; ok && j < ntiles; j += 2) {
            const int k = j >> 1, t0 = 128 * j;
            if (!(ok = wait_for(kBarSc + st, k & 1))) break;
            const int lim = min(seen, t_end) - t0;  // columns below lim are seen
            const uint32_t *gone = sgone + 4 * (j & 3);
            const bool edge = __any_sync(0xffffffffu, lim < 128) || (gone[0] | gone[1] | gone[2] | gone[3]);
            // Two passes over S (the maximum, then P, which takes S's place), 16 columns under way while 16 are worked on.
            float x[2][16], top = -INFINITY;
            auto masked = [&](int c, float(&y)[16]) {
                if (edge) {
                    const uint32_t gw = gone[c >> 1] >> (16 * (c & 1));
#pragma unroll
                    for (int e = 0; e < 16; ++e)
                        if (16 * c + e >= lim || (gw >> e & 1)) y[e] = -INFINITY;
                }
            };
            tmem_ld16_start(s_tm, x[0]);
#pragma unroll 1
            for (int c2 = 0; c2 < 8; c2 += 2)
#pragma unroll
                for (int u = 0; u < 2; ++u) {
                    const int c = c2 + u;
                    tmem_ld_wait(x[u]);
                    tmem_ld16_start(s_tm + 16 * ((c + 1) & 7), x[u ^ 1]);  // the last one is the second pass's first
                    masked(c, x[u]);
#pragma unroll
                    for (int e = 0; e < 16; ++e) top = fmaxf(top, x[u][e]);
                }
            top *= f;
            if (__any_sync(0xffffffffu, top > m + kLag)) {
                const float mn = fmaxf(m, top), fac = mn == -INFINITY ? 1.f : ex2(m - mn);
                l *= fac;
                m = mn;
                if (k > 0) {
                    if (!(ok = wait_for(kBarPv + st, (k - 1) & 1))) break;
#pragma unroll 1
                    for (int c = 0; c < D; c += 16) {
                        float o[16];
                        tmem_ld16(o_tm + c, o);
#pragma unroll
                        for (int e = 0; e < 16; ++e) o[e] *= fac;
                        tmem_st16(o_tm + c, o);
                    }
                }
            }
            const float off = m == -INFINITY ? 0.f : m;  // a row that has seen nothing yet keeps p = 2^-inf = 0
#pragma unroll 1
            for (int c2 = 0; c2 < 8; c2 += 2)
#pragma unroll
                for (int u = 0; u < 2; ++u) {
                    const int c = c2 + u;
                    float(&y)[16] = x[u];
                    tmem_ld_wait(y);
                    if (c < 7) tmem_ld16_start(s_tm + 16 * (c + 1), x[u ^ 1]);
                    masked(c, y);
                    uint32_t w[8];
#pragma unroll
                    for (int e = 0; e < 16; ++e) {
                        y[e] = ex2(fmaf(y[e], f, -off));
                        l += y[e];
                    }
#pragma unroll
                    for (int e = 0; e < 8; ++e) w[e] = f16x2(y[2 * e], y[2 * e + 1]);
                    tmem_st_u32(s_tm + 8 * c, w);  // over columns that have been read
                }
            tmem_st_wait();
            arrive(kBarP + st);
            if (issues) {
                if (!(ok = wait_for(kBarP + st, k & 1) && wait_for(kBarVt + st, k & 1))) break;
                output(k > 0);
                if (j + 2 < ntiles) {  // S over P, behind the product that reads it
                    if (!(ok = wait_for(kBarK + st, (k + 1) & 1))) break;
                    scores();
                }
            }
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
            const float inv = sum == 0.f ? 0.f : a.kv.v_scale / sum;
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
                    if (live) {
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
            }
        }
        if (issues && warp_failed(sfail)) {  // products that may still run
            if (lead) umma_commit(bar + kBarDrain + st);
            __syncwarp();
            bar_wait(bar + kBarDrain + st, 0);
        }
    } else {
        // A warp has 16 tokens, 8 at a time: lane (token, quarter of its channels), so that a warp's read is one run of
        // 8 D/2 bytes (a token a lane took 1800 cycles a tile in reads of 32 lines each) and 8 neighbouring lanes'
        // writes of a chunk fall into different banks.
        constexpr int W = D / 32;  // words of 8 codes in a quarter
        const int tok = 16 * (warp - kWide0) + (lane & 7), quarter = lane >> 3;
        const int64_t head_bytes = kv4_head_bytes(ps, D);
        struct Bytes {
            uint32_t k[2][W], v[2][W], ks[2], vs[2];
            uint32_t live, gone;  // bit u, of token tok + 8 u: to be read; to be read, but its page is not there
        };
        // The page of a warp's tokens is looked up a tile before their bytes are fetched, and those a tile before they
        // are widened.  Its place in the table and theirs in the page move on by a tile without a division.
        struct Page {
            int p, off;
        };
        const int step_pages = 128 / ps, step_off = 128 - step_pages * ps;
        int left = t_end - 16 * (warp - kWide0);  // tokens from this warp's first on
        int at = 16 * (warp - kWide0) / ps, off = 16 * (warp - kWide0) - at * ps;
        const int32_t *table = a.table + (int64_t)b * a.max_pages;
        auto page_of_next = [&] {
            const Page x{left > 0 ? table[at] : 0, off};
            at += step_pages;
            off += step_off;
            if (off >= ps) {
                off -= ps;
                ++at;
            }
            left -= 128;
            return x;
        };
        const int64_t page_bytes = a.kv.Hk * head_bytes;
        const uint8_t *head = a.cache + h * head_bytes;
        const int in_code = (lane & 7) * (D / 2) + quarter * (D / 8), in_scale = ps * (D / 2) + (lane & 7) * (D / 16) + quarter * (D / 64);
        // (Loads without a branch around them: one that joins a zero for what is not read waits for the load there.)
        auto fetch = [&](int j, const Page &pg) {
            Bytes x;
            x.live = x.gone = 0;
#pragma unroll
            for (int u = 0; u < 2; ++u) {
                const int page = pg.p;
                const bool want = 128 * j + tok + 8 * u < t_end, there = page >= 0 && page < a.kv.pages;
                x.live |= (uint32_t)(want && there) << u;
                x.gone |= (uint32_t)(want && !there) << u;
                const uint8_t *kp = head + (want && there ? page : 0) * page_bytes, *vp = kp + ps * (D * 9 / 16);
                const int o = pg.off + 8 * u, code = in_code + o * (D / 2), sc = in_scale + o * (D / 16);
                if constexpr (D == 128) {
                    const uint4 kw = *reinterpret_cast<const uint4 *>(kp + code), vw = *reinterpret_cast<const uint4 *>(vp + code);
                    x.k[u][0] = kw.x; x.k[u][1] = kw.y; x.k[u][2] = kw.z; x.k[u][3] = kw.w;
                    x.v[u][0] = vw.x; x.v[u][1] = vw.y; x.v[u][2] = vw.z; x.v[u][3] = vw.w;
                    x.ks[u] = *reinterpret_cast<const uint16_t *>(kp + sc);
                    x.vs[u] = *reinterpret_cast<const uint16_t *>(vp + sc);
                } else {
                    const uint2 kw = *reinterpret_cast<const uint2 *>(kp + code), vw = *reinterpret_cast<const uint2 *>(vp + code);
                    x.k[u][0] = kw.x; x.k[u][1] = kw.y;
                    x.v[u][0] = vw.x; x.v[u][1] = vw.y;
                    x.ks[u] = kp[sc];
                    x.vs[u] = vp[sc];
                }
            }
            return x;
        };
        auto put = [&](uint8_t *to, const uint32_t (&codes)[2][W], const uint32_t (&scales)[2], uint32_t live) {
#pragma unroll
            for (int u = 0; u < 2; ++u) {
                const uint32_t s2 = live >> u & 1 ? scales2(scales[u]) : 0;  // what is not there holds zeros
#pragma unroll
                for (int w = 0; w < W; ++w) {
                    uint32_t hh[4];
                    widen(codes[u][w], hh);
                    const uint32_t s = __byte_perm(s2, s2, w < 2 ? 0x1010 : 0x3232);
                    *reinterpret_cast<uint4 *>(to + sw128_chunk(tok + 8 * u, quarter * W + w, 128)) =
                        make_uint4(mul2(hh[0], s), mul2(hh[1], s), mul2(hh[2], s), mul2(hh[3], s));
                }
            }
        };
        Page page = page_of_next();
        Bytes cur = fetch(0, page);
        page = page_of_next();
        for (int j = 0; j < ntiles; ++j) {
            const int st = j & 1, k = j >> 1, t = 128 * j + tok;
            const Bytes next = fetch(j + 1, page);
            page = page_of_next();
            if (j >= 2 && !wait_for(kBarSc + st, (k - 1) & 1)) break;
            uint32_t gone = 0;  // bit of every token of the warp (its quarters agree)
#pragma unroll
            for (int u = 0; u < 2; ++u) gone |= (__ballot_sync(0xffffffffu, cur.gone >> u & 1) & 0xff) << (8 * u);
            if (lane == 0) {
                reinterpret_cast<uint16_t *>(sgone)[8 * (j & 3) + warp - kWide0] = (uint16_t)gone;
                if (gone) report_opt(a.err, DEV_BAD_PAGE, b, h, 128 * j);
            }
            put(sm + L::kKt + st * L::kTileB, cur.k, cur.ks, cur.live);
            fence_async_smem();
            arrive(kBarK + st);
            // A NaN value leaves the product (0 NaN is NaN); the first token with one is kept for its block.
#pragma unroll
            for (int u = 0; u < 2; ++u)
#pragma unroll
                for (int e = 0; e < D / 64; ++e)
                    if ((cur.live >> u & 1) && ((cur.vs[u] >> (8 * e)) & 0x7f) == 0x7f) {
                        atomicMin(snan + quarter * (D / 64) + e, t + 8 * u);
                        cur.vs[u] &= ~(0xffu << (8 * e));
                    }
            if (j >= 2 && !wait_for(kBarPv + st, (k - 1) & 1)) break;
            put(sm + L::kVt + st * L::kTileB, cur.v, cur.vs, cur.live);
            fence_async_smem();
            arrive(kBarVt + st);
            cur = next;
        }
    }
    tc_fence_before();
    __syncthreads();
    if (*sfail && tid == 0) report_opt(a.err, DEV_PIPE_TIMEOUT, b, h, row0);
    if (warp == 0) tmem_dealloc(tmem, 512);
}

template <int D> cudaError_t launch(const AttendArgs &a, cudaStream_t st) {
    // One CTA has the SM's tensor memory: a second one (which D = 64 would leave room for) could only wait for it.
    const int need = TilesSmem<D>::kBytes + 1024, smem = need > 116 * 1024 ? need : 116 * 1024;
    const cudaError_t e = cudaFuncSetAttribute(attend_tiles_kernel<D>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    if (e != cudaSuccess) return e;
    attend_tiles_kernel<D><<<a.packed ? dim3(a.packed, a.kv.Hk) : dim3(a.tiles, a.kv.Hk, a.B), kTilesThreads, smem, st>>>(a);
    return cudaGetLastError();
}

}  // namespace

cudaError_t attend_tiles_launch(const AttendArgs &a, cudaStream_t st) {
    return a.kv.D == 64 ? launch<64>(a, st) : launch<128>(a, st);
}

}  // namespace rssm
