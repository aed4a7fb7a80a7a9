// rssm_kv4_attend.cu -- causal grouped-query attention over the paged 4-bit cache
// (rssm_kv4_attend), for one decode token, the drafts of a verify or a prompt chunk.
//
//   out = sum_j p_j V_j / sum_j p_j,  p_j = 2^{s_j - m},  s_j = sm_scale log2(e) q . K_j
//
// The cache is read once per tile of 16 or 32 query rows (a request's rows times the
// query heads of one key/value head).  At 0.56 bytes an element the work that
// dequantising asks for is next to the bytes what bounds the kernel, so the codes go from
// shared memory to matrix-instruction operands inside a thread's registers and are
// never written back wide.  What makes that possible is that the channel order of
// the first product and the token order of the second are free, as long as both
// operands agree:
//   scores: lane (g, c) holds token g's channels [c D/4, (c+1) D/4), a 16-byte run of
//           codes with two block scales; k-step s multiplies its channels 4s .. 4s+3.
//   output: lane (r, c) holds the 16 (D = 64: 8) channels of block r of four tokens;
//           column r of n-tile j is channel j of block r.  Operands pair two tokens, so
//           the two tokens' nibbles are merged before they are widened.
// e2m1 x e4m3 has 6 significant bits, so the fp16 operands are exact.  Queries are scaled
// by a power of two per row (their bf16 bits fit fp16, smaller than 2^-33 of the row's
// largest is dropped); probabilities are fp16 (2^-11 of each), their sums, the
// running maximum and the accumulators fp32.  m trails the true maximum by up to
// 2^6, so that the accumulators are rescaled a few times per row and not each step.
//
// A warp streams its own tokens: 32 at a time, every kWarps-th group of 32 of the
// CTA's range, by asynchronous copies into a ring of kStages stages of its own; the warps of a
// CTA meet only at the end, to join their sums.  Long contexts are split over CTAs and
// joined by a second kernel, launched early.
//
// 256 requests of 4096 tokens, 2 heads of 128, 16 rows a tile: 116 us, 54% of the rate of a copy while it
// streams and 40% with the CTAs' start, tail and join; one request over 4096 tokens: 12.5 us,
// 8.5 of them start, one range and its end.  What bounds it in between is latency at 12 warps an SM: conversions, products and
// exponentials that wait for the one before use 53% of the issue slots and a third of the tensor pipe.  More rows a tile are
// nearly free (32 rows: two products for one widening).  Widening to shared memory first, wider copies and fewer warps with more stages were slower; a third
// CTA on the SM (160 registers a thread) is worth more than any of them.
#include <math.h>

#include "rssm_internal.h"
#include "rssm_kv4_attend.cuh"
#include "rssm_umma.cuh"

namespace rssm {

namespace {

constexpr int kWarps4 = 4;
constexpr int kStages = 3;
constexpr int kStep = 32;        // tokens a warp takes at a time

template <int D> struct Ring {
    static constexpr int kGran = 16 * D * 9 / 8;           // 16 tokens: K codes, K scales, V codes, V scales
    static constexpr int kPad = D == 128 ? 32 : 64;        // the second 16 tokens' rows fall into the other banks
    static constexpr int kStage = 2 * (kGran + kPad);
    static constexpr int kScale = 16 * D / 2;              // scales behind codes
    static constexpr int kV = 16 * D * 9 / 16;             // values behind keys
};
template <int D, int MT> struct Smem {
    static constexpr int kRing = kWarps4 * kStages * Ring<D>::kStage;
    static constexpr int kMerge = kWarps4 * 16 * (D + 4) * 4;  // over the ring, one 16-row tile at a time
    static constexpr int kQ = kRing > kMerge ? kRing : kMerge;
    static constexpr int kMl = kQ + MT * (D / 16) * 512;       // query operands: [mt][k-step][lane] 16 bytes
    static constexpr int kRow = kMl + kWarps4 * MT * 16 * 8;   // (m, l) of every warp and row
    static constexpr int kBytes = kRow + MT * 16 * 8;          // score factor and visible tokens of every row
};

__device__ __forceinline__ void mma16816(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    asm(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

template <int D, int MT>
__global__ void __launch_bounds__(32 * kWarps4, MT == 1 ? 3 : 2) attend_kernel(const AttendArgs a) {
    using R = Ring<D>;
    using S = Smem<D, MT>;
    constexpr int KS = D / 16;   // k-steps of the scores
    constexpr int NT = D / 8;    // n-tiles of the output
    constexpr int RT = 16 * MT;  // rows of the tile
    extern __shared__ __align__(128) uint8_t sm[];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, g = lane >> 2, c = lane & 3;
    const int split = blockIdx.x, tile = blockIdx.y % a.tiles, h = blockIdx.y / a.tiles, b = blockIdx.z;
    const int ps = a.kv.ps, G = a.G;
    if (a.splits > 1) pdl_trigger();  // the joining kernel's CTAs may start, up to their wait
    // Beside the kernel of the 128-row tiles, which it may have been started before the end of, it does not end before that.
    auto end = [&] {
        if (a.few && (split | blockIdx.y | b) == 0) pdl_wait();
    };
    int r0, n, len;
    if (!attend_request(a, b, r0, n, len)) {
        if (tid == 0) report_opt(a.err, DEV_BAD_LENGTHS, b, 0, len);
        return end();
    }
    const int rows = n * G, row0 = tile * RT;
    if (row0 >= rows || !attend_mine(a, rows, false)) return end();
    // tokens that the tile's last row sees
    const int last = min(row0 + RT, rows) - 1;
    const int tlen = max(0, len - n + last / G + 1);
    const int ns = max(1, (tlen + a.L - 1) / a.L);
    if (split >= ns) return end();
    const int t_begin = split * a.L, t_end = min(tlen, t_begin + a.L);
    const int first_seen = len - n + row0 / G + 1;  // tokens that the tile's first row sees

    uint8_t *ring = sm + warp * kStages * R::kStage;
    uint4 *sq = reinterpret_cast<uint4 *>(sm + S::kQ);
    float2 *sml = reinterpret_cast<float2 *>(sm + S::kMl);
    float *sf = reinterpret_cast<float *>(sm + S::kRow);
    int *sseen = reinterpret_cast<int *>(sm + S::kRow) + RT;

    // Query operands, [mt][k-step][lane]: warp w makes those of the rows g + 8 (w & 1) of 16-row tile w >> 1.  Its rows
    // are on their way while the page table is.
    const int mt = warp >> 1, u = warp & 1, row = row0 + 16 * mt + g + 8 * u;
    const bool live = row < rows;
    const int i = live ? row / G : 0, hd = live ? row - i * G : 0;
    const uint4 *src =
        reinterpret_cast<const uint4 *>(a.q + ((int64_t)(r0 + i) * a.Hq + h * G + hd) * D + c * (D / 4));
    uint4 raw[D / 32];
#pragma unroll
    for (int k = 0; k < D / 32; ++k) raw[k] = warp < 2 * MT && live ? src[k] : make_uint4(0, 0, 0, 0);

    // This warp's steps: tokens t_begin + 32 (warp + kWarps4 i).  Lane l keeps the page of
    // 16-token group l & 1 of step l >> 1 of a window of 16 steps, -1 for one that is not
    // read (behind the last token, or outside the cache).
    const int steps_all = (max(0, t_end - t_begin) + kStep - 1) / kStep;
    const int steps = steps_all > warp ? (steps_all - warp + kWarps4 - 1) / kWarps4 : 0;
    // The group's place in its page goes with it: 16 page + place (ps <= 256).
    auto pages_of = [&](int win) {
        const int i = win * 16 + (lane >> 1);
        const int t = t_begin + kStep * (warp + kWarps4 * i) + 16 * (lane & 1);
        int page = -1;
        if (i < steps && t < t_end) {
            const int at = t / ps;
            page = a.table[(int64_t)b * a.max_pages + at];
            if (page < 0 || page >= a.kv.pages) {
                report_opt(a.err, DEV_BAD_PAGE, b, h, page);
                page = -1;
            } else {
                page = page * 16 + ((t - at * ps) >> 4);
            }
        }
        return page;
    };
    int pg = pages_of(0), pg_next = pages_of(1);
    const int64_t head_bytes = kv4_head_bytes(ps, D);
    // Start the copies of step i into stage sg, 16 bytes a lane at a time: the codes of a group are D / 64
    // such rounds for keys and as many for values, the scales of both groups are one round.  A group that
    // is not read is filled with zeros.
    const int64_t page_bytes = a.kv.Hk * head_bytes;
    const int v_src = ps * (D * 9 / 16);  // values behind keys in a page
    const int sc_gr = lane / (D / 8), sc_v = (lane / (D / 16)) & 1, sc_at = (lane % (D / 16)) * 16;
    const int sc_src = sc_v * v_src + ps * (D / 2) + sc_at;
    uint8_t *sc_dst = ring + (sc_gr & 1) * (R::kGran + R::kPad) + sc_v * R::kV + R::kScale + sc_at;
    auto issue = [&](int i, int sg, int window) {
        const int gp = (i >> 4) == window ? pg : pg_next;
        const uint8_t *sc_from = a.cache;
        int sc_live = 0;
#pragma unroll
        for (int gr = 0; gr < 2; ++gr) {
            const int at = __shfl_sync(0xffffffffu, gp, 2 * (i & 15) + gr);
            const bool live = at >= 0;
            const int page = live ? at >> 4 : 0, place = live ? at & 15 : 0;
            const uint8_t *src = a.cache + page * page_bytes + h * head_bytes;
            uint8_t *dst = ring + sg * R::kStage + gr * (R::kGran + R::kPad) + lane * 16;
#pragma unroll
            for (int k = 0; k < D / 64; ++k) {
                cp_async16_or_zero(dst + 512 * k, src + place * R::kScale + lane * 16 + 512 * k, live);
                cp_async16_or_zero(dst + R::kV + 512 * k, src + v_src + place * R::kScale + lane * 16 + 512 * k, live);
            }
            if (sc_gr == gr) {
                sc_from = src + place * D + sc_src;
                sc_live = live;
            }
        }
        if (sc_gr < 2) cp_async16_or_zero(sc_dst + sg * R::kStage, sc_from, sc_live);
    };
#pragma unroll 1
    for (int i = 0; i < kStages - 1; ++i) {
        if (i < steps) issue(i, i, 0);
        cp_async_commit();
    }

    if (warp < 2 * MT) {
        float top = 0.f;
#pragma unroll
        for (int k = 0; k < D / 32; ++k) {
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const uint32_t x = (&raw[k].x)[e];
                top = fmaxf(top, fmaxf(fabsf(bf16_bits_to_float(x & 0xffff)), fabsf(bf16_bits_to_float(x >> 16))));
            }
        }
        top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 1));
        top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 2));
        const int ex = row_exponent(top);
        // 2^-ex as two factors: one alone may leave fp32's range.
        const float s0 = copysignf(pow2f(-(ex / 2)), a.scale);
        const float s1 = a.scale == 0.f ? 0.f : pow2f(-(ex - ex / 2));
        if (c == 0) {
            const int seen = live ? len - n + i + 1 : 0;
            sf[16 * mt + g + 8 * u] = row_factor(a.scale, ex, top, seen > 0);
            sseen[16 * mt + g + 8 * u] = seen;
        }
        uint32_t *dst = reinterpret_cast<uint32_t *>(sq) + (mt * KS * 32 + lane) * 4 + u;
#pragma unroll
        for (int k = 0; k < D / 32; ++k)
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const uint32_t x = (&raw[k].x)[e];
                dst[(2 * k + (e >> 1)) * 128 + 2 * (e & 1)] =
                    f16x2(bf16_bits_to_float(x & 0xffff) * s0 * s1, bf16_bits_to_float(x >> 16) * s0 * s1);
            }
    }
    __syncthreads();
    float f[MT][2];   // factor of this lane's rows' scores
    int seen[MT][2];  // tokens that they see
#pragma unroll
    for (int mt = 0; mt < MT; ++mt)
#pragma unroll
        for (int u = 0; u < 2; ++u) {
            f[mt][u] = sf[16 * mt + g + 8 * u];
            seen[mt][u] = sseen[16 * mt + g + 8 * u];
        }

    float o[MT][NT][4], m[MT][2], l[MT][2];
#pragma unroll
    for (int mt = 0; mt < MT; ++mt) {
#pragma unroll
        for (int j = 0; j < NT; ++j)
#pragma unroll
            for (int e = 0; e < 4; ++e) o[mt][j][e] = 0.f;
        m[mt][0] = m[mt][1] = -INFINITY;
        l[mt][0] = l[mt][1] = 0.f;
    }

    // Token of a step: group (16), then 4 x n-tile + 2 e + (e ^ parity), so that neighbouring lanes of either
    // product's loads read rows an odd number apart (no bank conflicts).
    const int ge = g & 1, gc = (g >> 1) & 1;
    const int k_at = (g >> 2) * (R::kGran + R::kPad) + (2 * ge + (ge ^ gc)) * (D / 2) + c * (D / 8);
    const int ks_at = (g >> 2) * (R::kGran + R::kPad) + R::kScale + (2 * ge + (ge ^ gc)) * (D / 16) + c * (D / 64);
    const int v_at = (c >> 1) * (R::kGran + R::kPad) + R::kV + g * (D / 16);
    const int vs_at = (c >> 1) * (R::kGran + R::kPad) + R::kV + R::kScale + (D == 128 ? g : g >> 1);
    const int par = c & 1;

    uint32_t nan_cols = 0;  // bit 2 (2 mt + k) + e: row g + 8 k saw a NaN value in block 2 c + e
    int sg = 0;
    for (int i = 0; i < steps; ++i) {
        const int window = i >> 4;
        if ((i & 15) == 0 && i > 0) {
            pg = pg_next;
            pg_next = pages_of(window + 1);
        }
        if (i + kStages - 1 < steps) issue(i + kStages - 1, sg == 0 ? kStages - 1 : sg - 1, window);
        cp_async_commit();
        cp_async_wait_group<kStages - 1>();
        __syncwarp();  // the other lanes' copies are there too
        const uint8_t *st = ring + sg * R::kStage;
        if (++sg == kStages) sg = 0;
        const int t0 = t_begin + kStep * (warp + kWarps4 * i);
        const int page0 = __shfl_sync(0xffffffffu, pg, 2 * (i & 15)), page1 = __shfl_sync(0xffffffffu, pg, 2 * (i & 15) + 1);
        // a step where some row does not see every token, or a page is not there
        const bool edge = t0 + kStep > first_seen || t0 + kStep > t_end || page0 < 0 || page1 < 0;

        // Scores: the four n-tiles side by side, so that their chains of k-steps overlap.
        float x[MT][4][4];
        uint32_t code[4][D / 32], ksc[4];
#pragma unroll
        for (int u = 0; u < 4; ++u) {
#pragma unroll
            for (int mt = 0; mt < MT; ++mt)
#pragma unroll
                for (int e = 0; e < 4; ++e) x[mt][u][e] = 0.f;
            if constexpr (D == 128) {
                const uint4 w = *reinterpret_cast<const uint4 *>(st + k_at + 4 * u * (D / 2));
                code[u][0] = w.x; code[u][1] = w.y; code[u][2] = w.z; code[u][3] = w.w;
                ksc[u] = scales2(*reinterpret_cast<const uint16_t *>(st + ks_at + 4 * u * (D / 16)));
            } else {
                const uint2 w = *reinterpret_cast<const uint2 *>(st + k_at + 4 * u * (D / 2));
                code[u][0] = w.x; code[u][1] = w.y;
                ksc[u] = scales2(st[ks_at + 4 * u * (D / 16)]);
            }
        }
#pragma unroll
        for (int w = 0; w < D / 32; ++w) {
            uint32_t hh[4][4];
#pragma unroll
            for (int u = 0; u < 4; ++u) {
                const uint32_t sc = __byte_perm(ksc[u], ksc[u], w < D / 64 ? 0x1010 : D == 128 ? 0x3232 : 0x1010);
                widen(code[u][w], hh[u]);
#pragma unroll
                for (int e = 0; e < 4; ++e) hh[u][e] = mul2(hh[u][e], sc);
            }
#pragma unroll
            for (int e = 0; e < 2; ++e)
#pragma unroll
                for (int mt = 0; mt < MT; ++mt) {
                    const uint4 qa = sq[(mt * KS + 2 * w + e) * 32 + lane];
                    const uint32_t av[4] = {qa.x, qa.y, qa.z, qa.w};
#pragma unroll
                    for (int u = 0; u < 4; ++u) mma16816(x[mt][u], av, hh[u][2 * e], hh[u][2 * e + 1]);
                }
        }

        // Softmax: running maximum and sum of this lane's two rows a tile.
        const bool gone[2] = {page0 < 0, page1 < 0};
        const bool mine_gone = gone[c >> 1];
        uint32_t p[MT][2][4];
#pragma unroll
        for (int mt = 0; mt < MT; ++mt) {
            float top[2] = {-INFINITY, -INFINITY};
            if (edge) {
                const int lim[2] = {mine_gone ? 0 : min(seen[mt][0], t_end) - t0 - 16 * (c >> 1),
                                    mine_gone ? 0 : min(seen[mt][1], t_end) - t0 - 16 * (c >> 1)};
#pragma unroll
                for (int u = 0; u < 4; ++u)
#pragma unroll
                    for (int e = 0; e < 4; ++e)
                        if (4 * u + 2 * (e & 1) + ((e & 1) ^ par) >= lim[e >> 1]) x[mt][u][e] = -INFINITY;
            }
#pragma unroll
            for (int u = 0; u < 4; ++u)
#pragma unroll
                for (int e = 0; e < 4; ++e) top[e >> 1] = fmaxf(top[e >> 1], x[mt][u][e]);
#pragma unroll
            for (int k = 0; k < 2; ++k) {
                top[k] = fmaxf(top[k], __shfl_xor_sync(0xffffffffu, top[k], 1));
                top[k] = fmaxf(top[k], __shfl_xor_sync(0xffffffffu, top[k], 2)) * f[mt][k];
            }
            if (__any_sync(0xffffffffu, top[0] > m[mt][0] + kLag || top[1] > m[mt][1] + kLag)) {
                float fac[2];
#pragma unroll
                for (int k = 0; k < 2; ++k) {
                    const float mn = fmaxf(m[mt][k], top[k]);
                    fac[k] = mn == -INFINITY ? 1.f : ex2(m[mt][k] - mn);
                    m[mt][k] = mn;
                    l[mt][k] *= fac[k];
                }
#pragma unroll
                for (int j = 0; j < NT; ++j)
#pragma unroll
                    for (int e = 0; e < 4; ++e) o[mt][j][e] *= fac[e >> 1];
            }
            // a row that has seen nothing yet keeps m = -inf and p = 2^-inf = 0
            const float base[2] = {m[mt][0] == -INFINITY ? 0.f : m[mt][0], m[mt][1] == -INFINITY ? 0.f : m[mt][1]};
#pragma unroll
            for (int u = 0; u < 4; ++u) {
                float e4[4];
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    e4[e] = ex2(fmaf(x[mt][u][e], f[mt][e >> 1], -base[e >> 1]));
                    l[mt][e >> 1] += e4[e];
                }
                p[mt][u >> 1][2 * (u & 1)] = f16x2(e4[0], e4[1]);
                p[mt][u >> 1][2 * (u & 1) + 1] = f16x2(e4[2], e4[3]);
            }
        }

        // Output.
        uint32_t vsc[8];  // this lane's scales: [16-token step][n-tile of the scores][token of the pair]
#pragma unroll
        for (int k = 0; k < 8; ++k) vsc[k] = st[vs_at + (4 * (k >> 1) + 2 * (k & 1) + ((k & 1) ^ par)) * (D / 16)];
        if (edge) {
            // What no row sees has weight 0 and may hold anything: its scale is set to 0.  A NaN belongs to
            // the rows that see its token and to no other (0 NaN is NaN): it leaves the product, and the
            // rows that see it are marked.
            const int lim = mine_gone ? 0 : t_end - t0 - 16 * (c >> 1);
#pragma unroll
            for (int k = 0; k < 8; ++k) {
                const int idx = 4 * (k >> 1) + 2 * (k & 1) + ((k & 1) ^ par);
                if (idx >= lim) vsc[k] = 0;
                uint32_t bad = __ballot_sync(0xffffffffu, (vsc[k] & 0x7f) == 0x7f);
                if ((vsc[k] & 0x7f) == 0x7f) vsc[k] = 0;
                for (; bad; bad &= bad - 1) {
                    const int col = (__ffs(bad) - 1) >> 2, cc = (__ffs(bad) - 1) & 3;
                    const int t = t0 + 16 * (cc >> 1) + 4 * (k >> 1) + 2 * (k & 1) + ((k & 1) ^ (cc & 1));
#pragma unroll
                    for (int r = 0; r < 2 * MT; ++r)
                        if (c == col >> 1 && t < seen[r >> 1][r & 1]) nan_cols |= 1u << (2 * r + (col & 1));
                }
            }
        }
#pragma unroll
        for (int ms = 0; ms < 2; ++ms) {
            uint32_t code[2][2][D / 64], sc[2];  // [n-tile of the scores][token of the pair]
#pragma unroll
            for (int nt = 0; nt < 2; ++nt) {
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    const int idx = 8 * ms + 4 * nt + 2 * e + (e ^ par);
                    if constexpr (D == 128) {
                        const uint2 w = *reinterpret_cast<const uint2 *>(st + v_at + idx * (D / 2));
                        code[nt][e][0] = w.x; code[nt][e][1] = w.y;
                    } else {
                        code[nt][e][0] = *reinterpret_cast<const uint32_t *>(st + v_at + idx * (D / 2));
                    }
                }
                sc[nt] = scales2(vsc[4 * ms + 2 * nt] | vsc[4 * ms + 2 * nt + 1] << 8);
            }
#pragma unroll
            for (int w = 0; w < D / 64; ++w) {
                uint32_t ev[2][4], od[2][4];  // channels 8 w + {0, 2, 4, 6} and + {1, 3, 5, 7}, as token pairs
#pragma unroll
                for (int nt = 0; nt < 2; ++nt) {
                    const uint32_t w0 = code[nt][0][w], w1 = code[nt][1][w];
                    widen((w0 & 0x0f0f0f0fu) | ((w1 << 4) & 0xf0f0f0f0u), ev[nt]);
                    widen(((w0 >> 4) & 0x0f0f0f0fu) | (w1 & 0xf0f0f0f0u), od[nt]);
                }
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    const uint32_t e0 = mul2(ev[0][k], sc[0]), e1 = mul2(ev[1][k], sc[1]);
                    const uint32_t d0 = mul2(od[0][k], sc[0]), d1 = mul2(od[1][k], sc[1]);
#pragma unroll
                    for (int mt = 0; mt < MT; ++mt) {
                        mma16816(o[mt][8 * w + 2 * k], p[mt][ms], e0, e1);
                        mma16816(o[mt][8 * w + 2 * k + 1], p[mt][ms], d0, d1);
                    }
                }
            }
        }
        __syncwarp();  // the stage is free
    }
#pragma unroll
    for (int mt = 0; mt < MT; ++mt)
#pragma unroll
        for (int k = 0; k < 2; ++k) {
            l[mt][k] += __shfl_xor_sync(0xffffffffu, l[mt][k], 1);
            l[mt][k] += __shfl_xor_sync(0xffffffffu, l[mt][k], 2);
            if (c == 0) sml[(warp * MT + mt) * 16 + g + 8 * k] = make_float2(m[mt][k], l[mt][k]);
        }
    __syncthreads();

    // Join the warps: each scales its rows to the common maximum, then the sums are added from shared memory.
    float *so = reinterpret_cast<float *>(sm);
    constexpr int kRow = D + 4;
    const int64_t unit = (((int64_t)b * a.kv.Hk + h) * a.tiles + tile) * a.splits + split;
#pragma unroll
    for (int mt = 0; mt < MT; ++mt) {
        if (mt) __syncthreads();
#pragma unroll
        for (int k = 0; k < 2; ++k) {
            float top = -INFINITY;
#pragma unroll
            for (int w = 0; w < kWarps4; ++w) top = fmaxf(top, sml[(w * MT + mt) * 16 + g + 8 * k].x);
            const float scale = m[mt][k] == -INFINITY ? 1.f : ex2(m[mt][k] - top);
            float *dst = so + (warp * 16 + g + 8 * k) * kRow;
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                const float fac = (nan_cols >> (2 * (2 * mt + k) + e)) & 1 ? NAN : scale;
#pragma unroll
                for (int j = 0; j < NT; j += 4)
                    *reinterpret_cast<float4 *>(dst + (2 * c + e) * (D / 8) + j) =
                        make_float4(o[mt][j][2 * k + e] * fac, o[mt][j + 1][2 * k + e] * fac,
                                    o[mt][j + 2][2 * k + e] * fac, o[mt][j + 3][2 * k + e] * fac);
            }
        }
        __syncthreads();
        // 8 threads a row, D / 8 channels each
        const int row = tid >> 3, at = (tid & 7) * (D / 8);
        float top = -INFINITY, sum = 0.f;
#pragma unroll
        for (int w = 0; w < kWarps4; ++w) top = fmaxf(top, sml[(w * MT + mt) * 16 + row].x);
#pragma unroll
        for (int w = 0; w < kWarps4; ++w) {
            const float2 ml = sml[(w * MT + mt) * 16 + row];
            sum += ml.x == -INFINITY ? ml.y : ml.y * ex2(ml.x - top);
        }
        float acc[D / 8];
#pragma unroll
        for (int j = 0; j < D / 8; ++j) acc[j] = 0.f;
#pragma unroll 1
        for (int w = 0; w < kWarps4; ++w)
#pragma unroll
            for (int j = 0; j < D / 8; j += 4) {
                const float4 v = *reinterpret_cast<const float4 *>(so + (w * 16 + row) * kRow + at + j);
                acc[j] += v.x; acc[j + 1] += v.y; acc[j + 2] += v.z; acc[j + 3] += v.w;
            }
        const int grow = row0 + 16 * mt + row;
        if (grow >= rows) continue;
        if (ns == 1) {
            const float inv = sum == 0.f ? 0.f : a.kv.v_scale / sum;
            const int i = grow / G, hd = grow - i * G;
            uint32_t w[D / 16];
#pragma unroll
            for (int j = 0; j < D / 16; ++j) {
                const __nv_bfloat162 v = __floats2bfloat162_rn(acc[2 * j] * inv, acc[2 * j + 1] * inv);
                w[j] = *reinterpret_cast<const uint32_t *>(&v);
            }
            uint4 *dst = reinterpret_cast<uint4 *>(a.out + ((int64_t)(r0 + i) * a.Hq + h * G + hd) * D + at);
#pragma unroll
            for (int j = 0; j < D / 64; ++j) dst[j] = make_uint4(w[4 * j], w[4 * j + 1], w[4 * j + 2], w[4 * j + 3]);
        } else {
            float4 *dst = reinterpret_cast<float4 *>(a.part + (unit * RT + 16 * mt + row) * D + at);
#pragma unroll
            for (int j = 0; j < D / 32; ++j) dst[j] = make_float4(acc[4 * j], acc[4 * j + 1], acc[4 * j + 2], acc[4 * j + 3]);
            if ((tid & 7) == 0) {
                float2 *ml = reinterpret_cast<float2 *>(a.part + (int64_t)a.B * a.kv.Hk * a.tiles * a.splits * RT * D);
                ml[unit * RT + 16 * mt + row] = make_float2(top, sum);
            }
        }
    }
    end();
}

// Join the splits of a tile's rows: out = sum_s 2^{m_s - m} O_s / sum_s 2^{m_s - m} l_s.  D / 4 threads have a row, or,
// where there are few tiles and many splits, two such groups with every second split each, and each group of rows a
// CTA of its own (in sequence by one group, 79 splits of a long context took longer than the attention itself).
template <int D, int MT> struct Join {
    static constexpr int kThreads = 256, kLanes = D / 4;
};
template <int D, int MT>
__global__ void __launch_bounds__(Join<D, MT>::kThreads) attend_join_kernel(const AttendArgs a) {
    using J = Join<D, MT>;
    constexpr int RT = 16 * MT;
    __shared__ float4 part[J::kThreads / 2];
    const int at_once = gridDim.x / (a.tiles * a.kv.Hk), th = blockIdx.x / at_once, halves = at_once > 1 ? 2 : 1;
    const int at_a_time = J::kThreads / (halves * J::kLanes);  // rows
    const int tile = th % a.tiles, h = th / a.tiles, b = blockIdx.y;
    pdl_wait();  // first of all: no CTA ends before the kernel whose results it joins
    int r0, n, len;
    if (!attend_request(a, b, r0, n, len)) return;  // reported by the first kernel
    const int rows = n * a.G, row0 = tile * RT;
    if (row0 >= rows || !attend_mine(a, rows, false)) return;
    const int last = min(row0 + RT, rows) - 1;
    const int ns = (max(0, len - n + last / a.G + 1) + a.L - 1) / a.L;
    if (ns <= 1) return;
    const int l = threadIdx.x % J::kLanes, half = threadIdx.x / J::kLanes % halves, rl = threadIdx.x / (halves * J::kLanes);
    const int64_t unit = (((int64_t)b * a.kv.Hk + h) * a.tiles + tile) * a.splits;
    const float2 *ml0 = reinterpret_cast<const float2 *>(a.part + (int64_t)a.B * a.kv.Hk * a.tiles * a.splits * RT * D) + unit * RT;
    for (int r1st = blockIdx.x % at_once * at_a_time; r1st < RT; r1st += at_once * at_a_time) {
        const int r = r1st + rl;
        const float2 *ml = ml0 + r;
        float top = -INFINITY, sum = 0.f;
        for (int s = l; s < ns; s += J::kLanes) top = fmaxf(top, ml[s * RT].x);
#pragma unroll
        for (int o = 1; o < J::kLanes; o <<= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
        for (int s = l; s < ns; s += J::kLanes) {
            const float2 v = ml[s * RT];
            sum += v.x == -INFINITY ? v.y : v.y * ex2(v.x - top);
        }
#pragma unroll
        for (int o = 1; o < J::kLanes; o <<= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
        const float *src = a.part + (unit * RT + r) * D + 4 * l;
        float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 4
        for (int s = half; s < ns; s += halves) {
            const float m = ml[s * RT].x, fac = m == -INFINITY ? 1.f : ex2(m - top);
            const float4 x = *reinterpret_cast<const float4 *>(src + (int64_t)s * RT * D);
            acc.x = fmaf(x.x, fac, acc.x); acc.y = fmaf(x.y, fac, acc.y); acc.z = fmaf(x.z, fac, acc.z); acc.w = fmaf(x.w, fac, acc.w);
        }
        float4 x = make_float4(0.f, 0.f, 0.f, 0.f);
        if (halves == 2) {
            if (half) part[rl * J::kLanes + l] = acc;
            __syncthreads();
            x = part[rl * J::kLanes + l];
            __syncthreads();
        }
        if (!half && row0 + r < rows) {
            const float inv = sum == 0.f ? 0.f : a.kv.v_scale / sum;
            const int i = (row0 + r) / a.G, hd = row0 + r - i * a.G;
            const __nv_bfloat162 lo = __floats2bfloat162_rn((acc.x + x.x) * inv, (acc.y + x.y) * inv);
            const __nv_bfloat162 hi = __floats2bfloat162_rn((acc.z + x.z) * inv, (acc.w + x.w) * inv);
            *reinterpret_cast<uint2 *>(a.out + ((int64_t)(r0 + i) * a.Hq + h * a.G + hd) * D + 4 * l) =
                make_uint2(*reinterpret_cast<const uint32_t *>(&lo), *reinterpret_cast<const uint32_t *>(&hi));
        }
    }
}

float score_scale(float sm_scale, float k_scale) { return sm_scale * k_scale * 1.4426950408889634f; }

constexpr int64_t kMaxL = 2048, kWaves = 2;
constexpr int64_t kTileRows = 128, kTileUnits = 32, kPackTiles = 2;

// Sizes of the launch.  Row tiles of 32 where a request can have more than 16 rows.
struct Plan {
    int mt, tiles, splits, L;
    int few_mt, packed;  // 128-row tiles: the tiles (x 16 rows) of the kernel beside them, and how they are numbered (AttendArgs)
    size_t bytes;
};

// Cached tokens of one CTA: a share of the work that fills the machine (148 SMs, 3 CTAs each) kWaves times over,
// between 256 (a shorter one is all start and join) and kMaxL (a longer one makes a long tail).
void split_context(int64_t seq, int64_t units, Plan *p) {
    const int64_t want = 148 * 3 * kWaves;
    int64_t L = (seq * units + want - 1) / want;
    L = L < 256 ? 256 : L > kMaxL ? kMaxL : L;
    L = (L + 127) / 128 * 128;
    p->splits = (int)((seq + L - 1) / L);
    p->L = (int)L;
}

bool attend_plan(const rssm_kv4_config *c, const rssm_attend_config *t, Kv4Args *kv, Plan *p) {
    if (!kv4_args(c, kv) || !t) return false;
    if (t->batch < 1 || t->batch > 65535 || t->n_q_heads < 1 || t->n_q_heads > 65535 || t->n_q_heads % kv->Hk != 0)
        return false;
    if (t->tokens < 1 || t->max_pages < 1 || t->max_q < 1 || t->max_seq < 1) return false;
    if (!isfinite(score_scale(t->sm_scale, kv->k_scale))) return false;
    const int64_t max_q = t->max_q < t->tokens ? t->max_q : t->tokens;
    const int64_t rows = max_q * (t->n_q_heads / kv->Hk);
    if (rows > 0x3fffffff) return false;
    // Tiles of 128 rows where a request has as many and there are enough of them; they are not split.
    const int64_t big = (rows + 127) / 128;
    p->mt = rows >= kTileRows && (int64_t)t->batch * kv->Hk * big >= kTileUnits ? 8 : rows > 16 ? 2 : 1;
    const int64_t tiles = (rows + 16 * p->mt - 1) / (16 * p->mt);
    if (p->mt != 8 && tiles * kv->Hk > 65535) return false;
    int64_t seq = (int64_t)t->max_pages * kv->ps;
    if (t->max_seq < seq) seq = t->max_seq;
    if (seq > 1 << 30) return false;  // positions and their strides are int32
    p->tiles = (int)tiles;
    // Beside the 128-row tiles, which are not split, single tokens and drafts of one small tile keep the kernel that is:
    // a prompt's chunk in the batch would else leave each of them to one CTA for its whole context (15 tokens over 32768 and a
    // chunk of 512 over 2048: 892 us, now 102, apart 66 and 47).
    const int64_t G = t->n_q_heads / kv->Hk;
    p->few_mt = p->mt != 8 ? 0 : G <= 16 ? 1 : G <= 32 ? 2 : 0;
    const int64_t units = (int64_t)t->batch * kv->Hk * (p->few_mt ? 1 : tiles), rows_of = p->few_mt ? p->few_mt : p->mt;
    if (p->mt == 8 && !p->few_mt) {
        p->splits = 1;
        p->L = (int)((seq + 127) / 128 * 128);
    } else {
        split_context(seq, units, p);
    }
    p->bytes = p->splits > 1 ? (size_t)(units * p->splits * 16 * rows_of) * (size_t)(kv->D + 2) * 4 : 0;
    // A grid row of tiles for each request is mostly CTAs without work where one of them is long: then the tiles that so many
    // rows can make are numbered through, and a CTA looks its own up.  (The grid's CTAs over the tiles: 1.7, 8 chunks of 100 to
    // 512, 272 us against 311 numbered through; 2.1, one of 512 and 7 of 200, 161 against 162; 5, one of 512 and 31 of 100, 211
    // against 201; 46, one of 512 and 255 tokens, 127 numbered through.)
    const int64_t most = (int64_t)t->tokens * G / 128 + (t->batch < t->tokens ? t->batch : t->tokens);
    p->packed = p->few_mt && t->batch * tiles > kPackTiles * most ? (int)most : 0;
    return true;
}

template <int D, int MT>
cudaError_t attend_launch(const AttendArgs &a, cudaStream_t st) {
    cudaError_t e = cudaFuncSetAttribute(attend_kernel<D, MT>, cudaFuncAttributeMaxDynamicSharedMemorySize, Smem<D, MT>::kBytes);
    if (e != cudaSuccess) return e;
    cudaLaunchConfig_t cfg{};
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.gridDim = dim3(a.splits, a.tiles * a.kv.Hk, a.B);
    cfg.blockDim = dim3(32 * kWarps4);
    cfg.dynamicSmemBytes = Smem<D, MT>::kBytes;
    cfg.stream = st;
    cfg.attrs = attr;
    cfg.numAttrs = a.few ? 1 : 0;  // beside the 128-row tiles it need not wait for their end
    e = cudaLaunchKernelEx(&cfg, attend_kernel<D, MT>, a);
    if (e != cudaSuccess || a.splits == 1) return e;
    // (one request over 4096 / 20000 tokens: 12.5 / 25 us against 18.6 / 50 with one CTA a tile; 256 requests: 116
    // against 119 the other way about)
    const bool few = (int64_t)a.B * a.tiles * a.kv.Hk < 148;
    cfg.gridDim = dim3(a.tiles * a.kv.Hk * (few ? 16 * MT * 2 * Join<D, MT>::kLanes / Join<D, MT>::kThreads : 1), a.B);
    cfg.blockDim = dim3(Join<D, MT>::kThreads);
    cfg.dynamicSmemBytes = 0;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, attend_join_kernel<D, MT>, a);
}

}  // namespace

}  // namespace rssm

extern "C" {

RSSM_API size_t rssm_kv4_attend_workspace_bytes(const rssm_kv4_config *cfg, const rssm_attend_config *att) {
    rssm::Kv4Args kv;
    rssm::Plan p;
    return rssm::attend_plan(cfg, att, &kv, &p) ? p.bytes : 0;
}

RSSM_API rssm_status rssm_kv4_attend(const rssm_kv4_config *cfg, const rssm_attend_config *att, const void *q,
                                     const void *cache, const int32_t *block_table, const int32_t *seq_len,
                                     const int32_t *cu_q, void *out, void *workspace, size_t workspace_bytes,
                                     int32_t *dev_error, void *stream) {
    using namespace rssm;
    AttendArgs a{};
    Plan p;
    if (!attend_plan(cfg, att, &a.kv, &p) || !q || !cache || !block_table || !seq_len || !cu_q || !out)
        return RSSM_EINVAL;
    if (!aligned16(q) || !aligned16(cache) || !aligned16(out)) return RSSM_EINVAL;
    if (p.bytes && (!workspace || workspace_bytes < p.bytes || ((uintptr_t)workspace & 255))) return RSSM_EINVAL;
    a.B = att->batch; a.Hq = att->n_q_heads; a.G = att->n_q_heads / a.kv.Hk; a.tokens = att->tokens;
    a.max_pages = att->max_pages; a.max_q = att->max_q; a.max_seq = att->max_seq;
    a.tiles = p.tiles; a.splits = p.splits; a.L = p.L;
    a.scale = score_scale(att->sm_scale, a.kv.k_scale);
    a.q = (const __nv_bfloat16 *)q; a.cache = (const uint8_t *)cache;
    a.table = block_table; a.seq_len = seq_len; a.cu = cu_q; a.out = (__nv_bfloat16 *)out; a.part = (float *)workspace;
    a.err = dev_error;
    const cudaStream_t st = (cudaStream_t)stream;
    const bool wide = a.kv.D == 128;
    cudaError_t e = cudaSuccess;
    int mt = p.mt;
    if (mt == 8) {
        a.few = 16 * p.few_mt;
        a.packed = p.packed;
        e = attend_tiles_launch(a, st);
        a.tiles = 1;
        mt = p.few_mt;
    }
    if (e == cudaSuccess && mt == 2) e = wide ? attend_launch<128, 2>(a, st) : attend_launch<64, 2>(a, st);
    if (e == cudaSuccess && mt == 1) e = wide ? attend_launch<128, 1>(a, st) : attend_launch<64, 1>(a, st);
    return e == cudaSuccess ? RSSM_OK : RSSM_ECUDA;
}

}  // extern "C"
