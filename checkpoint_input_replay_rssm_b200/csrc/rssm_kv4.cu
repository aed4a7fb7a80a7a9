// rssm_kv4.cu -- writing and reading back the paged 4-bit key/value cache
// (rssm_kv4_append, rssm_kv4_export).
//
// Per block of 16 channels: s = e4m3(max|x| / (6 g)), code = e2m1(x / (s g)), both
// round to nearest even and saturating, g the tensor scale.  g is a power of two, so
// x / g is exact; x is bf16 (8 significant bits), s has 4 and a border between two codes
// (1/4, 3/4, 5/4, 7/4, 5/2, 7/2, 5) 3, so that x and border * s, at most 7 bits, are
// multiples of one unit of x's last place: a quotient that is not on a border is at least
// 2^-8 of itself away from it.  The quotients are therefore formed as x * (1 / (s g)), which
// errs by less than 2^-22, and rounded to 14 significant bits, which puts those that belong
// on a border back on it and takes no other across one: the stored codes are those of exact
// arithmetic, at three instructions an element where a division takes about ten.
//
// Both kernels are bound by HBM (2 bytes in, 9/16 out per element, and the
// reverse): one thread per block of keys and the same block of values, the 16 channels as two
// 16-byte accesses, the codes as one 8-byte access; 4 or 8 neighbouring threads cover a token's
// head.  65521 tokens, 8 heads of 64, 172 MB each way: 33 us written (5.2 TB/s) and 28 us
// read back (6.1 TB/s), of 26 at the rate of a copy; 256 tokens: about 4 us each, the
// latency of three dependent accesses.  A thread per tensor took 43 and 41 us, too
// few loads in flight; a division an element and 64-bit indexes 68 us.
#include <cuda_bf16.h>

#include <math.h>

#include "rssm_internal.h"
#include "rssm_kv4.cuh"

namespace rssm {

bool kv4_args(const rssm_kv4_config *c, Kv4Args *a) {
    if (!c || c->n_kv_heads < 1 || c->n_kv_heads > 65535 || (c->head_dim != 64 && c->head_dim != 128)) return false;
    if (c->page_size < 16 || c->page_size > 256 || c->page_size % 16 != 0 || c->num_pages < 1) return false;
    if ((int64_t)c->num_pages * c->page_size > 0x7fffffffLL) return false;
    auto pow2 = [](float s) {
        int e;
        return s > 0.f && isfinite(s) && frexpf(s, &e) == 0.5f && e - 1 >= -64 && e - 1 <= 64;
    };
    if (!pow2(c->k_scale) || !pow2(c->v_scale)) return false;
    if (a) *a = Kv4Args{c->n_kv_heads, c->head_dim, c->page_size, c->num_pages, 1.f / c->k_scale, 1.f / c->v_scale,
                        c->k_scale, c->v_scale};
    return true;
}

namespace {

constexpr int kKvThreads = 256;

// Two fp32 values to a byte of two e2m1 codes (lo in the low half).
__device__ __forceinline__ uint32_t e2m1x2(float lo, float hi) {
    uint32_t r;
    asm("{\n .reg .b8 t;\n cvt.rn.satfinite.e2m1x2.f32 t, %1, %2;\n cvt.u32.u8 %0, t;\n}\n" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
}
// A byte of two e2m1 codes to two fp16 values.
__device__ __forceinline__ uint32_t e2m1x2_f16x2(uint32_t b) {
    uint32_t r;
    asm("{\n .reg .b8 t;\n cvt.u8.u32 t, %1;\n cvt.rn.f16x2.e2m1x2 %0, t;\n}\n" : "=r"(r) : "r"(b));
    return r;
}
__device__ __forceinline__ uint32_t e4m3_of(float v) {
    uint16_t r;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(0.f), "f"(v));
    return r & 0xff;
}
__device__ __forceinline__ float e4m3_value(uint32_t b) {
    uint32_t r;
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(r) : "h"((uint16_t)b));
    return __half2float(__ushort_as_half((unsigned short)(r & 0xffff)));
}

// v to 14 significant bits (13 behind the leading one), to nearest (an infinity stays one).
__device__ __forceinline__ float to14bits(float v) {
    return __uint_as_float((__float_as_uint(v) + 0x200u) & 0xfffffc00u);
}

// The lanes of this warp whose index is below n; n is a multiple of 4, so that pairs stay whole.
__device__ __forceinline__ uint32_t live_lanes(uint32_t i, uint32_t n) {
    const uint32_t left = n - (i & ~31u);
    return left >= 32 ? ~0u : (1u << left) - 1;
}
// v of the other lane of a pair.
__device__ __forceinline__ uint4 swap1(uint32_t mask, const uint4 &v) {
    return make_uint4(__shfl_xor_sync(mask, v.x, 1), __shfl_xor_sync(mask, v.y, 1), __shfl_xor_sync(mask, v.z, 1),
                      __shfl_xor_sync(mask, v.w, 1));
}

// One thread per (token, head, block of 16 channels), for the keys and the values both: the loads
// of the two are in flight together, which these kernels' time hangs on.
template <int D>
__global__ void __launch_bounds__(kKvThreads) kv4_append_kernel(const Kv4Args a, uint32_t blocks, const uint4 *k,
                                                                const uint4 *v, const int32_t *slots,
                                                                uint8_t *cache, int32_t *err) {
    constexpr int nb = D >> 4;
    const uint32_t i = blockIdx.x * kKvThreads + threadIdx.x;
    if (i >= blocks) return;
    const uint4 *ks = k + 2 * (int64_t)i, *vs = v + 2 * (int64_t)i;
    const uint4 w[4] = {ks[0], ks[1], vs[0], vs[1]};
    const uint32_t t = i / (uint32_t)(a.Hk * nb), r = i - t * (uint32_t)(a.Hk * nb);
    const int h = (int)(r / nb), blk = (int)(r % nb);
    const int slot = slots[t];
    if (slot < 0) return;
    const int page = slot / a.ps, off = slot - page * a.ps;
    if (page >= a.pages) {
        report_opt(err, DEV_BAD_PAGE, (int)t, h, slot);
        return;
    }
    uint8_t *dst = cache + ((int64_t)page * a.Hk + h) * kv4_head_bytes(a.ps, D);
#pragma unroll
    for (int kv = 0; kv < 2; ++kv) {
        const float inv = kv ? a.inv_v : a.inv_k;
        uint32_t x[8];  // pairs of bf16
        __nv_bfloat162 top2 = __float2bfloat162_rn(0.f);
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            x[j] = (&w[2 * kv + (j >> 2)].x)[j & 3];
            top2 = __hmax2_nan(top2, __habs2(*reinterpret_cast<const __nv_bfloat162 *>(&x[j])));
        }
        const float top = __bfloat162float(__hmax_nan(__low2bfloat16(top2), __high2bfloat16(top2))) * inv;
        const uint32_t sb = top != top ? 0x7fu : e4m3_of(top / 6.f);
        const float s = e4m3_value(sb);
        const bool some = s > 0.f;  // a block below the smallest scale holds zeros, one with a NaN too
        const float inv_s = inv / s;
        uint32_t c[2] = {0, 0};
#pragma unroll
        for (int j = 0; j < 8; ++j)
            c[j >> 2] |= e2m1x2(to14bits(__uint_as_float(x[j] << 16) * inv_s),
                                to14bits(__uint_as_float(x[j] & 0xffff0000u) * inv_s))
                         << (8 * (j & 3));
        *reinterpret_cast<uint2 *>(dst + off * (D >> 1) + 8 * blk) = some ? make_uint2(c[0], c[1]) : make_uint2(0, 0);
        dst[a.ps * (D >> 1) + off * nb + blk] = (uint8_t)sb;
        dst += a.ps * (D * 9 / 16);
    }
}

// The two 16-byte words of a block's bf16 values are swapped within pairs of lanes, so that each
// store of a pair fills a 32-byte sector (41 -> 28 us at 65521 tokens, 8 heads of 64).
template <int D>
__global__ void __launch_bounds__(kKvThreads) kv4_export_kernel(const Kv4Args a, uint32_t blocks, const int32_t *slots,
                                                                const uint8_t *cache, uint4 *k, uint4 *v,
                                                                int32_t *err) {
    constexpr int nb = D >> 4;
    const uint32_t i = blockIdx.x * kKvThreads + threadIdx.x;
    if (i >= blocks) return;
    const uint32_t live = live_lanes(i, blocks);
    const bool odd = i & 1;
    const uint32_t t = i / (uint32_t)(a.Hk * nb), r = i - t * (uint32_t)(a.Hk * nb);
    const int h = (int)(r / nb), blk = (int)(r % nb);
    const int slot = slots[t], page = slot / a.ps, off = slot - page * a.ps;
    uint2 c[2] = {make_uint2(0, 0), make_uint2(0, 0)};
    uint32_t sb[2] = {0, 0};
    if (slot >= 0 && page < a.pages) {
        const uint8_t *src = cache + ((int64_t)page * a.Hk + h) * kv4_head_bytes(a.ps, D);
#pragma unroll
        for (int kv = 0; kv < 2; ++kv) {
            c[kv] = *reinterpret_cast<const uint2 *>(src + off * (D >> 1) + 8 * blk);
            sb[kv] = src[a.ps * (D >> 1) + off * nb + blk];
            src += a.ps * (D * 9 / 16);
        }
    } else if (slot >= 0) {
        report_opt(err, DEV_BAD_PAGE, (int)t, h, slot);
    }
#pragma unroll
    for (int kv = 0; kv < 2; ++kv) {
        const float s = e4m3_value(sb[kv]) * (kv ? a.v_scale : a.k_scale);
        uint4 out[2];
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const uint32_t p = e2m1x2_f16x2(((j < 4 ? c[kv].x : c[kv].y) >> (8 * (j & 3))) & 0xff);
            const float2 f = __half22float2(*reinterpret_cast<const __half2 *>(&p));
            const __nv_bfloat162 b = __floats2bfloat162_rn(f.x * s, f.y * s);
            (&out[j >> 2].x)[j & 3] = *reinterpret_cast<const uint32_t *>(&b);
        }
        const uint4 got = swap1(live, odd ? out[0] : out[1]);
        uint4 *dst = (kv ? v : k) + 2 * (int64_t)(i & ~1u) + odd;
        dst[0] = odd ? got : out[0];
        dst[2] = odd ? out[1] : got;
    }
}

// Blocks of one tensor, 0 where they are not counted in 32 bits (two tensors of 137 GB).
uint32_t blocks_of(const Kv4Args &a, int32_t tokens) {
    const int64_t n = (int64_t)tokens * a.Hk * (a.D >> 4);
    return n <= 0xffffff00LL ? (uint32_t)n : 0;
}

}  // namespace

}  // namespace rssm

extern "C" {

RSSM_API size_t rssm_kv4_cache_bytes(const rssm_kv4_config *cfg) {
    rssm::Kv4Args a;
    if (!rssm::kv4_args(cfg, &a)) return 0;
    return (size_t)a.pages * a.Hk * (size_t)rssm::kv4_head_bytes(a.ps, a.D);
}

RSSM_API rssm_status rssm_kv4_append(const rssm_kv4_config *cfg, int32_t tokens, const void *k, const void *v,
                                     const int32_t *slot_map, void *cache, int32_t *dev_error, void *stream) {
    using namespace rssm;
    Kv4Args a;
    if (!kv4_args(cfg, &a) || tokens < 1 || !k || !v || !slot_map || !cache) return RSSM_EINVAL;
    if (!aligned16(k) || !aligned16(v) || !aligned16(cache)) return RSSM_EINVAL;
    const uint32_t n = blocks_of(a, tokens);
    if (!n) return RSSM_EINVAL;
    auto kernel = a.D == 64 ? kv4_append_kernel<64> : kv4_append_kernel<128>;
    kernel<<<(n + kKvThreads - 1) / kKvThreads, kKvThreads, 0, (cudaStream_t)stream>>>(
        a, n, (const uint4 *)k, (const uint4 *)v, slot_map, (uint8_t *)cache, dev_error);
    return cudaGetLastError() == cudaSuccess ? RSSM_OK : RSSM_ECUDA;
}

RSSM_API rssm_status rssm_kv4_export(const rssm_kv4_config *cfg, int32_t tokens, const int32_t *slot_map,
                                     const void *cache, void *k, void *v, int32_t *dev_error, void *stream) {
    using namespace rssm;
    Kv4Args a;
    if (!kv4_args(cfg, &a) || tokens < 1 || !k || !v || !slot_map || !cache) return RSSM_EINVAL;
    if (!aligned16(k) || !aligned16(v) || !aligned16(cache)) return RSSM_EINVAL;
    const uint32_t n = blocks_of(a, tokens);
    if (!n) return RSSM_EINVAL;
    auto kernel = a.D == 64 ? kv4_export_kernel<64> : kv4_export_kernel<128>;
    kernel<<<(n + kKvThreads - 1) / kKvThreads, kKvThreads, 0, (cudaStream_t)stream>>>(
        a, n, slot_map, (const uint8_t *)cache, (uint4 *)k, (uint4 *)v, dev_error);
    return cudaGetLastError() == cudaSuccess ? RSSM_OK : RSSM_ECUDA;
}

}  // extern "C"
