// rssm_kv4.cu -- writing and reading back the paged 4-bit key/value cache
// (rssm_kv4_append, rssm_kv4_export).
//
// Per block of 16 channels: s = e4m3(max|x| / (6 g)), code = e2m1(x / (s g)), both
// round to nearest even and saturating, g the tensor scale.  g is a power of two, so
// x / g is exact; x is bf16 (8 significant bits) and s has 4, so neither division
// can round across a border of the narrower format (a quotient that is not on a
// border is at least 2^-12 of itself away from it, an fp32 division errs by 2^-24):
// the stored codes are those of exact arithmetic.
//
// Both kernels are bound by HBM (2 bytes in, 9/16 out per element, and the
// reverse): one thread per block, its 16 channels as two 16-byte accesses, its codes
// as one 8-byte access; 4 or 8 neighbouring threads cover a token's head.
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

// blockIdx.y: 0 keys, 1 values.  One thread per (token, head, block of 16 channels).
__global__ void __launch_bounds__(kKvThreads) kv4_append_kernel(const Kv4Args a, int64_t blocks, const uint4 *k,
                                                                const uint4 *v, const int32_t *slots,
                                                                uint8_t *cache, int32_t *err) {
    const int64_t i = (int64_t)blockIdx.x * kKvThreads + threadIdx.x;
    if (i >= blocks) return;
    const bool isv = blockIdx.y != 0;
    const int nb = a.D >> 4, per = a.Hk * nb;
    const int64_t t = i / per;
    const int r = (int)(i - t * per), h = r / nb, blk = r - h * nb;
    const int slot = slots[t];
    if (slot < 0) return;
    const int page = slot / a.ps, off = slot - page * a.ps;
    if (page >= a.pages) {
        report_opt(err, DEV_BAD_PAGE, (int)t, h, slot);
        return;
    }
    const uint4 *src = (isv ? v : k) + 2 * i;
    const uint4 w[2] = {src[0], src[1]};
    const float inv = isv ? a.inv_v : a.inv_k;
    float x[16], top = 0.f;
    bool nan = false;
#pragma unroll
    for (int j = 0; j < 16; ++j) {
        const uint32_t word = (&w[j >> 3].x)[(j >> 1) & 3];
        x[j] = bf16_bits_to_float((j & 1) ? word >> 16 : word & 0xffff) * inv;
        nan |= x[j] != x[j];
        top = fmaxf(top, fabsf(x[j]));
    }
    const uint32_t sb = nan ? 0x7fu : e4m3_of(top / 6.f);
    const float s = e4m3_value(sb);
    const bool some = s > 0.f;  // a block below the smallest scale holds zeros
    uint32_t c[2] = {0, 0};
#pragma unroll
    for (int j = 0; j < 16; j += 2)
        c[j >> 3] |= e2m1x2(some ? x[j] / s : 0.f, some ? x[j + 1] / s : 0.f) << (4 * (j & 7));
    uint8_t *dst = cache + ((int64_t)page * a.Hk + h) * kv4_head_bytes(a.ps, a.D) + (isv ? a.ps * (a.D * 9 / 16) : 0);
    *reinterpret_cast<uint2 *>(dst + off * (a.D >> 1) + 8 * blk) = make_uint2(c[0], c[1]);
    dst[a.ps * (a.D >> 1) + off * nb + blk] = (uint8_t)sb;
}

__global__ void __launch_bounds__(kKvThreads) kv4_export_kernel(const Kv4Args a, int64_t blocks, const int32_t *slots,
                                                                const uint8_t *cache, uint4 *k, uint4 *v,
                                                                int32_t *err) {
    const int64_t i = (int64_t)blockIdx.x * kKvThreads + threadIdx.x;
    if (i >= blocks) return;
    const bool isv = blockIdx.y != 0;
    const int nb = a.D >> 4, per = a.Hk * nb;
    const int64_t t = i / per;
    const int r = (int)(i - t * per), h = r / nb, blk = r - h * nb;
    const int slot = slots[t], page = slot / a.ps, off = slot - page * a.ps;
    uint4 out[2] = {make_uint4(0, 0, 0, 0), make_uint4(0, 0, 0, 0)};
    if (slot >= 0 && page < a.pages) {
        const uint8_t *src =
            cache + ((int64_t)page * a.Hk + h) * kv4_head_bytes(a.ps, a.D) + (isv ? a.ps * (a.D * 9 / 16) : 0);
        const uint2 c = *reinterpret_cast<const uint2 *>(src + off * (a.D >> 1) + 8 * blk);
        const float s = e4m3_value(src[a.ps * (a.D >> 1) + off * nb + blk]) * (isv ? a.v_scale : a.k_scale);
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const uint32_t p = e2m1x2_f16x2(((j < 4 ? c.x : c.y) >> (8 * (j & 3))) & 0xff);
            const float2 f = __half22float2(*reinterpret_cast<const __half2 *>(&p));
            const __nv_bfloat162 b = __floats2bfloat162_rn(f.x * s, f.y * s);
            (&out[j >> 2].x)[j & 3] = *reinterpret_cast<const uint32_t *>(&b);
        }
    } else if (slot >= 0) {
        report_opt(err, DEV_BAD_PAGE, (int)t, h, slot);
    }
    uint4 *dst = (isv ? v : k) + 2 * i;
    dst[0] = out[0];
    dst[1] = out[1];
}

// Blocks of one tensor, 0 where the launch would not fit a grid.
int64_t blocks_of(const Kv4Args &a, int32_t tokens) {
    const int64_t n = (int64_t)tokens * a.Hk * (a.D >> 4);
    return (n + kKvThreads - 1) / kKvThreads <= 0x7fffffffLL ? n : 0;
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
    const int64_t n = blocks_of(a, tokens);
    if (!n) return RSSM_EINVAL;
    kv4_append_kernel<<<dim3((unsigned)((n + kKvThreads - 1) / kKvThreads), 2), kKvThreads, 0, (cudaStream_t)stream>>>(
        a, n, (const uint4 *)k, (const uint4 *)v, slot_map, (uint8_t *)cache, dev_error);
    return cudaGetLastError() == cudaSuccess ? RSSM_OK : RSSM_ECUDA;
}

RSSM_API rssm_status rssm_kv4_export(const rssm_kv4_config *cfg, int32_t tokens, const int32_t *slot_map,
                                     const void *cache, void *k, void *v, int32_t *dev_error, void *stream) {
    using namespace rssm;
    Kv4Args a;
    if (!kv4_args(cfg, &a) || tokens < 1 || !k || !v || !slot_map || !cache) return RSSM_EINVAL;
    if (!aligned16(k) || !aligned16(v) || !aligned16(cache)) return RSSM_EINVAL;
    const int64_t n = blocks_of(a, tokens);
    if (!n) return RSSM_EINVAL;
    kv4_export_kernel<<<dim3((unsigned)((n + kKvThreads - 1) / kKvThreads), 2), kKvThreads, 0, (cudaStream_t)stream>>>(
        a, n, slot_map, (const uint8_t *)cache, (uint4 *)k, (uint4 *)v, dev_error);
    return cudaGetLastError() == cudaSuccess ? RSSM_OK : RSSM_ECUDA;
}

}  // extern "C"
