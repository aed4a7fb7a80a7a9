// rssm_kv4.cuh -- byte layout of the paged 4-bit key/value cache.
//
// One page and head of `ps` tokens and D channels: K codes [ps][D/2], K block scales
// [ps][D/16], V codes, V block scales.  Keys and values of a page and head lie
// together, so that the attention kernel's reads of one page are one run of
// ps * 9/8 * D bytes.
#pragma once

#include "rssm_packed.cuh"

namespace rssm {

struct Kv4Args {
    int Hk, D, ps, pages;
    float inv_k, inv_v;  // 1 / tensor scales, exact
    float k_scale, v_scale;
};

__host__ __device__ inline int64_t kv4_head_bytes(int ps, int D) { return (int64_t)ps * D * 9 / 8; }

// Validates a cache config; false where a field is out of range.
bool kv4_args(const rssm_kv4_config *c, Kv4Args *a);

}  // namespace rssm
