// rssm_gdn_prefill.h -- arguments and launchers of the packed gated delta rule.
#pragma once

#include <cuda_runtime.h>
#include <stddef.h>
#include <stdint.h>

namespace rssm {

struct GdnPreArgs {
    int B, H, P, tokens;
    const void *q, *k, *v;      // [tokens][H][N], [tokens][H][N], [tokens][H][P]
    const float *alpha, *beta;  // [tokens][H]
    const int32_t *cu;          // [B + 1]
    const float *S0;            // [B][H][P][N] or nullptr
    float *y, *S_out;
    uint8_t *ws;  // chunk operands (chunked form)
    int32_t *err;
};

// Chunked form on the tensor cores: N = 128, bf16 inputs, P a multiple of 64.
size_t gdn_chunk_bytes(int B, int H, int tokens);
cudaError_t gdn_chunk_launch(const GdnPreArgs &a, cudaStream_t st);

}  // namespace rssm
