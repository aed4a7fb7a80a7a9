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
    // chunked form, in the workspace
    int slots;       // chunks that there is room for
    int32_t *first;  // [B] slot of each request's first chunk
    uint8_t *ws;     // [slots][H] chunk operands
    int32_t *err;
};

// Chunked form on the tensor cores: N = 128, bf16 inputs, P a multiple of 8.  Its part of the workspace, and the call.
size_t gdn_chunk_bytes(int B, int H, int tokens);
cudaError_t gdn_chunk_launch(GdnPreArgs a, uint8_t *workspace, cudaStream_t st);

}  // namespace rssm
