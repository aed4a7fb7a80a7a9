// rssm_gdn_prefill.h -- arguments and launchers of the packed gated delta rule.
#pragma once

#include <cuda_runtime.h>
#include <stddef.h>
#include <stdint.h>

namespace rssm {

constexpr int kGdnChunk = 64;

// Requests of up to this many tokens are left to the recurrence where there is a chunked form.  Its time is the tokens'
// chain; in chunks a request is one wave of large CTAs however short it is.  64 equal prompts, 32 heads of 128 x 128 (us):
// 1 token 65 against 179, 8 tokens 132 against 184, 16 tokens 189 against 186, 32 tokens 366 against 193.  (With fewer heads
// and requests than fill the machine the chain is ahead for longer; 12 is for a full one.)
constexpr int kGdnShort = 12;

struct GdnPreArgs {
    int B, H, P, tokens;
    const void *q, *k, *v;      // [tokens][H][N], [tokens][H][N], [tokens][H][P]
    const float *alpha, *beta;  // [tokens][H]
    const int32_t *cu;          // [B + 1]
    const float *S0;            // [B][H][P][N] or nullptr
    float *y, *S_out;
    // chunked form, in the workspace
    int slots;      // chunks that there is room for
    int32_t *plan;  // rssm_gdn_plan.cuh
    uint8_t *ws;    // [slots][H] chunk operands
    int32_t *err;
};

// A launch whose CTAs may start once those of the kernel before have all started or ended (pdl_trigger).
inline cudaError_t launch_early(void (*kernel)(GdnPreArgs), dim3 grid, int threads, size_t smem, const GdnPreArgs &a, cudaStream_t st) {
    cudaLaunchConfig_t cfg{};
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.gridDim = grid;
    cfg.blockDim = dim3(threads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = st;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kernel, a);
}

// Recurrent form, of every request or, behind the chunked form (a.plan is set), of the short ones.
template <typename IN> cudaError_t gdn_recurrent_launch(const GdnPreArgs &a, int N, cudaStream_t st);

// Chunked form on the tensor cores: N = 128, bf16 inputs, P a multiple of 8.  Its workspace, and the call, which serves
// the short requests by the recurrent form.
size_t gdn_chunk_bytes(int B, int H, int tokens);
cudaError_t gdn_chunk_launch(GdnPreArgs a, uint8_t *workspace, cudaStream_t st);

}  // namespace rssm
