// latent_args.cuh -- handles and launchers of the FP8 products and the latent
// attention (moe_quant_act_fp8, moe_fp8_linear, moe_latent_*).  Internal.
#pragma once

#include "attn_args.cuh"

namespace moe {

// What a latent attention handle holds; part: the pieces of requests that
// blocks share.
struct LatentHandle {
    uint32_t magic;
    int device, num_sms;
    MoeLatentDesc d;
    float *part;
};

cudaError_t launch_quant_act_fp8(const void *x, int act_type, int64_t x_stride, int n_tokens, int dim, uint8_t *x8,
                                 int64_t x8_stride, float *scale, cudaStream_t s);
cudaError_t launch_fp8_linear(const MoeFp8LinearArgs &a, cudaStream_t s);
// Bytes of a handle's workspace; sets the kernels' attributes.
cudaError_t latent_prepare(const MoeLatentDesc &d, int num_sms, size_t *bytes);
cudaError_t launch_latent_decode(const LatentHandle &h, const MoeLatentArgs &a, cudaStream_t s);
cudaError_t launch_latent_prompt(const MoePromptArgs &a, cudaStream_t s);
// The flags that a file's kernels left on the current device, read and cleared.
cudaError_t fp8_linear_flags(int32_t *out);
cudaError_t latent_decode_flags(int32_t *out);
cudaError_t latent_prompt_flags(int32_t *out);

}  // namespace moe
