// k_latent.cu -- attention of one new token per request over a paged cache of
// latent rows (moe_latent_decode): one block a (request, head).
#include "latent_args.cuh"

namespace moe {
namespace {

__device__ __forceinline__ float elem(const void *p, int64_t i, int type) {
    if (type == MOE_F16) return __half2float(static_cast<const __half *>(p)[i]);
    if (type == MOE_BF16) return __bfloat162float(static_cast<const __nv_bfloat16 *>(p)[i]);
    const __half_raw h = __nv_cvt_fp8_to_halfraw(static_cast<const uint8_t *>(p)[i], __NV_E4M3);
    return __half2float(__half(h));
}

__global__ void __launch_bounds__(128) latent_decode_simple(MoeLatentArgs a, MoeLatentDesc d) {
    after_previous();
    __shared__ float q[576], part[4], o_max, o_sum;
    const int h = blockIdx.x % d.n_heads, b = blockIdx.x / d.n_heads, dim = d.latent_dim + d.rope_dim, tid = threadIdx.x;
    for (int i = tid; i < dim; i += 128) q[i] = elem(a.q, b * a.q_stride_b + h * a.q_stride_h + i, a.act_type);
    const int n = min(a.seq_len[b], a.max_pages * a.page_size);
    float m = -INFINITY;
    double l = 0, acc[4] = {};
    __syncthreads();
    for (int j = 0; j < n; ++j) {
        const int page = a.block_table[b * a.table_stride + j / a.page_size];
        if (page < 0 || page >= a.n_pages) continue;
        const int64_t row = page * a.c_stride_page + (j % a.page_size) * a.c_stride_tok;
        float s = 0.f;
        for (int i = tid; i < dim; i += 128) s += q[i] * elem(a.cache, row + i, a.cache_type);
#pragma unroll
        for (int k = 16; k; k >>= 1) s += __shfl_xor_sync(0xffffffffu, s, k);
        if ((tid & 31) == 0) part[tid >> 5] = s;
        __syncthreads();
        s = (part[0] + part[1] + part[2] + part[3]) * a.scale * a.k_scale;
        const float top = fmaxf(m, s), f = __expf(m - top), p = __expf(s - top);
        m = top;
        l = l * f + p;
        for (int i = 0; i < 4; ++i)
            if (tid + 128 * i < d.latent_dim) acc[i] = acc[i] * f + p * elem(a.cache, row + tid + 128 * i, a.cache_type);
        __syncthreads();
    }
    for (int i = 0; i < 4; ++i) {
        if (tid + 128 * i >= d.latent_dim) continue;
        const int64_t at = b * a.out_stride_b + h * a.out_stride_h + tid + 128 * i;
        const float v = l > 0 ? (float)(acc[i] / l) * a.k_scale : 0.f;
        if (a.act_type == MOE_F16) static_cast<__half *>(a.out)[at] = __float2half_rn(v);
        else static_cast<__nv_bfloat16 *>(a.out)[at] = __float2bfloat16_rn(v);
    }
    if (!tid && a.lse) a.lse[b * d.n_heads + h] = m + logf((float)l);
}

}  // namespace

cudaError_t latent_prepare(const MoeLatentDesc &, int, size_t *bytes) {
    *bytes = 0;
    return cudaSuccess;
}

cudaError_t launch_latent_decode(const LatentHandle &h, const MoeLatentArgs &a, cudaStream_t s) {
    MoeLatentArgs p = a;
    MoeLatentDesc d = h.d;
    void *args[] = {&p, &d};
    return launch_after((const void *)latent_decode_simple, a.n_requests * d.n_heads, 128, 0, s, args);
}

}  // namespace moe
