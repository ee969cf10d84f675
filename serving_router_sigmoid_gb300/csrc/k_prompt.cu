// k_prompt.cu -- attention of ragged prompts over expanded keys and values
// (moe_latent_prompt): one warp a (query, head).
#include "latent_args.cuh"

namespace moe {
namespace {

template <typename T>
__global__ void __launch_bounds__(256) latent_prompt_simple(MoePromptArgs a) {
    after_previous();
    const int lane = threadIdx.x & 31;
    const int64_t w = (int64_t)blockIdx.x * 8 + (threadIdx.x >> 5);
    const int i = (int)(w / a.n_heads), h = (int)(w % a.n_heads);
    if (i >= a.n_queries) return;
    int b = 0;
    while (b < a.n_requests && a.q_start[b + 1] <= i) ++b;
    if (b == a.n_requests || i < a.q_start[b]) return;
    const int q1 = min(a.q_start[b + 1], a.n_queries), k0 = max(a.kv_start[b], 0), k1 = min(a.kv_start[b + 1], a.n_keys);
    const int end = a.causal ? min(k1, k1 - (q1 - i) + 1) : k1;
    const T *q = static_cast<const T *>(a.q) + i * a.q_stride_t + h * a.q_stride_h;
    double acc[8] = {}, l = 0;
    float m = -INFINITY;
    for (int j = k0; j < end; ++j) {
        const T *k = static_cast<const T *>(a.k) + j * a.k_stride_t + h * a.k_stride_h;
        const T *v = static_cast<const T *>(a.v) + j * a.v_stride_t + h * a.v_stride_h;
        float s = 0.f;
        for (int d = lane; d < a.nope_dim; d += 32) s += to_f32(q[d]) * to_f32(k[d]);
        for (int d = lane; d < a.rope_dim; d += 32)
            s += to_f32(q[a.nope_dim + d]) * to_f32(static_cast<const T *>(a.k_rope)[j * a.kr_stride_t + d]);
#pragma unroll
        for (int x = 16; x; x >>= 1) s += __shfl_xor_sync(0xffffffffu, s, x);
        s *= a.scale;
        const float top = fmaxf(m, s), f = __expf(m - top), p = __expf(s - top);
        m = top;
        l = l * f + p;
#pragma unroll
        for (int x = 0; x < 8; ++x)
            if (lane + 32 * x < a.v_dim) acc[x] = acc[x] * f + p * to_f32(v[lane + 32 * x]);
    }
#pragma unroll
    for (int x = 0; x < 8; ++x)
        if (lane + 32 * x < a.v_dim)
            from_f32(l > 0 ? (float)(acc[x] / l) : 0.f, static_cast<T *>(a.out)[i * a.out_stride_t + h * a.out_stride_h + lane + 32 * x]);
    if (!lane && a.lse) a.lse[(int64_t)i * a.n_heads + h] = m + logf((float)l);
}

}  // namespace

cudaError_t launch_latent_prompt(const MoePromptArgs &a, cudaStream_t s) {
    MoePromptArgs p = a;
    void *args[] = {&p};
    const void *fn = a.act_type == MOE_F16 ? (const void *)latent_prompt_simple<__half>
                                           : (const void *)latent_prompt_simple<__nv_bfloat16>;
    return launch_after(fn, (int)(((int64_t)a.n_queries * a.n_heads + 7) / 8), 256, 0, s, args);
}

}  // namespace moe
