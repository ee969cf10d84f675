// k_fp8lin.cu -- product of E4M3 activations and an E4M3 matrix with scales of
// 128-blocks (moe_fp8_linear), one warp an output.
#include "latent_args.cuh"

namespace moe {
namespace {

__device__ __forceinline__ float4 e4m3x4(uint32_t w) {
    uint32_t lo, hi;
    asm("{ .reg .b16 a, b; mov.b32 {a, b}, %2; cvt.rn.f16x2.e4m3x2 %0, a; cvt.rn.f16x2.e4m3x2 %1, b; }"
        : "=r"(lo), "=r"(hi) : "r"(w));
    const float2 a = half_pair(lo, __half()), b = half_pair(hi, __half());
    return make_float4(a.x, a.y, b.x, b.y);
}

template <typename T>
__global__ void __launch_bounds__(256) fp8_linear_simple(MoeFp8LinearArgs a) {
    after_previous();
    const int lane = threadIdx.x & 31, nb = (a.n_in + 127) / 128;
    const int64_t i = (int64_t)blockIdx.x * 8 + (threadIdx.x >> 5);
    if (i >= (int64_t)a.n_tokens * a.n_out) return;
    const int t = (int)(i / a.n_out), o = (int)(i - (int64_t)t * a.n_out);
    const uint8_t *x = a.x8 + t * a.x_stride, *w = a.w8 + o * a.w_stride;
    float sum = 0.f;
    for (int b = 0; b < nb; ++b) {
        const int at = b * 128 + 4 * lane;
        float d = 0.f;
        if (at < a.n_in) {
            const float4 u = e4m3x4(*reinterpret_cast<const uint32_t *>(x + at));
            const float4 v = e4m3x4(*reinterpret_cast<const uint32_t *>(w + at));
            d = u.x * v.x + u.y * v.y + u.z * v.z + u.w * v.w;
        }
        sum += d * (a.x_scale[(int64_t)t * nb + b] * a.w_scale[(int64_t)(o >> 7) * nb + b]);
    }
#pragma unroll
    for (int m = 16; m; m >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, m);
    if (!lane) from_f32(sum, static_cast<T *>(a.out)[t * a.out_stride + o]);
}

}  // namespace

cudaError_t launch_fp8_linear(const MoeFp8LinearArgs &a, cudaStream_t s) {
    const void *fn = a.out_type == MOE_F32 ? (const void *)fp8_linear_simple<float>
                     : a.out_type == MOE_F16 ? (const void *)fp8_linear_simple<__half>
                                             : (const void *)fp8_linear_simple<__nv_bfloat16>;
    MoeFp8LinearArgs p = a;
    void *args[] = {&p};
    return launch_after(fn, (int)(((int64_t)a.n_tokens * a.n_out + 7) / 8), 256, 0, s, args);
}

}  // namespace moe
