// k_actq8.cu -- activation rows as E4M3 codes with one scale for each 128
// elements (moe_quant_act_fp8):
//   s = max(max |x| / 448, 1e-12),  code = E4M3(x / s), nearest, ties to even
//
// HBM is its floor: x in, a byte an element out.  Measured 9.3 us for 2048 x 6144 in 16 bits
// (38 MB, 4.1 TB/s; 8.6 with x in L2): one load in flight a thread, then 16 divisions, which
// take half of the issue slots; neither is full.  A thread takes 16 elements (64 or
// 32 bytes in, 16 out), eight neighbouring lanes a group of 128, whose maximum
// takes three shuffles.  The divisions are IEEE ones, so codes and scales equal
// those of the formula bit for bit.
#include "latent_args.cuh"

namespace moe {
namespace {

constexpr int kThreads = 256;

// The larger one, NaN if either is: the formula's maximum.
__device__ __forceinline__ float max_nan(float a, float b) {
    float r;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
    return r;
}

template <typename T>
__global__ void __launch_bounds__(kThreads) quant_fp8_kernel(const T *x, int64_t x_stride, int dim, FastDiv by_row,
                                                             uint32_t units, uint8_t *x8, int64_t x8_stride,
                                                             float *scale) {
    after_previous();
    // units of 16 elements, 8 a group, groups of a row one after another
    const uint32_t u = blockIdx.x * kThreads + threadIdx.x;
    if ((u & ~7u) >= units) return;  // a group's lanes leave together
    const uint32_t t = by_row.div(u), at = (u - t * by_row.d) * 16;
    const bool live = at < (uint32_t)dim;
    float v[16], top = 0.f;
    if (live) load_vec<16>(x + (int64_t)t * x_stride + at, v);
#pragma unroll
    for (int i = 0; i < 16; ++i) {
        if (!live) v[i] = 0.f;
        top = max_nan(top, fabsf(v[i]));
    }
#pragma unroll
    for (int m = 4; m; m >>= 1) top = max_nan(top, __shfl_xor_sync(0xffu << (threadIdx.x & 24), top, m));
    const float s = max_nan(__fdiv_rn(top, 448.f), 1e-12f);
    if (live) {
        uint32_t w[4];
#pragma unroll
        for (int i = 0; i < 4; ++i)
            w[i] = f32x2_to_e4m3x2(__fdiv_rn(v[4 * i], s), __fdiv_rn(v[4 * i + 1], s)) |
                   f32x2_to_e4m3x2(__fdiv_rn(v[4 * i + 2], s), __fdiv_rn(v[4 * i + 3], s)) << 16;
        *reinterpret_cast<uint4 *>(x8 + (int64_t)t * x8_stride + at) = make_uint4(w[0], w[1], w[2], w[3]);
    }
    if (!(u & 7)) scale[u >> 3] = s;  // a row's groups follow one another, and rows do
}

template <typename T>
cudaError_t launch(const void *x, int64_t x_stride, int n, int dim, uint8_t *x8, int64_t x8_stride, float *scale,
                   cudaStream_t s) {
    const T *xp = static_cast<const T *>(x);
    const uint32_t row = (uint32_t)(dim + 127) / 128 * 8;
    // units are counted in 31 bits: a launch takes what fits
    const int64_t most = (1u << 30) / row;
    for (int64_t t0 = 0; t0 < n; t0 += most) {  // in 64 bits: the last step may pass 2^31
        const int64_t m = n - t0 < most ? n - t0 : most;
        const T *xt = xp + t0 * x_stride;
        uint8_t *ot = x8 + t0 * x8_stride;
        float *st = scale + t0 * (row / 8);
        FastDiv by_row(row);
        uint32_t units = (uint32_t)m * row;
        void *args[] = {&xt, &x_stride, &dim, &by_row, &units, &ot, &x8_stride, &st};
        const cudaError_t e = launch_after(reinterpret_cast<const void *>(quant_fp8_kernel<T>),
                                           (int)((units + kThreads - 1) / kThreads), kThreads, 0, s, args);
        if (e != cudaSuccess) return e;
    }
    return cudaSuccess;
}

}  // namespace

cudaError_t launch_quant_act_fp8(const void *x, int act_type, int64_t x_stride, int n_tokens, int dim, uint8_t *x8,
                                 int64_t x8_stride, float *scale, cudaStream_t s) {
    switch (act_type) {
        case MOE_F32: return launch<float>(x, x_stride, n_tokens, dim, x8, x8_stride, scale, s);
        case MOE_F16: return launch<__half>(x, x_stride, n_tokens, dim, x8, x8_stride, scale, s);
        default: return launch<__nv_bfloat16>(x, x_stride, n_tokens, dim, x8, x8_stride, scale, s);
    }
}

}  // namespace moe
