// k_attn.cu -- attention of one new token per request over the paged cache
// (moe_attn_decode): one block per query head, its warps take the tokens in
// turn with a running maximum and sum each, joined in shared memory.
#include "attn_args.cuh"

namespace moe {
namespace {

constexpr int kWarps = 8;
constexpr int kMaxHeadDim = 256;

template <int CT>
__device__ __forceinline__ float cached(const void *p, int64_t i) {
    if constexpr (CT == MOE_E4M3) {
        const uint32_t h = e4m3x2_to_f16x2(static_cast<const uint8_t *>(p)[i]);
        return __half2float(__ushort_as_half((unsigned short)(h & 0xFFFFu)));
    } else {
        return to_f32(static_cast<const typename Elem<CT>::type *>(p)[i]);
    }
}

__device__ __forceinline__ float act_at(const void *p, int type, int64_t i) {
    return type == MOE_F32   ? static_cast<const float *>(p)[i]
           : type == MOE_F16 ? __half2float(static_cast<const __half *>(p)[i])
                             : __bfloat162float(static_cast<const __nv_bfloat16 *>(p)[i]);
}

template <int CT>
__global__ void __launch_bounds__(32 * kWarps) attn_decode_kernel(const __grid_constant__ MoeAttnArgs a,
                                                                  const __grid_constant__ MoeAttnDesc d) {
    __shared__ float s_o[kWarps][kMaxHeadDim];
    __shared__ float s_m[kWarps], s_l[kWarps];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int b = blockIdx.x / d.n_heads, h = blockIdx.x - b * d.n_heads, kh = h / (d.n_heads / d.n_kv_heads);
    const long long cap = (long long)a.max_pages * a.page_size;
    const int len = (int)min((long long)max(a.seq_len[b], 0), cap);
    const int from = a.window > 0 ? max(0, len - a.window) : 0;
    float q[8], o[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const int e = lane + 32 * i;
        q[i] = e < d.k_dim ? act_at(a.q, a.act_type, b * a.q_stride_b + h * a.q_stride_h + e) : 0.f;
        o[i] = 0.f;
    }
    float m = -INFINITY, l = 0.f;
    for (int t = from + warp; t < len; t += kWarps) {
        const int col = t / a.page_size;
        const int page = a.block_table[b * a.table_stride + col];
        if (page < 0 || page >= a.n_pages) continue;
        const int at = t - col * a.page_size;
        const int64_t ko = page * a.kc_stride_page + at * a.kc_stride_tok + kh * a.kc_stride_head;
        const int64_t vo = page * a.vc_stride_page + at * a.vc_stride_tok + kh * a.vc_stride_head;
        float s = 0.f;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const int e = lane + 32 * i;
            if (e < d.k_dim) s = fmaf(q[i], cached<CT>(a.k_cache, ko + e), s);
        }
        s = warp_sum_f(s) * (a.scale * a.k_scale);
        const float mn = fmaxf(m, s);
        const float f = expf(m - mn), p = expf(s - mn);
        m = mn;
        l = l * f + p;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const int e = lane + 32 * i;
            if (e < d.v_dim) o[i] = fmaf(p, cached<CT>(a.v_cache, vo + e), o[i] * f);
        }
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) s_o[warp][lane + 32 * i] = o[i];
    if (lane == 0) s_m[warp] = m, s_l[warp] = l;
    __syncthreads();
    float top = -INFINITY, total = 0.f;
    for (int w = 0; w < kWarps; ++w) top = fmaxf(top, s_m[w]);
    for (int w = 0; w < kWarps; ++w)
        if (s_l[w] > 0.f) total += s_l[w] * expf(s_m[w] - top);
    for (int e = threadIdx.x; e < d.v_dim; e += 32 * kWarps) {
        float r = 0.f;
        for (int w = 0; w < kWarps; ++w)
            if (s_l[w] > 0.f) r += s_o[w][e] * expf(s_m[w] - top);
        r = total > 0.f ? r / total * a.v_scale : 0.f;
        const int64_t at = b * a.out_stride_b + h * a.out_stride_h + e;
        if (a.act_type == MOE_F32) static_cast<float *>(a.out)[at] = r;
        else if (a.act_type == MOE_F16) static_cast<__half *>(a.out)[at] = __float2half_rn(r);
        else static_cast<__nv_bfloat16 *>(a.out)[at] = __float2bfloat16_rn(r);
    }
    if (a.lse && threadIdx.x == 0) a.lse[(int64_t)b * d.n_heads + h] = total > 0.f ? top + logf(total) : -INFINITY;
}

}  // namespace

cudaError_t launch_attn_decode(const AttnHandle &h, const MoeAttnArgs &a, cudaStream_t s) {
    const int grid = a.n_requests * h.d.n_heads;
    switch (a.cache_type) {
        case MOE_F16: attn_decode_kernel<MOE_F16><<<grid, 32 * kWarps, 0, s>>>(a, h.d); break;
        case MOE_BF16: attn_decode_kernel<MOE_BF16><<<grid, 32 * kWarps, 0, s>>>(a, h.d); break;
        default: attn_decode_kernel<MOE_E4M3><<<grid, 32 * kWarps, 0, s>>>(a, h.d); break;
    }
    return cudaGetLastError();
}

}  // namespace moe
