// k_norm.cu -- the join between two blocks of a layer (moe_block_norm): the
// norm after a block, its gate and scale, the residual add and the norm before
// the next block in one pass.
//
//   u = y * rsqrt(mean(y^2) + eps) * w_post;  r = alpha x + beta act(g) u
//   n = r * rsqrt(mean(r^2) + eps) * w_pre
//
// Bound by HBM (each array once): a block holds one row in registers, so the
// two sums over the row (each a warp reduction and one barrier) need no second
// read.  Sums of squares and everything between are fp32; out and normed are
// rounded once, normed from the unrounded r.
#include "attn_args.cuh"

namespace moe {
namespace {

__device__ __forceinline__ float block_sum(float v, float *red, int nw) {
    v = warp_sum_f(v);
    if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = v;
    __syncthreads();
    float r = 0.f;
    for (int w = 0; w < nw; ++w) r += red[w];
    return r;
}

// V elements per access (8 or 4: aligned 16-byte pieces, 1: any alignment),
// M accesses per thread.
template <int DT, int V, int M>
__global__ void __launch_bounds__(V == 8 ? 512 : 1024) block_norm_kernel(const __grid_constant__ MoeNormArgs a) {
    using A = typename Elem<DT>::type;
    __shared__ float red[2][32];
    const int nw = blockDim.x >> 5;
    const int64_t t = blockIdx.x;
    const A *x = static_cast<const A *>(a.x) + t * a.x_stride;
    const A *y = a.y ? static_cast<const A *>(a.y) + t * a.y_stride : nullptr;
    const A *g = a.gate ? static_cast<const A *>(a.gate) + t * a.gate_stride_t : nullptr;
    A *out = static_cast<A *>(a.out) + t * a.out_stride;
    A *nrm = a.normed ? static_cast<A *>(a.normed) + t * a.normed_stride : nullptr;

    auto ld = [](const A *p, float(&v)[V]) {
        if constexpr (V == 1) v[0] = to_f32(*p);
        else load_vec(p, v);
    };
    auto ldw = [](const float *p, float(&v)[V]) {
#pragma unroll
        for (int j = 0; j < V; ++j) v[j] = __ldg(p + j);
    };
    auto st = [](A *p, const float(&v)[V]) {
        if constexpr (V == 1) from_f32(v[0], *p);
        else store_vec(p, v);
    };

    float r[M][V], u[M][V];
    float sq = 0.f;
#pragma unroll
    for (int m = 0; m < M; ++m) {
        const int d = (m * blockDim.x + threadIdx.x) * V;
#pragma unroll
        for (int j = 0; j < V; ++j) r[m][j] = u[m][j] = 0.f;
        if (d < a.dim) {
            ld(x + d, r[m]);
            if (y) ld(y + d, u[m]);
        }
    }
    float post = 1.f;
    if (y && a.w_post) {
#pragma unroll
        for (int m = 0; m < M; ++m)
#pragma unroll
            for (int j = 0; j < V; ++j) sq = fmaf(u[m][j], u[m][j], sq);
        post = rsqrtf(block_sum(sq, red[0], nw) / (float)a.dim + a.eps);
    }
    const float g1 = g && a.gate_stride_d == 0 ? to_f32(*g) : 1.f;
    sq = 0.f;
#pragma unroll
    for (int m = 0; m < M; ++m) {
        const int d = (m * blockDim.x + threadIdx.x) * V;
        if (d >= a.dim) continue;
        if (y) {
            float f[V];
#pragma unroll
            for (int j = 0; j < V; ++j) f[j] = g1;
            if (g && a.gate_stride_d) ld(g + d, f);
            if (g && a.gate_sigmoid)
#pragma unroll
                for (int j = 0; j < V; ++j) f[j] = __fdiv_rn(1.f, 1.f + expf(-f[j]));
            if (a.w_post) {
                float w[V];
                ldw(a.w_post + d, w);
#pragma unroll
                for (int j = 0; j < V; ++j) u[m][j] *= post * w[j];
            }
#pragma unroll
            for (int j = 0; j < V; ++j) r[m][j] = fmaf(a.beta * f[j], u[m][j], a.alpha * r[m][j]);
        } else {
#pragma unroll
            for (int j = 0; j < V; ++j) r[m][j] *= a.alpha;
        }
#pragma unroll
        for (int j = 0; j < V; ++j) sq = fmaf(r[m][j], r[m][j], sq);
        st(out + d, r[m]);
    }
    if (!nrm) return;
    const float pre = rsqrtf(block_sum(sq, red[1], nw) / (float)a.dim + a.eps);
#pragma unroll
    for (int m = 0; m < M; ++m) {
        const int d = (m * blockDim.x + threadIdx.x) * V;
        if (d >= a.dim) continue;
        float w[V];
#pragma unroll
        for (int j = 0; j < V; ++j) w[j] = 1.f;
        if (a.w_pre) ldw(a.w_pre + d, w);
#pragma unroll
        for (int j = 0; j < V; ++j) r[m][j] *= pre * w[j];
        st(nrm + d, r[m]);
    }
}

template <int DT, int V>
cudaError_t launch(const MoeNormArgs &a, cudaStream_t s) {
    // accesses per thread: as few as 512 threads allow, then 1024 threads
    const int acc = (a.dim + V - 1) / V;
    int m = 1;
    while (m < 16 && acc > m * (m < 4 ? 512 : 1024)) m *= 2;
    int threads = ((acc + m - 1) / m + 31) / 32 * 32;
    switch (m) {
        case 1: block_norm_kernel<DT, V, 1><<<a.n_tokens, threads, 0, s>>>(a); break;
        case 2: block_norm_kernel<DT, V, 2><<<a.n_tokens, threads, 0, s>>>(a); break;
        case 4: block_norm_kernel<DT, V, 4><<<a.n_tokens, threads, 0, s>>>(a); break;
        default:
            if constexpr (V == 1) {
                if (m == 8) block_norm_kernel<DT, V, 8><<<a.n_tokens, threads, 0, s>>>(a);
                else block_norm_kernel<DT, V, 16><<<a.n_tokens, threads, 0, s>>>(a);
            }
    }
    return cudaGetLastError();
}

template <int DT>
cudaError_t launch_dt(const MoeNormArgs &a, cudaStream_t s) {
    constexpr int V = DT == MOE_F32 ? 4 : 8;
    const auto on = [](const void *p, int64_t stride) {
        return reinterpret_cast<uintptr_t>(p) % 16 == 0 && stride % V == 0;
    };
    const bool vec = a.dim % V == 0 && on(a.x, a.x_stride) && on(a.y, a.y ? a.y_stride : 0) &&
                     on(a.out, a.out_stride) && on(a.normed, a.normed ? a.normed_stride : 0) &&
                     on(a.w_post, 0) && on(a.w_pre, 0) &&
                     (!a.gate || a.gate_stride_d == 0 || on(a.gate, a.gate_stride_t));
    return vec ? launch<DT, V>(a, s) : launch<DT, 1>(a, s);
}

}  // namespace

cudaError_t launch_block_norm(const MoeNormArgs &a, cudaStream_t s) {
    switch (a.act_type) {
        case MOE_F32: return launch_dt<MOE_F32>(a, s);
        case MOE_F16: return launch_dt<MOE_F16>(a, s);
        default: return launch_dt<MOE_BF16>(a, s);
    }
}

}  // namespace moe
