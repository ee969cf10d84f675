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
// rounded once, normed from the unrounded r.  2048 rows of 6144 fp32 with a full
// gate: 41 us, 6.2 TB/s; one row: 2.8 us.
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

// 1 / (1 + e^-x), within 6 ulp; for 16-bit types with the fast exponential,
// whose error (2^-22 and 2^-23 |x|) their rounding hides.
template <int DT>
__device__ __forceinline__ float sigmoid(float x) {
    return __fdividef(1.f, 1.f + (DT == MOE_F32 ? expf(-x) : __expf(-x)));
}

// V elements per access (8 or 4: aligned 16-byte pieces, 1: any alignment),
// M accesses per thread.
template <int DT, int V, int M, bool EARLY>
__global__ void __launch_bounds__(V == 1 ? 1024 : 512, EARLY || V == 1 ? 1 : V * M == 8 ? 3 : V * M == 16 ? 2 : 1)
    block_norm_kernel(const __grid_constant__ MoeNormArgs a) {
    using A = typename Elem<DT>::type;
    __shared__ float red[2][32];
    after_previous();
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
        for (int j = 0; j < V; j += V == 1 ? 1 : 4) {
            if constexpr (V == 1) {
                v[j] = ld_in(p + j);
            } else {
                const float4 w = ld_in4(p + j);
                v[j] = w.x; v[j + 1] = w.y; v[j + 2] = w.z; v[j + 3] = w.w;
            }
        }
    };
    auto st = [](A *p, const float(&v)[V]) {
        if constexpr (V == 1) from_f32(v[0], *p);
        else store_vec(p, v);
    };

    float u[M][V];               // the block's output, then r
    uint4 xr[V == 1 ? 1 : M];    // the residual stream as loaded
    float x1[V == 1 ? M : 1];
    auto ldx = [&](int m, int d) {
        if constexpr (V == 1) x1[m] = to_f32(x[d]);
        else xr[m] = ld_once16(x + d);
    };
    auto getx = [&](int m, float(&v)[V]) {
        if constexpr (V == 1) {
            v[0] = x1[m];
        } else {
            const uint32_t w[4] = {xr[m].x, xr[m].y, xr[m].z, xr[m].w};
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                if constexpr (V == 4) {
                    v[j] = __uint_as_float(w[j]);
                } else {
                    const float2 f = half_pair(w[j], A());
                    v[2 * j] = f.x;
                    v[2 * j + 1] = f.y;
                }
            }
        }
    };
    float wp[EARLY ? M : 1][V], wn[EARLY ? M : 1][V];
    auto weights = [&](const float *w, float(&v)[V], int d) {
#pragma unroll
        for (int j = 0; j < V; ++j) v[j] = 1.f;
        if (w && d < a.dim) ldw(w + d, v);
    };
    float sq = 0.f;
    const float g1 = g && a.gate_stride_d == 0 ? to_f32(*g) : 1.f;
    {
        float f[M][V];
#pragma unroll
        for (int m = 0; m < M; ++m) {
            const int d = (m * blockDim.x + threadIdx.x) * V;
#pragma unroll
            for (int j = 0; j < V; ++j) u[m][j] = 0.f, f[m][j] = g1;
            if (d < a.dim) {
                if (y) ld(y + d, u[m]);
                if (g && a.gate_stride_d) ld(g + d, f[m]);
                if (EARLY) ldx(m, d);
            }
            if constexpr (EARLY) {
                weights(a.w_post, wp[m], d);
                weights(nrm ? a.w_pre : nullptr, wn[m], d);
            }
        }
        // u takes gate and weight before its norm is known: what waits for the
        // sum is one factor
#pragma unroll
        for (int m = 0; m < M; ++m) {
            const int d = (m * blockDim.x + threadIdx.x) * V;
#pragma unroll
            for (int j = 0; j < V; ++j) sq = fmaf(u[m][j], u[m][j], sq);
            if (g && a.gate_sigmoid) {
#pragma unroll
                for (int j = 0; j < V; ++j) f[m][j] = sigmoid<DT>(f[m][j]);
            }
            float(&w)[V] = wp[EARLY ? m : 0];
            if constexpr (!EARLY) weights(a.w_post, w, d);
#pragma unroll
            for (int j = 0; j < V; ++j) u[m][j] *= f[m][j] * w[j];
        }
    }
    if constexpr (!EARLY) {
#pragma unroll
        for (int m = 0; m < M; ++m) {
            const int d = (m * blockDim.x + threadIdx.x) * V;
            if (d < a.dim) ldx(m, d);
        }
    }
    float post = a.beta;
    if (y && a.w_post) post *= rsqrtf(block_sum(sq, red[0], nw) / (float)a.dim + a.eps);
    sq = 0.f;
#pragma unroll
    for (int m = 0; m < M; ++m) {
        const int d = (m * blockDim.x + threadIdx.x) * V;
        if (d >= a.dim) continue;
        float v[V];
        getx(m, v);
#pragma unroll
        for (int j = 0; j < V; ++j) {
            u[m][j] = fmaf(post, u[m][j], a.alpha * v[j]);
            sq = fmaf(u[m][j], u[m][j], sq);
        }
        st(out + d, u[m]);
    }
    if (!nrm) return;
    const float pre = rsqrtf(block_sum(sq, red[1], nw) / (float)a.dim + a.eps);
#pragma unroll
    for (int m = 0; m < M; ++m) {
        const int d = (m * blockDim.x + threadIdx.x) * V;
        if (d >= a.dim) continue;
        float(&w)[V] = wn[EARLY ? m : 0];
        if constexpr (!EARLY) weights(a.w_pre, w, d);
#pragma unroll
        for (int j = 0; j < V; ++j) u[m][j] *= pre * w[j];
        st(nrm + d, u[m]);
    }
}

__device__ __forceinline__ void copy16(void *smem, const void *gmem) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"((uint32_t)__cvta_generic_to_shared(smem)), "l"(gmem)
                 : "memory");
}

// The same for many long rows: one block per SM goes through rows blockIdx,
// + gridDim, ...; a ring of row copies in shared memory keeps `stages` - 1 rows
// on their way while one is computed.  A thread copies just the pieces it will
// read, so its own wait_group is all the ring needs.  Both weights stay in
// registers (of four 16-bit pieces a thread, dim > 12288, some 18 of the 64
// spill: 1216 x 16384 bf16 49 us against 63 with a block a row).
constexpr int kRing = 220 * 1024;
template <int DT, int M>
__global__ void __launch_bounds__(512, 1)
    block_norm_ring_kernel(const __grid_constant__ MoeNormArgs a, int stages) {
    using A = typename Elem<DT>::type;
    constexpr int V = DT == MOE_F32 ? 4 : 8;
    extern __shared__ __align__(16) uint4 ring[];
    __shared__ float red[2][32];
    after_previous();
    const int nw = blockDim.x >> 5, n_arr = 1 + (a.y != nullptr) + (a.gate != nullptr && a.gate_stride_d != 0);
    auto slot = [&](int st, int arr, int m) -> uint4 & {
        return ring[((st * n_arr + arr) * M + m) * blockDim.x + threadIdx.x];
    };
    auto fetch = [&](int64_t t, int st) {
        if (t < a.n_tokens) {
#pragma unroll
            for (int m = 0; m < M; ++m) {
                const int d = (m * blockDim.x + threadIdx.x) * V;
                if (d >= a.dim) continue;
                copy16(&slot(st, 0, m), static_cast<const A *>(a.x) + t * a.x_stride + d);
                if (a.y) copy16(&slot(st, 1, m), static_cast<const A *>(a.y) + t * a.y_stride + d);
                if (n_arr == 3) copy16(&slot(st, 2, m), static_cast<const A *>(a.gate) + t * a.gate_stride_t + d);
            }
        }
        asm volatile("cp.async.commit_group;" ::: "memory");
    };
    auto get = [&](int st, int arr, int m, float(&v)[V]) {
        const uint4 w = slot(st, arr, m);
        const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            if constexpr (V == 4) {
                v[j] = __uint_as_float(u[j]);
            } else {
                const float2 f = half_pair(u[j], A());
                v[2 * j] = f.x;
                v[2 * j + 1] = f.y;
            }
        }
    };
    // three copies ahead at most: wait_group takes a constant
    for (int i = 0; i < stages - 1; ++i) fetch(blockIdx.x + (int64_t)i * gridDim.x, i);
    float wp[M][V], wn[M][V];
#pragma unroll
    for (int m = 0; m < M; ++m) {
        const int d = (m * blockDim.x + threadIdx.x) * V;
#pragma unroll
        for (int j = 0; j < V; j += 4) {
            float4 p = make_float4(1.f, 1.f, 1.f, 1.f), n = p;
            if (a.w_post && d < a.dim) p = ld_in4(a.w_post + d + j);
            if (a.w_pre && d < a.dim) n = ld_in4(a.w_pre + d + j);
            wp[m][j] = p.x; wp[m][j + 1] = p.y; wp[m][j + 2] = p.z; wp[m][j + 3] = p.w;
            wn[m][j] = n.x; wn[m][j + 1] = n.y; wn[m][j + 2] = n.z; wn[m][j + 3] = n.w;
        }
    }
    int st = 0;
    for (int64_t t = blockIdx.x; t < a.n_tokens; t += gridDim.x) {
        const float g1 = a.gate && a.gate_stride_d == 0
                             ? to_f32(static_cast<const A *>(a.gate)[t * a.gate_stride_t]) : 1.f;
        if (stages == 2) asm volatile("cp.async.wait_group 0;" ::: "memory");
        else if (stages == 3) asm volatile("cp.async.wait_group 1;" ::: "memory");
        else asm volatile("cp.async.wait_group 2;" ::: "memory");
        float u[M][V], r[M][V];
        float sq = 0.f;
#pragma unroll
        for (int m = 0; m < M; ++m) {
            const int d = (m * blockDim.x + threadIdx.x) * V;
            float f[V];
#pragma unroll
            for (int j = 0; j < V; ++j) u[m][j] = r[m][j] = 0.f, f[j] = g1;
            if (d < a.dim) {
                get(st, 0, m, r[m]);
                if (a.y) get(st, 1, m, u[m]);
                if (n_arr == 3) get(st, 2, m, f);
            }
#pragma unroll
            for (int j = 0; j < V; ++j) {
                sq = fmaf(u[m][j], u[m][j], sq);
                if (a.gate && a.gate_sigmoid) f[j] = sigmoid<DT>(f[j]);
                u[m][j] *= f[j] * wp[m][j];
            }
        }
        // this thread's pieces are read: the next row into the slot behind
        fetch(t + (int64_t)(stages - 1) * gridDim.x, st == 0 ? stages - 1 : st - 1);
        st = st + 1 == stages ? 0 : st + 1;
        float post = a.beta;
        if (a.y && a.w_post) post *= rsqrtf(block_sum(sq, red[0], nw) / (float)a.dim + a.eps);
        sq = 0.f;
#pragma unroll
        for (int m = 0; m < M; ++m) {
            const int d = (m * blockDim.x + threadIdx.x) * V;
#pragma unroll
            for (int j = 0; j < V; ++j) {
                r[m][j] = fmaf(post, u[m][j], a.alpha * r[m][j]);
                sq = fmaf(r[m][j], r[m][j], sq);
            }
            if (d < a.dim) store_vec(static_cast<A *>(a.out) + t * a.out_stride + d, r[m]);
        }
        if (a.normed) {
            const float pre = rsqrtf(block_sum(sq, red[1], nw) / (float)a.dim + a.eps);
#pragma unroll
            for (int m = 0; m < M; ++m) {
                const int d = (m * blockDim.x + threadIdx.x) * V;
#pragma unroll
                for (int j = 0; j < V; ++j) r[m][j] *= pre * wn[m][j];
                if (d < a.dim) store_vec(static_cast<A *>(a.normed) + t * a.normed_stride + d, r[m]);
            }
        }
        if (!a.normed || !(a.y && a.w_post)) __syncthreads();  // red is written again by the next row
    }
}

template <int DT, int M>
cudaError_t launch_ring(const MoeNormArgs &a, int threads, int stages, size_t smem, int num_sms, cudaStream_t s) {
    const cudaError_t ce = cudaFuncSetAttribute(block_norm_ring_kernel<DT, M>,
                                                cudaFuncAttributeMaxDynamicSharedMemorySize, kRing);
    if (ce != cudaSuccess) return ce;
    void *args[] = {const_cast<MoeNormArgs *>(&a), &stages};
    return launch_after(reinterpret_cast<const void *>(block_norm_ring_kernel<DT, M>), num_sms, threads, smem, s, args);
}

// One block a row, m accesses a thread.
template <int DT, int V, bool EARLY>
cudaError_t launch_rows(const MoeNormArgs &a, int m, int threads, cudaStream_t s) {
    void (*fn)(MoeNormArgs) = nullptr;
    switch (m) {
        case 1: fn = block_norm_kernel<DT, V, 1, EARLY>; break;
        case 2: fn = block_norm_kernel<DT, V, 2, EARLY>; break;
        case 4:
            if constexpr (!EARLY || V == 4) fn = block_norm_kernel<DT, V, 4, EARLY>;
            break;
        case 8:
            if constexpr (!EARLY && V <= 4) fn = block_norm_kernel<DT, V, 8, EARLY>;
            break;
        default:
            if constexpr (V == 1) fn = block_norm_kernel<DT, V, 16, EARLY>;
    }
    void *args[] = {const_cast<MoeNormArgs *>(&a)};
    return launch_after(reinterpret_cast<const void *>(fn), a.n_tokens, threads, 0, s, args);
}

// The form of the kernel, from sizes alone.  Measured on fp32 / bf16 rows with
// a full gate (us):
//   weights early     152 x 6144: 5.2 / 3.8 against 5.7 / 4.2, 608 x 4096: 9.7 /
//                     7.5 against 9.7 / 8.1; but 4096 x 4096 bf16: 43.6 against
//                     36.9 and 304 x 6144: 9.2 / 7.5 against 7.5 / 5.9 (registers:
//                     fewer rows an SM); so by the rows an SM, the fewer the more
//                     registers the weights take
//   ring of copies    from 8 rows an SM, where a block a row is few rows an SM
//                     (registers): of 16 bits, one row beyond 8192: 1216 x 9216 26.9
//                     against 52.8, 4096 x 16384 152 against 206; two beyond 5120:
//                     4096 x 8192 67.7 against 79.3, 4096 x 6144 59.9 against 66.5,
//                     1216 x 6144 19.6 against 19.2; three below: 4096 x 5120 58.3
//                     against 47.2.  fp32 brings twice the bytes a row: 4096 x 6144
//                     77.0 against 81.1, 2048 x 5632 39.9 against 40.3; but beyond, with
//                     fewer copies, 4096 x 8192 without a gate 93.0 against 81.9 (with
//                     one 100.6 against 104.7), and
//                     below, with three rows an SM, 4096 x 4096 54.8 against 53.7, 4096 x
//                     2304 46.2 against 29.9; and at 4 rows an SM 608 x 6144 14.5 / 11.8
//                     against 13.0 / 10.3
template <int DT>
cudaError_t launch_dt(const MoeNormArgs &a, int num_sms, cudaStream_t s) {
    constexpr int V = DT == MOE_F32 ? 4 : 8;
    const auto on = [](const void *p, int64_t stride) {
        return reinterpret_cast<uintptr_t>(p) % 16 == 0 && stride % V == 0;
    };
    const bool full_gate = a.gate && a.gate_stride_d != 0;
    const bool vec = a.dim % V == 0 && on(a.x, a.x_stride) && on(a.y, a.y ? a.y_stride : 0) &&
                     on(a.out, a.out_stride) && on(a.normed, a.normed ? a.normed_stride : 0) &&
                     on(a.w_post, 0) && on(a.w_pre, 0) && (!full_gate || on(a.gate, a.gate_stride_t));
    const int most = vec ? 512 : 1024;  // threads a block
    const int acc = vec ? a.dim / V : a.dim;
    int m = 1;
    while (acc > m * most) m *= 2;
    const int threads = ((acc + m - 1) / m + 31) / 32 * 32;
    const int pieces = (acc + 511) / 512;  // a thread of the ring
    if (vec && a.n_tokens >= 8 * (int64_t)num_sms && (m * V > 16 || (m * V == 16 && threads > 65536 / 64 / 3)) &&
        (DT != MOE_F32 || pieces == 3)) {
        const int ring = ((acc + pieces - 1) / pieces + 31) / 32 * 32;
        const size_t row = (size_t)16 * pieces * ring * (1 + (a.y != nullptr) + full_gate);
        const int stages = (int)(kRing / row < 4 ? kRing / row : 4);  // 2 at least: 96 KB are the longest rows
        if constexpr (DT != MOE_F32) {
            if (pieces == 2) return launch_ring<DT, 2>(a, ring, stages, row * stages, num_sms, s);
            if (pieces == 4) return launch_ring<DT, 4>(a, ring, stages, row * stages, num_sms, s);
        }
        return launch_ring<DT, 3>(a, ring, stages, row * stages, num_sms, s);
    }
    if (!vec) return launch_rows<DT, 1, false>(a, m, threads, s);
    const bool early = m * V <= 4 || a.n_tokens <= (m * V <= 8 ? 4 : m * V <= 16 ? 1 : 0) * (int64_t)num_sms;
    return early ? launch_rows<DT, V, true>(a, m, threads, s) : launch_rows<DT, V, false>(a, m, threads, s);
}

}  // namespace

cudaError_t launch_block_norm(const MoeNormArgs &a, cudaStream_t s) {
    int dev = 0, nsm = 0;
    cudaError_t ce = cudaGetDevice(&dev);
    if (ce == cudaSuccess) ce = cudaDeviceGetAttribute(&nsm, cudaDevAttrMultiProcessorCount, dev);
    if (ce != cudaSuccess) return ce;
    switch (a.act_type) {
        case MOE_F32: return launch_dt<MOE_F32>(a, nsm, s);
        case MOE_F16: return launch_dt<MOE_F16>(a, nsm, s);
        default: return launch_dt<MOE_BF16>(a, nsm, s);
    }
}

}  // namespace moe
