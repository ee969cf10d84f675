// k_rope.cu -- rotary positions on queries and keys, keys and values into the
// paged cache (moe_rope_append).
//
// Pair i of a rotated head turns by position * theta_i.  theta_i / (2 pi) is
// held as a fraction of 2^64, so the part of a turn is the low half of a
// 64-bit integer product, exact at every position, where an fp32 angle would
// lose 17 bits at position 131072; sincospif takes its top 32 bits as a signed
// fraction of half a turn.  (No 64-bit floating point: its rate on this part
// is 1/64 of fp32's.)
//
// Bound by HBM: each element is read once and written once.  A block handles a
// few tokens; it forms their cos and sin once in shared memory (every head of a
// token turns by the same angles) and then streams the rows of all heads, eight
// elements (a pair of eights in the halves layout) per thread and step.
#include "attn_args.cuh"

namespace moe {
namespace {

constexpr int kThreads = 256;
constexpr int kMaxTok = 8;     // tokens of a block, at most
constexpr int kMaxHalf = 256;  // pairs of a head, at most

struct RopeSplit {
    int tok;           // tokens a block handles
    int per_q, per_v;  // work items of a q / k head and of a v head
    int n_q, n_k, n_v; // work items of a token
    FastDiv by_token, by_qk, by_v, by_page;
};

__device__ __forceinline__ float2 turn(float a, float b, float2 cs) {
    return make_float2(a * cs.x - b * cs.y, a * cs.y + b * cs.x);
}

template <int CT>
struct CacheStore {
    using C = typename Elem<CT>::type;
    static __device__ __forceinline__ void put8(C *p, float (&v)[8], float scale) {
        if (CT == MOE_E4M3) {
#pragma unroll
            for (int i = 0; i < 8; ++i) v[i] = __fdiv_rn(v[i], scale);
        }
        store_vec(p, v);
    }
    static __device__ __forceinline__ void put1(C *p, float v, float scale) { from_f32(v, *p); }
};
template <>
__device__ __forceinline__ void CacheStore<MOE_E4M3>::put1(uint8_t *p, float v, float scale) {
    *p = (uint8_t)f32x2_to_e4m3x2(__fdiv_rn(v, scale), 0.f);
}

// cos and sin (times the amplitude) of the block's tokens: cs[token][pair].
__device__ __forceinline__ void fill_angles(const MoeRopeArgs &a, int t0, int nt, float2 *cs) {
    const int half = a.rot_dim >> 1;
    for (int i = threadIdx.x; i < nt * half; i += kThreads) {
        const int t = i / half, j = i - t * half;
        const uint64_t part = a.turns[j] * (uint64_t)(int64_t)__ldg(a.positions + t0 + t);
        // nearest signed 32-bit fraction of a turn = units of 2^-31 half turns
        const int32_t top = (int32_t)(uint32_t)((part + 0x80000000ull) >> 32);
        float s, c;
        sincospif((float)top * 0x1p-31f, &s, &c);
        cs[i] = make_float2(c * a.amplitude, s * a.amplitude);
    }
}

// Rows whose every piece of eight elements is aligned (checked by the host).
template <int AT, int CT>
__global__ void __launch_bounds__(kThreads) rope_append_kernel(const __grid_constant__ MoeRopeArgs a,
                                                               const __grid_constant__ RopeSplit w) {
    using A = typename Elem<AT>::type;
    using C = typename Elem<CT>::type;
    __shared__ float2 cs[kMaxTok * kMaxHalf];
    __shared__ long long s_slot[kMaxTok];
    const int t0 = blockIdx.x * w.tok, nt = min(w.tok, a.n_tokens - t0);
    fill_angles(a, t0, nt, cs);
    if (threadIdx.x < nt) s_slot[threadIdx.x] = a.slots[t0 + threadIdx.x];
    __syncthreads();
    const int half = a.rot_dim >> 1;
    const int per_tok = w.n_q + w.n_k + w.n_v;
    const long long n_slots = (long long)a.n_pages * a.page_size;
    for (int i = threadIdx.x; i < nt * per_tok; i += kThreads) {
        const int t = (int)w.by_token.div(i);
        int j = i - t * per_tok;
        const bool is_q = j < w.n_q;
        const bool is_v = j >= w.n_q + w.n_k;
        long long page = 0;
        int at = 0;
        if (!is_q) {
            const long long slot = s_slot[t];
            if (slot < 0 || slot >= n_slots) continue;
            // slots below 2^31 by multiplication, others by a 64-bit division
            page = slot < 0x80000000ll ? (long long)w.by_page.div((uint32_t)slot) : slot / a.page_size;
            at = (int)(slot - page * a.page_size);
        }
        const int tok = t0 + t;
        if (is_v) {
            j -= w.n_q + w.n_k;
            const int h = (int)w.by_v.div(j), d = 8 * (j - h * w.per_v);
            float x[8];
            load_vec(static_cast<const A *>(a.v) + tok * a.v_stride_t + h * a.v_stride_h + d, x);
            CacheStore<CT>::put8(static_cast<C *>(a.v_cache) + page * a.vc_stride_page + at * a.vc_stride_tok +
                                     h * a.vc_stride_head + d,
                                 x, a.v_scale);
            continue;
        }
        if (!is_q) j -= w.n_q;
        const int h = (int)w.by_qk.div(j);
        j -= h * w.per_q;
        const A *src = is_q ? static_cast<const A *>(a.q) + tok * a.q_stride_t + h * a.q_stride_h
                            : static_cast<const A *>(a.k) + tok * a.k_stride_t + h * a.k_stride_h;
        A *qo = static_cast<A *>(a.q_out) + tok * a.qo_stride_t + h * a.qo_stride_h;
        C *kc = static_cast<C *>(a.k_cache) + page * a.kc_stride_page + at * a.kc_stride_tok + h * a.kc_stride_head;
        auto put = [&](int d, float(&x)[8]) {
            if (is_q) store_vec(qo + d, x);
            else CacheStore<CT>::put8(kc + d, x, a.k_scale);
        };
        // items: the rotated pieces first, then the pieces that pass through
        const int n_rot = a.interleaved ? a.rot_dim >> 3 : a.rot_dim >> 4;
        const float2 *c = cs + t * half;
        if (j >= n_rot) {
            int d = 8 * (j - n_rot);
            if (d >= a.rot_offset) d += a.rot_dim;
            float x[8];
            load_vec(src + d, x);
            put(d, x);
        } else if (a.interleaved) {
            const int d = a.rot_offset + 8 * j;
            float x[8];
            load_vec(src + d, x);
#pragma unroll
            for (int p = 0; p < 4; ++p) {
                const float2 r = turn(x[2 * p], x[2 * p + 1], c[4 * j + p]);
                x[2 * p] = r.x;
                x[2 * p + 1] = r.y;
            }
            put(d, x);
        } else {
            const int d = a.rot_offset + 8 * j;
            float x[8], y[8];
            load_vec(src + d, x);
            load_vec(src + d + half, y);
#pragma unroll
            for (int p = 0; p < 8; ++p) {
                const float2 r = turn(x[p], y[p], c[8 * j + p]);
                x[p] = r.x;
                y[p] = r.y;
            }
            put(d, x);
            put(d + half, y);
        }
    }
}

// Any size, stride and alignment: one element, or one pair, at a time.
template <int AT, int CT>
__global__ void __launch_bounds__(kThreads) rope_append_any_kernel(const __grid_constant__ MoeRopeArgs a,
                                                                   const __grid_constant__ RopeSplit w) {
    using A = typename Elem<AT>::type;
    using C = typename Elem<CT>::type;
    __shared__ float2 cs[kMaxTok * kMaxHalf];
    const int t0 = blockIdx.x * w.tok, nt = min(w.tok, a.n_tokens - t0);
    fill_angles(a, t0, nt, cs);
    __syncthreads();
    const int half = a.rot_dim >> 1;
    const int per_tok = w.n_q + w.n_k + w.n_v;
    const long long n_slots = (long long)a.n_pages * a.page_size;
    for (int i = threadIdx.x; i < nt * per_tok; i += kThreads) {
        const int t = (int)w.by_token.div(i);
        int j = i - t * per_tok;
        const int tok = t0 + t;
        const bool is_q = j < w.n_q, is_v = j >= w.n_q + w.n_k;
        const long long slot = a.slots[tok];
        if (!is_q && (slot < 0 || slot >= n_slots)) continue;
        const long long page = is_q ? 0 : slot / a.page_size, at = is_q ? 0 : slot - page * a.page_size;
        if (is_v) {
            j -= w.n_q + w.n_k;
            const int h = (int)w.by_v.div(j), d = j - h * w.per_v;
            const float x = to_f32(static_cast<const A *>(a.v)[tok * a.v_stride_t + h * a.v_stride_h + d]);
            CacheStore<CT>::put1(static_cast<C *>(a.v_cache) + page * a.vc_stride_page + at * a.vc_stride_tok +
                                     h * a.vc_stride_head + d,
                                 x, a.v_scale);
            continue;
        }
        if (!is_q) j -= w.n_q;
        const int h = (int)w.by_qk.div(j);
        j -= h * w.per_q;
        const A *src = is_q ? static_cast<const A *>(a.q) + tok * a.q_stride_t + h * a.q_stride_h
                            : static_cast<const A *>(a.k) + tok * a.k_stride_t + h * a.k_stride_h;
        A *qo = static_cast<A *>(a.q_out) + tok * a.qo_stride_t + h * a.qo_stride_h;
        C *kc = static_cast<C *>(a.k_cache) + page * a.kc_stride_page + at * a.kc_stride_tok + h * a.kc_stride_head;
        auto put = [&](int d, float v) {
            if (is_q) from_f32(v, qo[d]);
            else CacheStore<CT>::put1(kc + d, v, a.k_scale);
        };
        if (j >= half) {
            int d = j - half;
            if (d >= a.rot_offset) d += a.rot_dim;
            put(d, to_f32(src[d]));
        } else {
            const int d0 = a.rot_offset + (a.interleaved ? 2 * j : j), d1 = a.interleaved ? d0 + 1 : d0 + half;
            const float2 r = turn(to_f32(src[d0]), to_f32(src[d1]), cs[t * half + j]);
            put(d0, r.x);
            put(d1, r.y);
        }
    }
}

template <int AT, int CT>
cudaError_t launch(const MoeRopeArgs &a, bool fast, int num_sms, cudaStream_t s) {
    RopeSplit w;
    const int n_rot = fast ? (a.interleaved ? a.rot_dim / 8 : a.rot_dim / 16) : a.rot_dim / 2;
    w.per_q = n_rot + (a.head_dim - a.rot_dim) / (fast ? 8 : 1);
    w.per_v = a.v_dim / (fast ? 8 : 1);
    w.n_q = a.n_heads * w.per_q;
    w.n_k = a.n_kv_heads * w.per_q;
    w.n_v = a.n_kv_heads * w.per_v;
    // enough blocks for four per SM first, then more tokens a block
    const int64_t per = a.n_tokens / (4 * (int64_t)num_sms);
    w.tok = per < 1 ? 1 : per > kMaxTok ? kMaxTok : (int)per;
    w.by_token = FastDiv((uint32_t)(w.n_q + w.n_k + w.n_v));
    w.by_qk = FastDiv((uint32_t)w.per_q);
    w.by_v = FastDiv((uint32_t)(w.per_v > 0 ? w.per_v : 1));
    w.by_page = FastDiv((uint32_t)a.page_size);
    const int grid = (a.n_tokens + w.tok - 1) / w.tok;
    if (fast)
        rope_append_kernel<AT, CT><<<grid, kThreads, 0, s>>>(a, w);
    else
        rope_append_any_kernel<AT, CT><<<grid, kThreads, 0, s>>>(a, w);
    return cudaGetLastError();
}

template <int AT>
cudaError_t launch_ct(const MoeRopeArgs &a, bool fast, int num_sms, cudaStream_t s) {
    switch (a.cache_type) {
        case MOE_F16: return launch<AT, MOE_F16>(a, fast, num_sms, s);
        case MOE_BF16: return launch<AT, MOE_BF16>(a, fast, num_sms, s);
        default: return launch<AT, MOE_E4M3>(a, fast, num_sms, s);
    }
}

// Base and strides keep every piece of eight elements on `bytes`.
bool pieces_on(const void *p, size_t elem, size_t bytes, int64_t s0, int64_t s1, int64_t s2 = 0) {
    return reinterpret_cast<uintptr_t>(p) % bytes == 0 && (s0 * (int64_t)elem) % (int64_t)bytes == 0 &&
           (s1 * (int64_t)elem) % (int64_t)bytes == 0 && (s2 * (int64_t)elem) % (int64_t)bytes == 0;
}

}  // namespace

cudaError_t launch_rope_append(const MoeRopeArgs &a, cudaStream_t s) {
    int dev = 0, nsm = 0;
    cudaError_t ce = cudaGetDevice(&dev);
    if (ce == cudaSuccess) ce = cudaDeviceGetAttribute(&nsm, cudaDevAttrMultiProcessorCount, dev);
    if (ce != cudaSuccess) return ce;
    const size_t ae = dtype_bytes(a.act_type), ce8 = dtype_bytes(a.cache_type), cb = ce8 == 1 ? 8 : 16;
    // the 16-byte kernel wants whole pieces of eight on both sides of the
    // rotated part and of its halves
    const bool fast = a.head_dim % 8 == 0 && a.v_dim % 8 == 0 && a.rot_offset % 8 == 0 &&
                      a.rot_dim % (a.interleaved ? 8 : 16) == 0 && pieces_on(a.q, ae, 16, a.q_stride_t, a.q_stride_h) &&
                      pieces_on(a.q_out, ae, 16, a.qo_stride_t, a.qo_stride_h) &&
                      pieces_on(a.k, ae, 16, a.k_stride_t, a.k_stride_h) &&
                      pieces_on(a.k_cache, ce8, cb, a.kc_stride_page, a.kc_stride_tok, a.kc_stride_head) &&
                      (a.v_dim == 0 || (pieces_on(a.v, ae, 16, a.v_stride_t, a.v_stride_h) &&
                                        pieces_on(a.v_cache, ce8, cb, a.vc_stride_page, a.vc_stride_tok,
                                                  a.vc_stride_head)));
    switch (a.act_type) {
        case MOE_F32: return launch_ct<MOE_F32>(a, fast, nsm, s);
        case MOE_F16: return launch_ct<MOE_F16>(a, fast, nsm, s);
        default: return launch_ct<MOE_BF16>(a, fast, nsm, s);
    }
}

}  // namespace moe
