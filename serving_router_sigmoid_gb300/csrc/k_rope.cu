// k_rope.cu -- rotary positions on queries and keys, keys and values into the
// paged cache (moe_rope_append).
//
// Pair i of a rotated head turns by position * theta_i.  theta_i / (2 pi) is
// held as a fraction of 2^64, so the part of a turn is the low half of a
// 64-bit integer product, exact at every position, where an fp32 angle would
// lose 17 bits at position 131072.  Quarter turns are taken off in integers, and
// sincospif takes what is left, rounded to fp32: off by 2^-24 of itself, 2^-27
// half turns at most, and by 2^-33.  (No 64-bit floating point, which is slow
// here.)
//
// Bound by HBM: each element is read once and written once.  A block handles a
// few tokens; it forms their cos and sin once in shared memory (every head of a
// token turns by the same angles) and then streams the rows of all heads, eight
// elements (a pair of eights in the halves layout) per thread and step.  16384
// tokens of 64 + 8 bf16 heads into E4M3: 107 us, 5.9 TB/s; 2048 tokens of 32 + 8
// fp32 heads: 18 us, 5.2 TB/s; one token: 3 us.
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
    int head_slots, v_slots;  // heads a block takes side by side
    FastDiv by_token, by_qk, by_v, by_heads, by_kv;
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
        const uint64_t part = a.turns[j] * (uint64_t)(int64_t)ld_in(a.positions + t0 + t);
        // the nearest quarter turn, and the rest in units of 2^-32 half turns (at
        // most 2^30 of them)
        const uint32_t quarter = (uint32_t)((part + (1ull << 61)) >> 62);
        const int64_t rest = (int64_t)(part - ((uint64_t)quarter << 62));
        float s, c;
        sincospif((float)(int32_t)((rest + (1ll << 30)) >> 31) * 0x1p-32f, &s, &c);
        if (quarter & 1) {
            const float t = c;
            c = -s;
            s = t;
        }
        if (quarter & 2) c = -c, s = -s;
        cs[i] = make_float2(c * a.amplitude, s * a.amplitude);
    }
}

// Eight consecutive elements as loaded.
template <int AT>
struct Piece {
    using A = typename Elem<AT>::type;
    uint4 w[AT == MOE_F32 ? 2 : 1];
    __device__ __forceinline__ void load(const A *p) {
        w[0] = ld_once16(p);
        if constexpr (AT == MOE_F32) w[1] = ld_once16(p + 4);
    }
    __device__ __forceinline__ void get(float (&v)[8]) const {
        if constexpr (AT == MOE_F32) {
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                v[4 * i] = __uint_as_float(w[i].x); v[4 * i + 1] = __uint_as_float(w[i].y);
                v[4 * i + 2] = __uint_as_float(w[i].z); v[4 * i + 3] = __uint_as_float(w[i].w);
            }
        } else {
            const uint32_t u[4] = {w[0].x, w[0].y, w[0].z, w[0].w};
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const float2 f = half_pair(u[i], A());
                v[2 * i] = f.x;
                v[2 * i + 1] = f.y;
            }
        }
    }
};

// Rows whose every piece of eight elements is aligned (checked by the host).
// A thread keeps one piece of the head (a pair of pieces in the halves layout)
// and goes through the block's (token, head) pairs, kBatch of them in flight.
// The angles and the cache rows of the tokens come from shared memory.
template <int AT, int CT, bool PAIRED>
__global__ void __launch_bounds__(kThreads, 3) rope_append_kernel(const __grid_constant__ MoeRopeArgs a,
                                                                  const __grid_constant__ RopeSplit w) {
    using A = typename Elem<AT>::type;
    using C = typename Elem<CT>::type;
    constexpr int kBatch = PAIRED && AT == MOE_F32 ? 1 : 2;
    __shared__ float2 cs[kMaxTok * kMaxHalf];
    __shared__ longlong2 row[kMaxTok];  // offsets of the token's rows in the caches; x < 0: not cached
    after_previous();
    const int t0 = blockIdx.x * w.tok, nt = min(w.tok, a.n_tokens - t0);
    const int half = a.rot_dim >> 1, n_rot = PAIRED ? a.rot_dim >> 4 : a.rot_dim >> 3;
    const int hs = (int)w.by_qk.div(threadIdx.x), j = threadIdx.x - hs * w.per_q;  // head slot, piece
    const int vh = (int)w.by_v.div(threadIdx.x), vj = threadIdx.x - vh * w.per_v;
    const bool rotated = j < n_rot, two = PAIRED && rotated;
    int d = 8 * (rotated ? j : j - n_rot);
    if (rotated || d >= a.rot_offset) d += rotated ? a.rot_offset : a.rot_dim;
    const int n_heads = a.n_heads + a.n_kv_heads, end = hs < w.head_slots ? nt * n_heads : 0;
    const int v_end = vh < w.v_slots ? nt * a.n_kv_heads : 0;
    const A *q = static_cast<const A *>(a.q) + t0 * a.q_stride_t + d;
    const A *k = static_cast<const A *>(a.k) + t0 * a.k_stride_t + d;
    const A *v = static_cast<const A *>(a.v) + t0 * a.v_stride_t + 8 * vj;
    A *qo = static_cast<A *>(a.q_out) + t0 * a.qo_stride_t + d;

    Piece<AT> x[kBatch], y[PAIRED ? kBatch : 1];
    auto load = [&](int e0) {
#pragma unroll
        for (int i = 0; i < kBatch; ++i) {
            const int e = e0 + i * w.head_slots;
            if (e >= end) break;
            const int t = (int)w.by_heads.div(e), h = e - t * n_heads;
            const A *p = h < a.n_heads ? q + t * a.q_stride_t + h * a.q_stride_h
                                       : k + t * a.k_stride_t + (h - a.n_heads) * a.k_stride_h;
            x[i].load(p);
            if (two) y[PAIRED ? i : 0].load(p + half);
        }
    };
    auto load_v = [&](int e0) {
#pragma unroll
        for (int i = 0; i < kBatch; ++i) {
            const int e = e0 + i * w.v_slots;
            if (e >= v_end) break;
            const int t = (int)w.by_kv.div(e), h = e - t * a.n_kv_heads;
            x[i].load(v + t * a.v_stride_t + h * a.v_stride_h);
        }
    };
    // the first rows are on their way while the angles are formed
    load(hs);
    if (threadIdx.x < nt) {
        const long long slot = ld_in(a.slots + t0 + threadIdx.x);
        longlong2 r = make_longlong2(-1, -1);
        if (slot >= 0 && slot < (long long)a.n_pages * a.page_size) {
            const long long page = slot / a.page_size, at = slot - page * a.page_size;
            r.x = page * a.kc_stride_page + at * a.kc_stride_tok;
            r.y = page * a.vc_stride_page + at * a.vc_stride_tok;
        }
        row[threadIdx.x] = r;
    }
    fill_angles(a, t0, nt, cs);
    __syncthreads();
#pragma unroll 1
    for (int e0 = hs; e0 < end; e0 += kBatch * w.head_slots) {
        Piece<AT> cx[kBatch], cy[PAIRED ? kBatch : 1];
#pragma unroll
        for (int i = 0; i < kBatch; ++i) {
            cx[i] = x[i];
            if (PAIRED) cy[i] = y[i];
        }
        load(e0 + kBatch * w.head_slots);
#pragma unroll
        for (int i = 0; i < kBatch; ++i) {
            const int e = e0 + i * w.head_slots;
            if (e >= end) break;
            const int t = (int)w.by_heads.div(e), h = e - t * n_heads;
            float u[8], z[8];
            cx[i].get(u);
            if (two) cy[PAIRED ? i : 0].get(z);
            if (rotated) {
                const float2 *c = cs + t * half + (PAIRED ? 8 : 4) * j;
                if constexpr (PAIRED) {
#pragma unroll
                    for (int m = 0; m < 8; ++m) {
                        const float2 r = turn(u[m], z[m], c[m]);
                        u[m] = r.x;
                        z[m] = r.y;
                    }
                } else {
#pragma unroll
                    for (int m = 0; m < 4; ++m) {
                        const float2 r = turn(u[2 * m], u[2 * m + 1], c[m]);
                        u[2 * m] = r.x;
                        u[2 * m + 1] = r.y;
                    }
                }
            }
            if (h < a.n_heads) {
                A *p = qo + t * a.qo_stride_t + h * a.qo_stride_h;
                store_vec(p, u);
                if (two) store_vec(p + half, z);
            } else if (row[t].x >= 0) {
                C *p = static_cast<C *>(a.k_cache) + row[t].x + (h - a.n_heads) * a.kc_stride_head + d;
                CacheStore<CT>::put8(p, u, a.k_scale);
                if (two) CacheStore<CT>::put8(p + half, z, a.k_scale);
            }
        }
    }
    load_v(vh);
#pragma unroll 1
    for (int e0 = vh; e0 < v_end; e0 += kBatch * w.v_slots) {
        Piece<AT> cx[kBatch];
#pragma unroll
        for (int i = 0; i < kBatch; ++i) cx[i] = x[i];
        load_v(e0 + kBatch * w.v_slots);
#pragma unroll
        for (int i = 0; i < kBatch; ++i) {
            const int e = e0 + i * w.v_slots;
            if (e >= v_end) break;
            const int t = (int)w.by_kv.div(e), h = e - t * a.n_kv_heads;
            if (row[t].x < 0) continue;
            float u[8];
            cx[i].get(u);
            CacheStore<CT>::put8(static_cast<C *>(a.v_cache) + row[t].y + h * a.vc_stride_head + 8 * vj, u, a.v_scale);
        }
    }
}

// Any size, stride and alignment: one element, or one pair, at a time (2048
// tokens bf16, 32 + 8 heads of 80 dimensions, 40 of them turned in halves: 50 us,
// where rows in 16-byte pieces, all 80 turned, take 8.8).
template <int AT, int CT>
__global__ void __launch_bounds__(kThreads) rope_append_any_kernel(const __grid_constant__ MoeRopeArgs a,
                                                                   const __grid_constant__ RopeSplit w) {
    using A = typename Elem<AT>::type;
    using C = typename Elem<CT>::type;
    __shared__ float2 cs[kMaxTok * kMaxHalf];
    after_previous();
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
    // tokens a block: the fewest in a row on one of the 3 blocks an SM holds,
    // waves * tok, and of those the most a block (16384 tokens: 6 waves of 6
    // against 5 of 8)
    int64_t best = INT64_MAX;
    for (int tok = 1; tok <= kMaxTok; ++tok) {
        const int64_t blocks = ((int64_t)a.n_tokens + tok - 1) / tok, row = (blocks + 3 * num_sms - 1) / (3 * num_sms) * tok;
        if (row <= best) best = row, w.tok = tok;
        if (blocks <= num_sms) break;
    }
    w.by_token = FastDiv((uint32_t)(w.n_q + w.n_k + w.n_v));
    w.by_qk = FastDiv((uint32_t)w.per_q);
    w.by_v = FastDiv((uint32_t)(w.per_v > 0 ? w.per_v : 1));
    w.by_heads = FastDiv((uint32_t)(a.n_heads + a.n_kv_heads));
    w.by_kv = FastDiv((uint32_t)(a.n_kv_heads > 0 ? a.n_kv_heads : 1));
    w.head_slots = kThreads / w.per_q;
    w.v_slots = w.per_v > 0 ? kThreads / w.per_v : 0;
    const int grid = (int)((a.n_tokens + (int64_t)w.tok - 1) / w.tok);
    void (*fn)(MoeRopeArgs, RopeSplit) = !fast            ? rope_append_any_kernel<AT, CT>
                                         : a.interleaved ? rope_append_kernel<AT, CT, false>
                                                         : rope_append_kernel<AT, CT, true>;
    void *args[] = {const_cast<MoeRopeArgs *>(&a), &w};
    return launch_after(reinterpret_cast<const void *>(fn), grid, kThreads, 0, s, args);
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
