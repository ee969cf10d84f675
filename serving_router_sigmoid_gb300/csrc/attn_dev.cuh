// attn_dev.cuh -- attention of one new token per request over the paged
// key-value cache: the kernel.
//
//   s_j = scale q . k_j,  out = sum_j e^(s_j) v_j / sum_j e^(s_j)
//
// Every cache row is read once, for 4 G flops a byte pair (G query heads share
// a key head): HBM bounds it as long as the bytes keep flowing.  So:
//
// - Work is split by bytes, not by request.  All (request, key head) segments
//   are cut into steps of TT tokens; the steps form one line, and every warp of
//   the grid (one block per SM) takes an equal run of it, found from a prefix
//   sum of the lengths that each block forms for itself.  A batch of one long
//   and many short requests keeps every SM busy to the end, with one launch
//   and no plan on the host.
// - A warp needs no other warp until its run ends.  Rows go from HBM straight
//   into the registers of the tensor-core fragments: with the tokens on the
//   MMA's M side a lane's 16-byte piece of a key row IS its A fragment (the
//   order of the contraction is free, the query takes the same order), and four
//   pieces of value rows become A fragments of V^T by byte permutes.  No shared
//   memory, no barrier, no transposition; 8 KB a warp stay in flight.
// - The heads of a group sit on N (8 a tile), so S^T = K q^T leaves each lane
//   the logits of its own two heads: the running maximum, the sum and the
//   rescale of O^T need no exchange.  The maximum moves only when a logit
//   passes it by 2^8 (one vote a step); weights stay below 2^8 and sums in fp32
//   do not care.
// - Where a run ends inside a segment, the warp leaves (O, m, l); the block
//   joins its warps' pieces in shared memory, and of the blocks that share a
//   segment the last to arrive joins their pieces in block order, so the result
//   does not depend on who is last.
//
// Precision: products of the cache's own type (E4M3 codes widen exactly to
// f16) accumulate in fp32; logits, m, l and O are fp32.  A weight enters the
// second product in NP terms of 16 bits: 2 terms keep 16 (bf16) or 22 (f16)
// bits of it, so that the output's own rounding is the only one that shows;
// fp32 queries enter in 2 (f16) or 3 (bf16) terms.  For f16 products each query
// row is scaled by a power of two to about 1, which the logit's factor undoes.
#pragma once

#include "attn_args.cuh"

namespace moe {
namespace attn {

struct Params {
    MoeAttnArgs a;
    int n_heads, n_kv, group, n_groups;  // query heads, key heads, heads a key head, 8*NT-head groups a key head
    int k_dim, v_dim;
    int q16, out16;       // rows of q / out start on 16 bytes
    int by16;             // pages hold whole runs of 16 tokens
    uint32_t n_pages;
    int64_t k_page, k_tok, k_tok8, k_head;  // strides in bytes (tok8: of 8 tokens)
    int64_t v_page, v_tok, v_tok8, v_head;
    FastDiv by_page;
    float *part;          // [2 grid] pieces
    int *arrived;         // [requests, key heads * groups]
    int min_steps;        // fewest steps worth a block
};

template <int CT, int DMAX, int NT, bool WIDE>
struct Cfg {
    static constexpr bool kF16 = CT != MOE_BF16;
    static constexpr int ES = CT == MOE_E4M3 ? 1 : 2;
    static constexpr int KCH = DMAX * ES / 64;                       // 16-byte pieces of a key row per lane
    static constexpr int VB = CT == MOE_E4M3 && DMAX == 64 ? 8 : 16;  // bytes of a piece of a value row
    static constexpr int VCH = DMAX * ES / (8 * VB);                 // pieces of a value row per lane
    static constexpr int VE = VB / ES;                               // elements of such a piece
    static constexpr int KSTEPS = DMAX / 16;
    static constexpr int VW = DMAX / 16;  // pairs of value dimensions per lane
    // 16-token tiles a step: 8 KB of keys and values a warp
    static constexpr int R = 32 * DMAX * ES >= 8192 ? 1 : 8192 / (32 * DMAX * ES);
    static constexpr int TT = 16 * R;
    static constexpr int NQ = !WIDE ? 1 : kF16 ? 2 : 3;
    static constexpr int NP = WIDE ? NQ : 2;
    static constexpr int ROWS = 8 * NT;
    static constexpr bool QS = NQ * NT * DMAX > 128;  // query fragments stay in shared memory
    // one block per SM; registers allow 12 warps of the plain form, and shared
    // memory 4 of the largest ones
    static constexpr int WARPS = DMAX <= 128 && NT == 1 && !WIDE ? 12 : WIDE && NT * DMAX == 256 ? 4 : 8;
    static constexpr int THREADS = 32 * WARPS;
    static constexpr int PIECE = ROWS * (DMAX + 2);  // floats of a piece: O, m, l
    static constexpr int QFRAGS = NQ * NT * KSTEPS;
    static constexpr size_t kQBytes = (size_t)WARPS * QFRAGS * 32 * 8;
    static constexpr size_t smem(int n_requests) {
        return ((size_t)(n_requests + 1) * 4 + 15) / 16 * 16 + kQBytes + (size_t)WARPS * 2 * PIECE * 4;
    }
    static_assert(((MOE_MAX_REQUESTS + 1) * 4 + 16) + kQBytes + WARPS * 2 * PIECE * 4 + 2048 <= 227 * 1024, "");
    // weights are held times 2^kOff: f16's subnormals then start at 2^-31 of the maximum
    static constexpr float kOff = kF16 ? 7.f : 0.f;
};

constexpr float kLazy = 8.f;        // the maximum moves when a logit passes it by 2^kLazy
constexpr float kFloor = -1e38f;    // running maximum before any token

template <bool F16>
__device__ __forceinline__ void mma(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                    uint32_t b1) {
    if constexpr (F16)
        asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
                     "{%0,%1,%2,%3};"
                     : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
                     : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
    else
        asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
                     "{%0,%1,%2,%3};"
                     : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
                     : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
__device__ __forceinline__ uint32_t transpose8x8(uint32_t v) {
    uint32_t r;
    asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(v));
    return r;
}
__device__ __forceinline__ float exp2_fast(float x) {  // within 2^-22
    float r;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
    return r;
}
__device__ __forceinline__ uint4 ld16(const char *p) {
    const int4 v = ld_stream16(p);
    return make_uint4(v.x, v.y, v.z, v.w);
}
__device__ __forceinline__ uint2 ld8(const char *p) {
    uint2 r;
    asm volatile("ld.global.nc.L1::no_allocate.L2::256B.v2.u32 {%0,%1}, [%2];" : "=r"(r.x), "=r"(r.y) : "l"(p));
    return r;
}
// Four e4m3 codes -> two pairs of f16 (exact).
__device__ __forceinline__ void e4m3x4_to_f16x4(uint32_t codes, uint32_t &lo, uint32_t &hi) {
    asm("{ .reg .b16 l, h; mov.b32 {l, h}, %2; cvt.rn.f16x2.e4m3x2 %0, l; cvt.rn.f16x2.e4m3x2 %1, h; }"
        : "=r"(lo), "=r"(hi)
        : "r"(codes));
}
template <bool F16>
__device__ __forceinline__ uint32_t pack2(float lo, float hi) {
    if constexpr (F16) return pack_pair(lo, hi, __half());
    else return pack_pair(lo, hi, __nv_bfloat16());
}
template <bool F16>
__device__ __forceinline__ float2 unpack2(uint32_t w) {
    if constexpr (F16) return half_pair(w, __half());
    else return half_pair(w, __nv_bfloat16());
}

__device__ __forceinline__ int last_le(const int *v, int n, int x) {
    int lo = 0, hi = n;
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (v[mid] <= x) lo = mid; else hi = mid;
    }
    return lo;
}

// The tokens of request b that are seen: [from, len).
__device__ __forceinline__ void seen(const MoeAttnArgs &a, int b, int &from, int &len) {
    len = min(max(__ldg(a.seq_len + b), 0), a.max_pages * a.page_size);
    from = a.window > 0 ? max(0, len - a.window) : 0;
}

// 8 consecutive elements of q as fp32.
__device__ __forceinline__ void load_q(const Params &p, int64_t at, float (&v)[8]) {
    if (p.a.act_type == MOE_F32) {
        const float *q = static_cast<const float *>(p.a.q) + at;
        if (p.q16) {
            load_vec(q, v);
        } else {
#pragma unroll
            for (int i = 0; i < 8; ++i) v[i] = q[i];
        }
        return;
    }
    const uint16_t *q = static_cast<const uint16_t *>(p.a.q) + at;
    uint32_t w[4];
    if (p.q16) {
        const uint4 x = *reinterpret_cast<const uint4 *>(q);
        w[0] = x.x; w[1] = x.y; w[2] = x.z; w[3] = x.w;
    } else {
#pragma unroll
        for (int i = 0; i < 4; ++i) w[i] = q[2 * i] | (uint32_t)q[2 * i + 1] << 16;
    }
    const bool h = p.a.act_type == MOE_F16;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float2 f = h ? half_pair(w[i], __half()) : half_pair(w[i], __nv_bfloat16());
        v[2 * i] = f.x;
        v[2 * i + 1] = f.y;
    }
}

// 4 consecutive outputs.
__device__ __forceinline__ void store_out(const Params &p, int64_t at, const float (&v)[4]) {
    if (p.a.act_type == MOE_F32) {
        float *o = static_cast<float *>(p.a.out) + at;
        if (p.out16) {
            store_vec(o, v);
        } else {
#pragma unroll
            for (int i = 0; i < 4; ++i) o[i] = v[i];
        }
        return;
    }
    uint16_t *o = static_cast<uint16_t *>(p.a.out) + at;
    const bool h = p.a.act_type == MOE_F16;
    const uint32_t x = h ? pack2<true>(v[0], v[1]) : pack2<false>(v[0], v[1]);
    const uint32_t y = h ? pack2<true>(v[2], v[3]) : pack2<false>(v[2], v[3]);
    if (p.out16) {
        *reinterpret_cast<uint2 *>(o) = make_uint2(x, y);
    } else {
        o[0] = (uint16_t)x; o[1] = (uint16_t)(x >> 16); o[2] = (uint16_t)y; o[3] = (uint16_t)(y >> 16);
    }
}

// One piece of a segment that a warp leaves to its block.
struct Slot {
    long long begin, end;  // the whole segment on the line of steps
    int b, hg;             // request, head group; b < 0: no piece
};

// Joins n pieces (O, m, l) of one segment, the i-th at piece(i), into the
// output, or into a piece `to` for the blocks' join; threads tid of nthr.
// (Rolled loops: this code runs once a segment, its size counts more.)
template <int ROWS, int DMAX, typename Piece>
__device__ __forceinline__ void join_pieces(const Params &p, Piece piece, int n, int b, int hg, float *to, int tid,
                                            int nthr) {
    const int kvh = hg / p.n_groups, h0 = kvh * p.group + (hg - kvh * p.n_groups) * ROWS;
    const int heads = min(ROWS, (kvh + 1) * p.group - h0);
#pragma unroll 1
    for (int e = tid; e < ROWS * (DMAX / 4); e += nthr) {
        const int row = e / (DMAX / 4), d = 4 * (e - row * (DMAX / 4));
        if (row >= heads || d >= p.v_dim) continue;
        float top = kFloor;
#pragma unroll 1
        for (int i = 0; i < n; ++i) top = fmaxf(top, piece(i)[ROWS * DMAX + row]);
        float sum = 0.f, x[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll 2
        for (int i = 0; i < n; ++i) {
            const float *q = piece(i);
            const float f = exp2_fast(q[ROWS * DMAX + row] - top);
            sum = fmaf(q[ROWS * (DMAX + 1) + row], f, sum);
            const float4 v = *reinterpret_cast<const float4 *>(q + row * DMAX + d);
            x[0] = fmaf(v.x, f, x[0]);
            x[1] = fmaf(v.y, f, x[1]);
            x[2] = fmaf(v.z, f, x[2]);
            x[3] = fmaf(v.w, f, x[3]);
        }
        if (to) {
            store_vec(to + row * DMAX + d, x);
            if (d == 0) {
                to[ROWS * DMAX + row] = top;
                to[ROWS * (DMAX + 1) + row] = sum;
            }
        } else {
            const bool none = sum == 0.f;  // no token seen (a NaN goes through)
            const float inv = none ? 0.f : p.a.v_scale / sum;
#pragma unroll
            for (int j = 0; j < 4; ++j) x[j] = none ? 0.f : x[j] * inv;
            store_out(p, b * p.a.out_stride_b + (h0 + row) * p.a.out_stride_h + d, x);
            if (d == 0 && p.a.lse)
                p.a.lse[(int64_t)b * p.n_heads + h0 + row] =
                    none ? -INFINITY : (top + log2f(sum)) * 0.6931471805599453f;
        }
    }
}

template <int CT, int DMAX, int NT, bool WIDE>
__global__ void __launch_bounds__(Cfg<CT, DMAX, NT, WIDE>::THREADS, 1)
    attn_decode_kernel(const __grid_constant__ Params p) {
    using C = Cfg<CT, DMAX, NT, WIDE>;
    constexpr bool F16 = C::kF16;
    extern __shared__ __align__(16) char smem[];
    __shared__ Slot slots[C::WARPS * 2], s_open[2];
    __shared__ int wsum[C::WARPS];
    __shared__ int s_join[2];  // blocks before the last of a shared segment to join, or -1
    const MoeAttnArgs &a = p.a;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, g = lane >> 2, c = lane & 3;
    const int n_req = a.n_requests, HG = p.n_kv * p.n_groups;
    int *prefix = reinterpret_cast<int *>(smem);
    char *after = smem + ((size_t)(n_req + 1) * 4 + 15) / 16 * 16;
    uint2 *qsm = reinterpret_cast<uint2 *>(after) + warp * C::QFRAGS * 32;
    float *pieces = reinterpret_cast<float *>(after + C::kQBytes);

    // prefix sum of the requests' steps
    int total = 0;
    for (int base = 0; base < n_req; base += C::THREADS) {
        const int b = base + tid;
        int n = 0;
        if (b < n_req) {
            int from, len;
            seen(a, b, from, len);
            n = len > from ? (len - 1) / C::TT - from / C::TT + 1 : 0;
        }
        int x = n;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int y = __shfl_up_sync(0xffffffffu, x, o);
            if (lane >= o) x += y;
        }
        if (base) __syncthreads();
        if (lane == 31) wsum[warp] = x;
        __syncthreads();
        int below = 0, all = 0;
#pragma unroll
        for (int w = 0; w < C::WARPS; ++w) {
            const int s = wsum[w];
            if (w < warp) below += s;
            all += s;
        }
        if (b < n_req) prefix[b] = total + below + x - n;
        total += all;
    }
    if (tid == 0) prefix[n_req] = total;
    if (lane < 2) slots[warp * 2 + lane].b = -1;
    if (tid < 2) s_join[tid] = -1;
    __syncthreads();
    // requests that see nothing, by the blocks in turn
    for (int b = blockIdx.x; b < n_req; b += gridDim.x) {
        if (prefix[b + 1] != prefix[b]) continue;
        const float z[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll 1
        for (int i = tid; i < p.n_heads * (p.v_dim / 4); i += C::THREADS) {
            const int h = i / (p.v_dim / 4), d = 4 * (i - h * (p.v_dim / 4));
            store_out(p, b * a.out_stride_b + h * a.out_stride_h + d, z);
        }
        if (a.lse)
            for (int h = tid; h < p.n_heads; h += C::THREADS) a.lse[(int64_t)b * p.n_heads + h] = -INFINITY;
    }

    // this block's and this warp's run of steps
    const long long U = (long long)total * HG;
    long long per = (U + gridDim.x - 1) / gridDim.x;
    if (per < p.min_steps) per = p.min_steps;
    const long long lo = blockIdx.x * per, hi = min(lo + per, U);
    if (lo >= U) return;
    const long long per_w = (hi - lo + C::WARPS - 1) / C::WARPS;
    const long long wb = min(lo + warp * per_w, hi), we = min(wb + per_w, hi);

    int b = 0, hg = 0, steps = 1;
    long long sb = 0;  // first step of the segment (b, hg)
    if (wb < we) {
        b = last_le(prefix, n_req, (int)(wb / HG));
        steps = prefix[b + 1] - prefix[b];
        sb = (long long)prefix[b] * HG;
        hg = (int)((wb - sb) / steps);
        sb += (long long)hg * steps;
    }
    for (long long u = wb; u < we;) {
        const long long se = sb + steps;
        const int first = (int)(u - sb), last = (int)(min(se, we) - sb);
        const int kvh = hg / p.n_groups, h0 = kvh * p.group + (hg - kvh * p.n_groups) * C::ROWS;
        const int heads = min(C::ROWS, (kvh + 1) * p.group - h0);
        int from, len;
        seen(a, b, from, len);
        const int tok0 = from / C::TT * C::TT;

        // page ids of the next 64 pages, a window of 32 in each register
        const int32_t *bt = a.block_table + b * a.table_stride;
        int wcol = 0, cur = -1, nxt = -1;
        const int ncol = (int)p.by_page.div(len - 1) + 1;
        if (p.by16) {
            wcol = (int)p.by_page.div(tok0 + first * C::TT);
            cur = wcol + lane < ncol ? __ldg(bt + wcol + lane) : -1;
            nxt = wcol + 32 + lane < ncol ? __ldg(bt + wcol + 32 + lane) : -1;
        }

        const char *kb = static_cast<const char *>(a.k_cache) + kvh * p.k_head + g * p.k_tok + c * 16;
        const char *vb = static_cast<const char *>(a.v_cache) + kvh * p.v_head + 2 * c * p.v_tok + g * C::VB;
        uint4 kr[C::R][2][C::KCH];
        uint32_t vr[C::R][4][C::VCH][C::VB / 4];
#pragma unroll
        for (int r = 0; r < C::R; ++r) {
#pragma unroll
            for (int h = 0; h < 2; ++h)
#pragma unroll
                for (int i = 0; i < C::KCH; ++i) kr[r][h][i] = make_uint4(0u, 0u, 0u, 0u);
#pragma unroll
            for (int k = 0; k < 4; ++k)
#pragma unroll
                for (int i = 0; i < C::VCH; ++i)
#pragma unroll
                    for (int j = 0; j < C::VB / 4; ++j) vr[r][k][i][j] = 0u;
        }

        // A step is `plain` when all its tokens are seen and lie on whole
        // pages: its rows are then at fixed distances from one address a tile.
        // (Pieces beyond the head's size stay the zeros they are.)
        int page[C::R], at[C::R];
        bool plain = false;
        uint32_t k_on = 0;  // else: bit 2 r + half, that key row is seen
        auto row_at = [&](int t, int r, int row, int64_t sp, int64_t st) -> int64_t {  // from row 0; -1: not seen
            const int tok = t + 16 * r + row;
            if (tok < from || tok >= len) return -1;
            int pg, in;
            if (p.by16) {
                pg = page[r];
                in = at[r] + row;
            } else {
                const int col = (int)p.by_page.div(tok);
                pg = __ldg(bt + col);
                in = tok - col * a.page_size;
            }
            return (uint32_t)pg < p.n_pages ? pg * sp + in * st : -1;
        };
        auto request_keys = [&](int t) {
            plain = p.by16 && t >= from && t + C::TT <= len;
            if (p.by16) {
#pragma unroll
                for (int r = 0; r < C::R; ++r) {
                    const int tok = t + 16 * r, col = (int)p.by_page.div(tok);
                    if (col - wcol >= 32) {
                        wcol += 32;
                        cur = nxt;
                        nxt = wcol + 32 + lane < ncol ? __ldg(bt + wcol + 32 + lane) : -1;
                    }
                    page[r] = __shfl_sync(0xffffffffu, cur, (col - wcol) & 31);
                    at[r] = tok - col * a.page_size;
                    plain = plain && (uint32_t)page[r] < p.n_pages;
                }
            }
            if (plain) {
#pragma unroll
                for (int r = 0; r < C::R; ++r) {
                    const char *k = kb + page[r] * p.k_page + at[r] * p.k_tok;
#pragma unroll
                    for (int h = 0; h < 2; ++h)
#pragma unroll
                        for (int i = 0; i < C::KCH; ++i)
                            if ((4 * i + c) * (16 / C::ES) < p.k_dim) kr[r][h][i] = ld16(k + h * p.k_tok8 + i * 64);
                }
            } else {
                k_on = 0;
#pragma unroll
                for (int r = 0; r < C::R; ++r)
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        const int64_t off = row_at(t, r, g + 8 * h, p.k_page, p.k_tok);
                        if (off >= 0) k_on |= 1u << (2 * r + h);
#pragma unroll
                        for (int i = 0; i < C::KCH; ++i) {
                            kr[r][h][i] = make_uint4(0u, 0u, 0u, 0u);
                            if (off >= 0 && (4 * i + c) * (16 / C::ES) < p.k_dim)
                                kr[r][h][i] = ld16(kb + (off - g * p.k_tok) + i * 64);
                        }
                    }
            }
        };
        auto ldv = [&](uint32_t(&w)[C::VB / 4], const char *q) {
            if constexpr (C::VB == 16) {
                const uint4 x = ld16(q);
                w[0] = x.x; w[1] = x.y; w[2] = x.z; w[3] = x.w;
            } else {
                const uint2 x = ld8(q);
                w[0] = x.x; w[1] = x.y;
            }
        };
        auto request_values = [&](int t) {
            if (plain) {
#pragma unroll
                for (int r = 0; r < C::R; ++r) {
                    const char *v = vb + page[r] * p.v_page + at[r] * p.v_tok;
#pragma unroll
                    for (int k = 0; k < 4; ++k)
#pragma unroll
                        for (int i = 0; i < C::VCH; ++i)
                            if ((8 * i + g) * C::VE < p.v_dim)
                                ldv(vr[r][k][i], v + (k & 1) * p.v_tok + (k >> 1) * p.v_tok8 + i * (8 * C::VB));
                }
            } else {
#pragma unroll
                for (int r = 0; r < C::R; ++r)
#pragma unroll
                    for (int k = 0; k < 4; ++k) {
                        const int64_t off = row_at(t, r, 2 * c + (k & 1) + 8 * (k >> 1), p.v_page, p.v_tok);
#pragma unroll
                        for (int i = 0; i < C::VCH; ++i) {
#pragma unroll
                            for (int j = 0; j < C::VB / 4; ++j) vr[r][k][i][j] = 0u;
                            if (off >= 0 && (8 * i + g) * C::VE < p.v_dim)
                                ldv(vr[r][k][i], vb + (off - 2 * c * p.v_tok) + i * (8 * C::VB));
                        }
                    }
            }
        };

        request_keys(tok0 + first * C::TT);

        // Query fragments, through this warp's shared memory.  fac: what turns
        // an accumulator into a logit in units of log 2.
        uint32_t qf[C::QS ? 1 : C::QFRAGS][2];
        float fac[NT][2];
        constexpr int EC = 16 / C::ES;
#pragma unroll 1
        for (int nt = 0; nt < NT; ++nt) {
            const bool on = nt * 8 + g < heads;
            const int64_t qat = b * a.q_stride_b + (int64_t)(h0 + nt * 8 + g) * a.q_stride_h;
            float pw = 1.f, inv = 1.f;
            if (F16) {
                float top = 0.f;
#pragma unroll 1
                for (int i = 0; i < C::KCH * (EC / 8); ++i) {
                    const int d = (4 * (i / (EC / 8)) + c) * EC + 8 * (i % (EC / 8));
                    float v[8];
                    if (!on || d >= p.k_dim) continue;
                    load_q(p, qat + d, v);
#pragma unroll
                    for (int e = 0; e < 8; ++e) top = fmaxf(top, fabsf(v[e]));
                }
                top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 1));
                top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 2));
                int ex = (int)(__float_as_uint(top) >> 23) - 127;
                ex = top > 0.f ? max(-126, min(126, ex)) : 0;
                pw = __uint_as_float((uint32_t)(127 + ex) << 23);
                inv = __uint_as_float((uint32_t)(127 - ex) << 23);
            }
#pragma unroll 1
            for (int i = 0; i < C::KCH * (EC / 8); ++i) {
                const int d = (4 * (i / (EC / 8)) + c) * EC + 8 * (i % (EC / 8));
                float v[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
                if (on && d < p.k_dim) load_q(p, qat + d, v);
#pragma unroll
                for (int w = 0; w < 2; ++w) {
                    float x[4];
#pragma unroll
                    for (int e = 0; e < 4; ++e) x[e] = v[4 * w + e] * inv;
#pragma unroll
                    for (int q = 0; q < C::NQ; ++q) {
                        const uint2 pk = make_uint2(pack2<F16>(x[0], x[1]), pack2<F16>(x[2], x[3]));
                        qsm[((q * NT + nt) * C::KSTEPS + 2 * i + w) * 32 + lane] = pk;
                        const float2 r0 = unpack2<F16>(pk.x), r1 = unpack2<F16>(pk.y);
                        x[0] -= r0.x; x[1] -= r0.y; x[2] -= r1.x; x[3] -= r1.y;
                    }
                }
            }
            const float f0 = a.scale * a.k_scale * 1.4426950408889634f;
            const float f1 = f0 * __shfl_sync(0xffffffffu, pw, (2 * c) * 4);
            const float f2 = f0 * __shfl_sync(0xffffffffu, pw, (2 * c + 1) * 4);
            if (NT == 1 || nt == 0) fac[0][0] = f1, fac[0][1] = f2;
            else fac[NT - 1][0] = f1, fac[NT - 1][1] = f2;
        }
        __syncwarp();
        if constexpr (!C::QS) {
#pragma unroll
            for (int f = 0; f < C::QFRAGS; ++f) {
                const uint2 w = qsm[f * 32 + lane];
                qf[f][0] = w.x;
                qf[f][1] = w.y;
            }
        }

        // mo: the running maximum less kOff, so that weights come out times 2^kOff
        float o[NT][C::VW][4], mo[NT][2], l[NT][2];
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
            for (int w = 0; w < C::VW; ++w)
#pragma unroll
                for (int i = 0; i < 4; ++i) o[nt][w][i] = 0.f;
            mo[nt][0] = mo[nt][1] = kFloor;
            l[nt][0] = l[nt][1] = 0.f;
        }

#pragma unroll 1
        for (int step = first; step < last; ++step) {
            const int t = tok0 + step * C::TT;
            request_values(t);
            // S^T = K q^T
            float s[C::R][NT][4];
#pragma unroll
            for (int r = 0; r < C::R; ++r) {
#pragma unroll
                for (int nt = 0; nt < NT; ++nt) s[r][nt][0] = s[r][nt][1] = s[r][nt][2] = s[r][nt][3] = 0.f;
#pragma unroll
                for (int i = 0; i < C::KCH; ++i) {
                    constexpr int WORDS = C::ES == 1 ? 8 : 4;
                    uint32_t x[2][WORDS];
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        const uint32_t w[4] = {kr[r][h][i].x, kr[r][h][i].y, kr[r][h][i].z, kr[r][h][i].w};
#pragma unroll
                        for (int j = 0; j < 4; ++j) {
                            if constexpr (C::ES == 1) e4m3x4_to_f16x4(w[j], x[h][2 * j], x[h][2 * j + 1]);
                            else x[h][j] = w[j];
                        }
                    }
#pragma unroll
                    for (int w = 0; w < WORDS / 2; ++w)
#pragma unroll
                        for (int q = 0; q < C::NQ; ++q)
#pragma unroll
                            for (int nt = 0; nt < NT; ++nt) {
                                const int f = (q * NT + nt) * C::KSTEPS + i * (WORDS / 2) + w;
                                uint2 qq;
                                if constexpr (C::QS) qq = qsm[f * 32 + lane];
                                else qq = make_uint2(qf[f][0], qf[f][1]);
                                mma<F16>(s[r][nt], x[0][2 * w], x[1][2 * w], x[0][2 * w + 1], x[1][2 * w + 1], qq.x,
                                         qq.y);
                            }
                }
            }
            const bool masked = !plain;
            const uint32_t on = k_on;
            if (step + 1 < last) request_keys(t + C::TT);

            // softmax weights against the running maximum
#pragma unroll
            for (int r = 0; r < C::R; ++r)
#pragma unroll
                for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        s[r][nt][i] *= fac[nt][i & 1];
                        if (masked && !(on >> (2 * r + (i >> 1)) & 1u)) s[r][nt][i] = -INFINITY;
                    }
            float top[NT][2];
            bool move = false;
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                for (int k = 0; k < 2; ++k) {
                    top[nt][k] = fmaxf(s[0][nt][k], s[0][nt][k + 2]);
#pragma unroll
                    for (int r = 1; r < C::R; ++r)
                        top[nt][k] = fmaxf(top[nt][k], fmaxf(s[r][nt][k], s[r][nt][k + 2]));
                    move |= top[nt][k] > mo[nt][k] + (kLazy + C::kOff);
                }
            if (__any_sync(0xffffffffu, move)) {
#pragma unroll
                for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                    for (int k = 0; k < 2; ++k) {
                        float x = top[nt][k];
                        x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 4));
                        x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 8));
                        x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 16));
                        x = fmaxf(x - C::kOff, mo[nt][k]);
                        const float f = exp2_fast(mo[nt][k] - x);
                        mo[nt][k] = x;
                        l[nt][k] *= f;
#pragma unroll
                        for (int w = 0; w < C::VW; ++w) {
                            o[nt][w][k] *= f;
                            o[nt][w][k + 2] *= f;
                        }
                    }
            }
            uint32_t pb[C::R][NT][C::NP][2];
#pragma unroll
            for (int r = 0; r < C::R; ++r)
#pragma unroll
                for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
                    for (int i = 0; i < 4; ++i) s[r][nt][i] = exp2_fast(s[r][nt][i] - mo[nt][i & 1]);
                    l[nt][0] += s[r][nt][0] + s[r][nt][2];
                    l[nt][1] += s[r][nt][1] + s[r][nt][3];
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        float x = s[r][nt][2 * h], y = s[r][nt][2 * h + 1];
#pragma unroll
                        for (int q = 0; q < C::NP; ++q) {
                            const uint32_t pk = pack2<F16>(x, y);
                            pb[r][nt][q][h] = transpose8x8(pk);
                            const float2 z = unpack2<F16>(pk);
                            x -= z.x;
                            y -= z.y;
                        }
                    }
                }
            // O^T += V^T P^T
#pragma unroll
            for (int r = 0; r < C::R; ++r)
#pragma unroll
                for (int i = 0; i < C::VCH; ++i)
#pragma unroll
                    for (int j = 0; j < C::VB / 4; ++j) {
                        constexpr int PER = C::ES == 1 ? 2 : 1;  // pairs of dimensions a word
                        uint32_t w[4][PER];
#pragma unroll
                        for (int k = 0; k < 4; ++k) {
                            if constexpr (C::ES == 1) e4m3x4_to_f16x4(vr[r][k][i][j], w[k][0], w[k][1]);
                            else w[k][0] = vr[r][k][i][j];
                        }
#pragma unroll
                        for (int e = 0; e < PER; ++e) {
                            const uint32_t a0 = __byte_perm(w[0][e], w[1][e], 0x5410);
                            const uint32_t a1 = __byte_perm(w[0][e], w[1][e], 0x7632);
                            const uint32_t a2 = __byte_perm(w[2][e], w[3][e], 0x5410);
                            const uint32_t a3 = __byte_perm(w[2][e], w[3][e], 0x7632);
#pragma unroll
                            for (int q = 0; q < C::NP; ++q)
#pragma unroll
                                for (int nt = 0; nt < NT; ++nt)
                                    mma<F16>(o[nt][i * (C::VE / 2) + j * PER + e], a0, a1, a2, a3, pb[r][nt][q][0],
                                             pb[r][nt][q][1]);
                        }
                    }
        }

        // the segment's end, or the run's: the piece to shared memory, and, if
        // it is the whole segment, on to the output
        const bool whole = sb >= wb && se <= we;
        float *pc = pieces + (warp * 2 + (sb < wb ? 0 : 1)) * C::PIECE;
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int k = 0; k < 2; ++k) {
                const int row = nt * 8 + 2 * c + k;
                float sum = l[nt][k];
                sum += __shfl_xor_sync(0xffffffffu, sum, 4);
                sum += __shfl_xor_sync(0xffffffffu, sum, 8);
                sum += __shfl_xor_sync(0xffffffffu, sum, 16);
#pragma unroll
                for (int i = 0; i < C::VCH; ++i) {
                    float x[C::VE];
#pragma unroll
                    for (int j = 0; j < C::VE / 2; ++j) {
                        x[2 * j] = o[nt][i * (C::VE / 2) + j][k];
                        x[2 * j + 1] = o[nt][i * (C::VE / 2) + j][k + 2];
                    }
                    store_vec(pc + row * DMAX + (8 * i + g) * C::VE, x);
                }
                if (g == 0) {
                    pc[C::ROWS * DMAX + row] = mo[nt][k];
                    pc[C::ROWS * (DMAX + 1) + row] = sum;
                }
            }
        __syncwarp();
        if (whole)
            join_pieces<C::ROWS, DMAX>(p, [&](int) { return pc; }, 1, b, hg, nullptr, lane, 32);
        else if (lane == 0)
            slots[warp * 2 + (sb < wb ? 0 : 1)] = Slot{sb, se, b, hg};
        __syncwarp();
        u = min(se, we);
        sb = se;
        if (++hg == HG && u < we) {
            hg = 0;
            do ++b; while (prefix[b + 1] == prefix[b]);
            steps = prefix[b + 1] - prefix[b];
        }
    }
    __syncthreads();

    // the warps' pieces of each segment, in order
    int n_open = 0;
#pragma unroll 1
    for (int i = 0; i < 2 * C::WARPS;) {
        if (slots[i].b < 0) {
            ++i;
            continue;
        }
        const Slot sl = slots[i];
        // a warp leaves at most one piece of a segment: in its second place if
        // the segment starts there, in the first otherwise
        const int i0 = i;
        int n = 0;
        for (; i < 2 * C::WARPS; ++i) {
            if (slots[i].b < 0) continue;
            if (slots[i].begin != sl.begin) break;
            ++n;
        }
        const bool inside = sl.begin >= lo && sl.end <= hi;
        float *to = inside ? nullptr : p.part + (size_t)(2 * blockIdx.x + (sl.begin < lo ? 0 : 1)) * C::PIECE;
        if (!inside) {
            if (tid == 0) s_open[n_open] = sl;
            ++n_open;
        }
        join_pieces<C::ROWS, DMAX>(
            p, [&](int k) { return pieces + (k == 0 ? i0 : (i0 & ~1) + 2 * k) * C::PIECE; }, n, sl.b, sl.hg, to, tid,
            C::THREADS);
    }
    if (n_open == 0) return;

    // Segments shared with other blocks: the last block to arrive joins them.
    __threadfence();
    __syncthreads();
    if (tid < n_open) {
        const Slot &sl = s_open[tid];
        const int n = (int)((sl.end - 1) / per - sl.begin / per);
        int *cnt = p.arrived + sl.b * HG + sl.hg;
        if (atomicAdd(cnt, 1) == n) {
            *cnt = 0;  // for the next launch
            s_join[tid] = n;
        }
        __threadfence();
    }
    __syncthreads();
    for (int k = 0; k < n_open; ++k) {
        const int n = s_join[k] + 1;
        if (n == 0) continue;
        // A block's piece of a segment lies in its second place if the segment
        // starts there, in the first otherwise.  Maxima and sums come first, in
        // one round trip, as weights into shared memory (the warps' pieces have
        // been read); then the sums of O, eight pieces in flight.
        const Slot sl = s_open[k];
        const int c0 = (int)(sl.begin / per);
        auto piece = [&](int i) { return p.part + (size_t)(2 * (c0 + i) + (i == 0 ? 1 : 0)) * C::PIECE; };
        float *wm = pieces, *ws = pieces + n * C::ROWS;
        for (int e = tid; e < n * C::ROWS; e += C::THREADS) {
            const float *q = piece(e / C::ROWS) + C::ROWS * DMAX + e % C::ROWS;
            wm[e] = __ldcg(q);
            ws[e] = __ldcg(q + C::ROWS);
        }
        __syncthreads();
        const int kvh = sl.hg / p.n_groups, h0 = kvh * p.group + (sl.hg - kvh * p.n_groups) * C::ROWS;
        const int heads = min(C::ROWS, (kvh + 1) * p.group - h0);
#pragma unroll 1
        for (int e = tid; e < heads * (DMAX / 4); e += C::THREADS) {
            const int row = e / (DMAX / 4), d = 4 * (e - row * (DMAX / 4));
            if (d >= p.v_dim) continue;
            float top = kFloor, sum = 0.f, x[4] = {0.f, 0.f, 0.f, 0.f};
            for (int i = 0; i < n; ++i) top = fmaxf(top, wm[i * C::ROWS + row]);
#pragma unroll 1
            for (int i0 = 0; i0 < n; i0 += 8) {
                float4 v[8];
#pragma unroll
                for (int i = 0; i < 8; ++i)
                    if (i0 + i < n) v[i] = __ldcg(reinterpret_cast<const float4 *>(piece(i0 + i) + row * DMAX + d));
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    if (i0 + i >= n) break;
                    const float f = exp2_fast(wm[(i0 + i) * C::ROWS + row] - top);
                    sum = fmaf(ws[(i0 + i) * C::ROWS + row], f, sum);
                    x[0] = fmaf(v[i].x, f, x[0]);
                    x[1] = fmaf(v[i].y, f, x[1]);
                    x[2] = fmaf(v[i].z, f, x[2]);
                    x[3] = fmaf(v[i].w, f, x[3]);
                }
            }
            const bool none = sum == 0.f;
            const float inv = none ? 0.f : a.v_scale / sum;
#pragma unroll
            for (int j = 0; j < 4; ++j) x[j] = none ? 0.f : x[j] * inv;
            store_out(p, sl.b * a.out_stride_b + (h0 + row) * a.out_stride_h + d, x);
            if (d == 0 && a.lse)
                a.lse[(int64_t)sl.b * p.n_heads + h0 + row] =
                    none ? -INFINITY : (top + log2f(sum)) * 0.6931471805599453f;
        }
        __syncthreads();
    }
}

// Host: the kernel's function, its shared memory and its block for one form.
struct Form {
    void (*fn)(Params);
    size_t (*smem)(int);
    int threads, rows, step, piece;
};
template <int CT, int DMAX, int NT, bool WIDE>
Form form_of() {
    using C = Cfg<CT, DMAX, NT, WIDE>;
    return Form{attn_decode_kernel<CT, DMAX, NT, WIDE>, [](int n) { return C::smem(n); }, C::THREADS, C::ROWS, C::TT,
                C::PIECE};
}
// dmax 64, 128 or 256; groups of more than 8 heads take two tiles (not at 256,
// whose sums would not fit the registers: there a key head's groups share L2).
template <int CT>
Form pick(int dim, int group, bool wide) {
    const bool two = group > 8;
    if (dim <= 64) {
        if (two) return wide ? form_of<CT, 64, 2, true>() : form_of<CT, 64, 2, false>();
        return wide ? form_of<CT, 64, 1, true>() : form_of<CT, 64, 1, false>();
    }
    if (dim <= 128) {
        if (two) return wide ? form_of<CT, 128, 2, true>() : form_of<CT, 128, 2, false>();
        return wide ? form_of<CT, 128, 1, true>() : form_of<CT, 128, 1, false>();
    }
    return wide ? form_of<CT, 256, 1, true>() : form_of<CT, 256, 1, false>();
}
Form pick_f16(int dim, int group, bool wide);
Form pick_bf16(int dim, int group, bool wide);
Form pick_e4m3(int dim, int group, bool wide);

}  // namespace attn
}  // namespace moe
