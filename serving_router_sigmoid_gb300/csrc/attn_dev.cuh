// attn_dev.cuh -- attention of one new token per request over the paged
// key-value cache: the kernel.
//
//   s_j = scale q . k_j,  out = sum_j e^(s_j) v_j / sum_j e^(s_j)
//
// Every cache row is read once for 16 query heads of its key head (8 above 128
// dimensions), for 4 G flops a byte pair (G such heads): HBM bounds it as long as
// the bytes keep flowing.  So:
//
// - Work is split by cost, not by request.  All (request, key head) segments
//   are cut into steps of TT tokens; the steps, and kSegCost more for what a
//   segment costs by itself, form one line, and every warp of the grid (one
//   block per SM) takes an equal run of it, found from the lengths by each warp
//   itself.  A batch of one long and many short requests keeps every SM busy to
//   the end, with one launch and no plan on the host.
// - A warp needs no other warp until its run ends.  Rows go from HBM straight
//   into the registers of the tensor cores' fragments: with the tokens on the
//   MMA's M side a lane's 16 bytes of a key row ARE its A fragment (the order of
//   the contraction is free, the query takes the same order), and four pieces of
//   value rows become A fragments of V^T by byte permutes.  No shared memory, no
//   barrier, no transposition; a step is 8 KB (16 at 256 dimensions), its values
//   requested at its start and the next step's keys once its own are read.  (A
//   ring of cp.async copies in shared memory, 128 to 192 KB in flight, was slower
//   in every form: 64 x 4096 tokens E4M3 113 against 97 us.)
// - The heads of a group sit on N (8 a tile), so S^T = K q^T leaves each lane
//   the logits of its own two heads: the running maximum, the sum and the
//   rescale of O^T need no exchange.  The maximum moves only when a logit
//   passes it by 2^8 (one vote a step); weights stay below 2^8 and sums in fp32
//   do not care.
// - Where a run ends inside a segment, the warp leaves (O, m, l); the block
//   joins its warps' pieces, and of the blocks that share a segment the last to
//   arrive joins their pieces in block order, so the result does not depend on
//   who is last.
//
// Precision: products of the cache's own type (E4M3 codes widen exactly to
// f16) accumulate in fp32; logits, m, l and O are fp32.  A weight enters the
// second product in NP terms of 16 bits: 3 terms of bf16 keep 24 bits of it, 2
// of f16 keep 22; fp32 queries enter in as many.  For f16 products, and where a
// first bf16 term could round to infinity, each query row is scaled by a power of
// two to about 1, which the logit's factor undoes.  A weight below 2^-32 of the
// running maximum has no f16 term: it is in l, not in O.  16-bit queries on f16 and E4M3
// caches add every product to the running sum, which loses half an ulp at each (2 x
// 131072 tokens E4M3: 1.1% of the f16 outputs are not the rounded result, 0.7% of a
// plain fp32 form's; a rounded add a step brings 0.3%, and 112 us in place of 100
// for 64 x 4096 tokens).
//
// Measured: 64 requests of up to 32768 tokens, bf16, 8 key heads of 128 (1.8 GB):
// 272 us, 6.7 TB/s; 2 x 131072 tokens E4M3 (537 MB): 95 to 100 us, 5.5 TB/s; short
// calls are a chain of round trips (lengths, page ids, rows, joins): 1 x 777 tokens
// 9.6 us, 32 x 1024 fp32 queries, 16 key heads of 64: 24.8 us.  Pages that are no
// multiple of 16 tokens cost a division and a table load a row: 64 x 4096 tokens bf16
// 191 us in pages of 8 and 24, 226 of 1, against 169.5.
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
    int k_page, k_tok, k_head, v_page, v_tok, v_head;  // strides in bytes
    FastDiv by_page, by_hg;
    float *part;          // [2 grid] pieces
    int *arrived;         // [requests, key heads * groups]
};

constexpr int kSegCost = 4;         // what a segment costs besides its steps, in steps
constexpr int kShort = 4;           // steps a warp up to which a segment is not shared among blocks
constexpr int kGroupReq = 32;       // requests whose costs are summed together
constexpr float kLazy = 8.f;        // the maximum moves when a logit passes it by 2^kLazy
constexpr float kFloor = -3.4028235e38f;  // running maximum before any token: no logit lies below

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
    static constexpr int NP = kF16 ? 2 : 3;
    // Weighted values are summed over SUM tiles by the tensor cores and then added
    // to O in fp32; 0: every product goes straight into O (see the second product).
    static constexpr int SUM = WIDE ? 1 : kF16 ? 0 : R;
    static constexpr int ROWS = 8 * NT;
    static constexpr bool QS = NQ * NT * DMAX > 128;  // query fragments stay in shared memory
    // One block per SM.  12 warps of 168 registers up to 128 dimensions and 8 heads
    // (fp32 queries against 8 warps: 64 x 4096 tokens of 128 dimensions bf16 189 ->
    // 177 us, E4M3 121 -> 106, 32 ragged windows of 64 f16 26.8 -> 24.7, E4M3 22.3 ->
    // 23.4).  Larger forms would spill (256 dimensions E4M3 106 -> 145): 8, or the
    // 7 that shared memory holds with the largest query fragments.
    static constexpr int WARPS = DMAX <= 128 && NT == 1 ? 12 : DMAX * NT * NQ > 512 ? 7 : 8;
    static constexpr int THREADS = 32 * WARPS;
    static constexpr int PIECE = ROWS * (DMAX + 2);  // floats of a piece: O, m, l
    static constexpr int QFRAGS = NQ * NT * KSTEPS;
    static constexpr int QBYTES = QS ? QFRAGS * 256 : 0;
    // shared memory: a warp's first and last piece, and its query fragments
    static constexpr size_t kSmem = (size_t)WARPS * (2 * PIECE * 4 + QBYTES);
    static_assert(kSmem <= 227 * 1024 - 2048, "");
    // weights are held times 2^kOff: f16's subnormals then start at 2^-31 of the maximum
    static constexpr float kOff = kF16 ? 7.f : 0.f;
};

template <bool F16>
__device__ __forceinline__ void mma(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                    uint32_t b1) {
    if constexpr (F16)
        asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
                     "{%0,%1,%2,%3};"
                     : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
                     : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
    else
        asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
                     "{%0,%1,%2,%3};"
                     : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
                     : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
__device__ __forceinline__ uint32_t transpose8x8(uint32_t v) {
    uint32_t r;
    asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(v));
    return r;
}
__device__ __forceinline__ float exp2_fast(float x) {  // within 2^-22
    float r;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
    return r;
}
// A piece of a row, read once.  (No L2 prefetch beyond it: where a head's row is shorter than 256 bytes
// it fetches other heads' rows, whose readers come at other times.  64 x 4096
// tokens, 16 key heads of 64 dimensions, bf16: 239 us with 256-byte prefetches,
// 171 without; rows of 256 bytes lose 1% at most.)
__device__ __forceinline__ uint4 ld16(const char *p) {
    uint4 r;
    asm volatile("ld.global.L1::no_allocate.v4.u32 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r.x), "=r"(r.y), "=r"(r.z), "=r"(r.w)
                 : "l"(p));
    return r;
}
__device__ __forceinline__ uint2 ld8(const char *p) {
    uint2 r;
    asm volatile("ld.global.L1::no_allocate.v2.u32 {%0,%1}, [%2];" : "=r"(r.x), "=r"(r.y) : "l"(p));
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

// The tokens of request b that are seen: [from, len).
__device__ __forceinline__ void seen(const MoeAttnArgs &a, int b, int &from, int &len) {
    len = min(max(ld_in(a.seq_len + b), 0), a.max_pages * a.page_size);
    from = a.window > 0 ? max(0, len - a.window) : 0;
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

// A segment that several warps of a block share, or that reaches beyond it.
struct Shared {
    int b, hg;         // request, head group
    int warp, n;       // first warp that has a piece of it, warps that have
    int before, more;  // of its blocks, how many precede this one; how many there are beyond one
};

// Joins n pieces (O, m, l) of one segment, the i-th at piece(i): row and
// dimensions [d, d + 4) of it, into the output or into a piece `to`.
template <int ROWS, int DMAX, int BATCH, typename Piece>
__device__ __forceinline__ void join_pieces(const Params &p, Piece piece, int n, int b, int hg, int row, int d, float *to) {
    const int kvh = hg / p.n_groups, h0 = kvh * p.group + (hg - kvh * p.n_groups) * ROWS;
    if (h0 + row >= (kvh + 1) * p.group || d >= p.v_dim) return;
    float top = kFloor, sum = 0.f, x[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll 1
    for (int i0 = 0; i0 < n; i0 += BATCH) {  // a batch's loads go out together
        float pm[BATCH], pl[BATCH];
        float4 po[BATCH];
#pragma unroll
        for (int i = 0; i < BATCH; ++i) {
            pm[i] = kFloor;
            pl[i] = 0.f;
            po[i] = make_float4(0.f, 0.f, 0.f, 0.f);
            if (i0 + i < n) {
                const float *q = piece(i0 + i);
                pm[i] = q[ROWS * DMAX + row];
                pl[i] = q[ROWS * (DMAX + 1) + row];
                po[i] = *reinterpret_cast<const float4 *>(q + row * DMAX + d);
            }
        }
        float high = top;
#pragma unroll
        for (int i = 0; i < BATCH; ++i) high = fmaxf(high, pm[i]);
        const float keep = exp2_fast(top - high);
        top = high;
        sum *= keep;
#pragma unroll
        for (int j = 0; j < 4; ++j) x[j] *= keep;
#pragma unroll
        for (int i = 0; i < BATCH; ++i) {
            const float f = exp2_fast(pm[i] - top);
            sum = fmaf(pl[i], f, sum);
            x[0] = fmaf(po[i].x, f, x[0]);
            x[1] = fmaf(po[i].y, f, x[1]);
            x[2] = fmaf(po[i].z, f, x[2]);
            x[3] = fmaf(po[i].w, f, x[3]);
        }
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

__device__ __forceinline__ int warp_scan(int v, int lane) {  // inclusive
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int y = __shfl_up_sync(0xffffffffu, v, o);
        if (lane >= o) v += y;
    }
    return v;
}

template <int CT, int DMAX, int NT, bool WIDE>
__global__ void __launch_bounds__(Cfg<CT, DMAX, NT, WIDE>::THREADS, 1)
    attn_decode_kernel(const __grid_constant__ Params p) {
    using C = Cfg<CT, DMAX, NT, WIDE>;
    constexpr bool F16 = C::kF16;
    extern __shared__ __align__(16) char smem[];
    __shared__ int group_cost[MOE_MAX_REQUESTS / kGroupReq];
    __shared__ Shared shared[C::WARPS + 1];
    __shared__ int n_shared, last_of[2];
    after_previous();
    const MoeAttnArgs &a = p.a;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, g = lane >> 2, c = lane & 3;
    const int n_req = a.n_requests, HG = p.n_kv * p.n_groups;
    float *pieces = reinterpret_cast<float *>(smem);  // [2 warps]
    float *my_piece = pieces + 2 * warp * C::PIECE;   // a segment that began before the run; one that starts in it
    uint2 *qsm = reinterpret_cast<uint2 *>(pieces + 2 * C::WARPS * C::PIECE) + warp * C::QFRAGS * 32;

    // cost of each run of 32 requests (steps, and kSegCost for each request that has any)
    auto cost_of = [&](int b) {
        if (b >= n_req) return 0;
        int from, len;
        seen(a, b, from, len);
        return len > from ? (len - 1) / C::TT - from / C::TT + 1 + kSegCost : 0;
    };
    if (tid == 0) n_shared = 0;
    if (tid < 2) last_of[tid] = -1;
    const int n_run = (n_req + kGroupReq - 1) / kGroupReq;
    const int own_cost = n_run <= 1 ? cost_of(lane) : 0;
    for (int r = warp; r < n_run; r += C::WARPS) {
        const int b = r * kGroupReq + lane, n = n_run == 1 ? own_cost : cost_of(b);
        const int sum = warp_sum_i(n);
        if (lane == 0) group_cost[r] = sum;
        // requests that see nothing: zeros, by the blocks in turn
        unsigned none = __ballot_sync(0xffffffffu, b < n_req && n == 0 && b % gridDim.x == blockIdx.x);
        while (none) {
            const int e = r * kGroupReq + __ffs(none) - 1;
            none &= none - 1;
            const float z[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll 1
            for (int i = lane; i < p.n_heads * (p.v_dim / 4); i += 32) {
                const int h = i / (p.v_dim / 4), d = 4 * (i - h * (p.v_dim / 4));
                store_out(p, e * a.out_stride_b + h * a.out_stride_h + d, z);
            }
            if (a.lse)
                for (int h = lane; h < p.n_heads; h += 32) a.lse[(int64_t)e * p.n_heads + h] = -INFINITY;
        }
    }
    __syncthreads();
    // (one run of requests at most: every warp has looked at it itself)
    int run = -1, run_below = 0, run_cost = 0, run_before = 0;  // the run last looked at: its costs and their sums
    int total = 0;
    if (n_run <= 1) {
        run = 0;
        run_cost = own_cost;
        total = warp_scan(run_cost, lane);
        run_before = total - run_cost;
        total = __shfl_sync(0xffffffffu, total, 31);
    } else {
        for (int r = lane; r < n_run; r += 32) total += group_cost[r];
        total = warp_sum_i(total);
    }
    const int U = total * HG;

    // The segment at a place of the line: its request, head group, first place
    // (kSegCost before its first step) and cost; by the warp, from the runs of 32
    // requests and then the run's requests.
    struct Segment { int b, hg, begin, cost; };
    auto locate = [&](int x) {
        const int key = (int)p.by_hg.div(x);  // place / head groups
        int r = 0, below = 0;
#pragma unroll 1
        for (int r0 = 0; n_run > 1 && r0 < n_run; r0 += 32) {
            const int v = r0 + lane < n_run ? group_cost[r0 + lane] : 0, s = warp_scan(v, lane) - v;
            const unsigned m = __ballot_sync(0xffffffffu, v > 0 && below + s <= key);
            const int all = __shfl_sync(0xffffffffu, s + v, 31);
            if (m && key < below + all) {
                const int l = 31 - __clz(m);
                below += __shfl_sync(0xffffffffu, s, l);
                r = r0 + l;
                break;
            }
            below += all;
        }
        if (r != run) {
            run = r;
            run_below = below;
            run_cost = cost_of(r * kGroupReq + lane);
            run_before = warp_scan(run_cost, lane) - run_cost;
        }
        const unsigned m = __ballot_sync(0xffffffffu, run_cost > 0 && run_below + run_before <= key);
        const int l = 31 - __clz(m);
        Segment sg;
        sg.b = run * kGroupReq + l;
        sg.cost = __shfl_sync(0xffffffffu, run_cost, l);
        sg.begin = (run_below + __shfl_sync(0xffffffffu, run_before, l)) * HG;
        sg.hg = (x - sg.begin) / sg.cost;
        sg.begin += sg.hg * sg.cost;
        return sg;
    };

    // This block's run of the line.  A boundary inside a short segment moves to
    // its nearer end: sharing a segment among blocks costs more (some 4 us: fence,
    // arrival, the last block's join) than the steps it would even out.
    int per = (U + gridDim.x - 1) / gridDim.x;
    if (per < C::WARPS) per = C::WARPS;
    auto boundary = [&](long long x) {
        if (x >= U) return U;
        if (x == 0) return 0;
        const Segment sg = locate((int)x);
        if (sg.cost > kShort * C::WARPS) return (int)x;
        return 2 * ((int)x - sg.begin) < sg.cost ? sg.begin : sg.begin + sg.cost;
    };
    if ((long long)blockIdx.x * per >= U) return;
    const int lo = boundary((long long)blockIdx.x * per), hi = boundary((long long)(blockIdx.x + 1) * per);
    if (lo >= hi) return;
    // and this warp's
    const int per_w = (hi - lo + C::WARPS - 1) / C::WARPS;
    const int wb = min(lo + warp * per_w, hi), we = min(wb + per_w, hi);

    int b = 0, hg = 0, from = 0, len = 0, steps = 0;
    int sb = 0;  // first step of the segment (b, hg) on the line, past its own cost
    if (wb < we) {
        const Segment sg = locate(wb);
        b = sg.b;
        hg = sg.hg;
        sb = sg.begin + kSegCost;
        steps = sg.cost - kSegCost;
        seen(a, b, from, len);
    }
    for (int u = wb; u < we;) {
        const int se = sb + steps;
        const int first = max(u, sb) - sb, last = min(se, we) - sb;
        if (first < last) {
            const int kvh = hg / p.n_groups, h0 = kvh * p.group + (hg - kvh * p.n_groups) * C::ROWS;
            const int heads = min(C::ROWS, (kvh + 1) * p.group - h0);
            const int tok0 = from / C::TT * C::TT;

            // page ids of the next 64 pages, a window of 32 in each register
            const int32_t *bt = a.block_table + b * a.table_stride;
            int wcol = 0, cur = -1, nxt = -1;
            const int ncol = (int)p.by_page.div(len - 1) + 1;
            if (p.by16) {
                wcol = (int)p.by_page.div(tok0 + first * C::TT);
                cur = wcol + lane < ncol ? ld_in(bt + wcol + lane) : -1;
                nxt = wcol + 32 + lane < ncol ? ld_in(bt + wcol + 32 + lane) : -1;
            }

            // this lane's pieces of the query, on their way before the first keys
            constexpr int EC = 16 / C::ES, NI = C::KCH * EC / 8;
            uint4 qraw[NT][NI][WIDE ? 2 : 1];
            auto q_dim = [&](int i) { return (4 * (i / (EC / 8)) + c) * EC + 8 * (i % (EC / 8)); };
            const int q_bytes = a.act_type == MOE_F32 ? 4 : 2;
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
                const char *q = static_cast<const char *>(a.q) +
                                (b * a.q_stride_b + (int64_t)(h0 + nt * 8 + g) * a.q_stride_h) * q_bytes;
#pragma unroll
                for (int i = 0; i < NI; ++i) {
                    const bool in = nt * 8 + g < heads && q_dim(i) < p.k_dim;
                    const char *s = q + q_dim(i) * q_bytes;
                    if (!p.q16) {  // rows off 16 bytes: by twos, through shared memory
                        char *mine = reinterpret_cast<char *>(my_piece + C::PIECE) + lane * 32;
#pragma unroll 1
                        for (int e = 0; in && e < 8 * q_bytes; e += 2)
                            *reinterpret_cast<uint16_t *>(mine + e) = *reinterpret_cast<const uint16_t *>(s + e);
                        s = mine;
                    }
                    qraw[nt][i][0] = make_uint4(0u, 0u, 0u, 0u);
                    if (WIDE) qraw[nt][i][WIDE ? 1 : 0] = make_uint4(0u, 0u, 0u, 0u);
                    if (in) {
                        qraw[nt][i][0] = *reinterpret_cast<const uint4 *>(s);
                        if (WIDE && q_bytes == 4) qraw[nt][i][WIDE ? 1 : 0] = *reinterpret_cast<const uint4 *>(s + 16);
                    }
                }
            }
            if (!p.q16) __syncwarp();

            const char *kb = static_cast<const char *>(a.k_cache) + (int64_t)kvh * p.k_head +
                             (int64_t)g * p.k_tok + c * 16;
            const char *vb = static_cast<const char *>(a.v_cache) + (int64_t)kvh * p.v_head +
                             2 * (int64_t)c * p.v_tok + g * C::VB;
            // A step is `plain` when all its tokens are seen and lie on whole
            // pages: its rows are then at fixed distances from one address a tile.
            // (One branch for all of them: a branch a row cost 800 of a step's 3300
            // cycles.  Pieces beyond the head's size stay the zeros they are.)
            uint4 kr[C::R][2][C::KCH];
            uint32_t vr[C::R][4][C::VCH][C::VB / 4];
#pragma unroll
            for (int r = 0; r < C::R; ++r) {
#pragma unroll
                for (int i = 0; i < 2 * C::KCH; ++i) kr[r][i / C::KCH][i % C::KCH] = make_uint4(0u, 0u, 0u, 0u);
#pragma unroll
                for (int k = 0; k < 4; ++k)
#pragma unroll
                    for (int i = 0; i < C::VCH; ++i)
#pragma unroll
                        for (int j = 0; j < C::VB / 4; ++j) vr[r][k][i][j] = 0u;
            }
            int page[C::R], at[C::R];
            bool plain = false, holes = false;  // holes: a page that is none came by
            auto row_at = [&](int t, int r, int row, int sp, int st) -> int64_t {  // from row 0; -1: not seen
                const int tok = t + 16 * r + row;
                if (tok < from || tok >= len) return -1;
                int pg, in;
                if (p.by16) {
                    pg = page[r];
                    in = at[r] + row;
                } else {
                    const int col = (int)p.by_page.div(tok);
                    pg = ld_in(bt + col);
                    in = tok - col * a.page_size;
                }
                if ((uint32_t)pg >= p.n_pages) {
                    holes = true;
                    return -1;
                }
                return (int64_t)pg * sp + (int64_t)in * st;
            };
            auto fetch_key = [&](int r, int h, int i, const char *k) {
                if ((4 * i + c) * EC < p.k_dim) kr[r][h][i] = ld16(k + i * 64);
            };
            auto fetch_value = [&](int r, int k, int i, const char *v) {
                if ((8 * i + g) * C::VE >= p.v_dim) return;
                uint32_t(&w)[C::VB / 4] = vr[r][k][i];
                if constexpr (C::VB == 16) {
                    const uint4 x = ld16(v + i * 128);
                    w[0] = x.x; w[1] = x.y; w[2] = x.z; w[3] = x.w;
                } else {
                    const uint2 x = ld8(v + i * 64);
                    w[0] = x.x; w[1] = x.y;
                }
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
                            nxt = wcol + 32 + lane < ncol ? ld_in(bt + wcol + 32 + lane) : -1;
                        }
                        page[r] = __shfl_sync(0xffffffffu, cur, (col - wcol) & 31);
                        at[r] = tok - col * a.page_size;
                        plain = plain && (uint32_t)page[r] < p.n_pages;
                    }
                }
                if (plain) {
#pragma unroll
                    for (int r = 0; r < C::R; ++r) {
                        const char *k = kb + (int64_t)page[r] * p.k_page + (int64_t)at[r] * p.k_tok;
#pragma unroll
                        for (int h = 0; h < 2; ++h)
#pragma unroll
                            for (int i = 0; i < C::KCH; ++i) fetch_key(r, h, i, k + h * 8 * (int64_t)p.k_tok);
                    }
                    return;
                }
#pragma unroll
                for (int r = 0; r < C::R; ++r)
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        const int64_t off = row_at(t, r, g + 8 * h, p.k_page, p.k_tok);
#pragma unroll
                        for (int i = 0; i < C::KCH; ++i) {
                            kr[r][h][i] = make_uint4(0u, 0u, 0u, 0u);
                            if (off >= 0) fetch_key(r, h, i, kb + (off - (int64_t)g * p.k_tok));
                        }
                    }
            };
            auto request_values = [&](int t) {
                if (plain) {
#pragma unroll
                    for (int r = 0; r < C::R; ++r) {
                        const char *v = vb + (int64_t)page[r] * p.v_page + (int64_t)at[r] * p.v_tok;
#pragma unroll
                        for (int k = 0; k < 4; ++k)
#pragma unroll
                            for (int i = 0; i < C::VCH; ++i)
                                fetch_value(r, k, i, v + ((k & 1) + (k >> 1) * 8) * (int64_t)p.v_tok);
                    }
                    return;
                }
#pragma unroll
                for (int r = 0; r < C::R; ++r)
#pragma unroll
                    for (int k = 0; k < 4; ++k) {
                        const int64_t off = row_at(t, r, 2 * c + (k & 1) + 8 * (k >> 1), p.v_page, p.v_tok);
#pragma unroll
                        for (int i = 0; i < C::VCH; ++i) {
#pragma unroll
                            for (int j = 0; j < C::VB / 4; ++j) vr[r][k][i][j] = 0u;
                            if (off >= 0) fetch_value(r, k, i, vb + (off - 2 * (int64_t)c * p.v_tok));
                        }
                    }
            };

            // Query fragments.  fac: what turns an accumulator into a logit in
            // units of log 2.
            uint32_t qf[C::QS ? 1 : C::QFRAGS][2];
            float fac[NT][2];
            auto build_query = [&]() {
#pragma unroll
                for (int nt = 0; nt < NT; ++nt) {
                    float v[NI][8];
    #pragma unroll
                    for (int i = 0; i < NI; ++i) {
                        const uint4 x = qraw[nt][i][0], y = qraw[nt][i][WIDE ? 1 : 0];
                        const uint32_t w[8] = {x.x, x.y, x.z, x.w, y.x, y.y, y.z, y.w};
                        if (WIDE && a.act_type == MOE_F32) {
    #pragma unroll
                            for (int e = 0; e < 8; ++e) v[i][e] = __uint_as_float(w[e]);
                        } else {
    #pragma unroll
                            for (int e = 0; e < 4; ++e) {
                                const float2 f = a.act_type == MOE_F16 ? half_pair(w[e], __half())
                                                                       : half_pair(w[e], __nv_bfloat16());
                                v[i][2 * e] = f.x;
                                v[i][2 * e + 1] = f.y;
                            }
                        }
                    }
                    float pw = 1.f;
                    if (F16 || WIDE) {
                        float top = 0.f;
    #pragma unroll
                        for (int i = 0; i < NI; ++i)
    #pragma unroll
                            for (int e = 0; e < 8; ++e) top = fmaxf(top, fabsf(v[i][e]));
                        top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 1));
                        top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 2));
                        int ex = (int)(__float_as_uint(top) >> 23) - 127;
                        ex = top > 0.f ? max(-126, min(126, ex)) : 0;
                        pw = __uint_as_float((uint32_t)(127 + ex) << 23);
                        const float inv = __uint_as_float((uint32_t)(127 - ex) << 23);
    #pragma unroll
                        for (int i = 0; i < NI; ++i)
    #pragma unroll
                            for (int e = 0; e < 8; ++e) v[i][e] *= inv;
                    }
    #pragma unroll
                    for (int i = 0; i < NI; ++i)
    #pragma unroll
                        for (int w = 0; w < 2; ++w) {
                            float x[4] = {v[i][4 * w], v[i][4 * w + 1], v[i][4 * w + 2], v[i][4 * w + 3]};
    #pragma unroll
                            for (int q = 0; q < C::NQ; ++q) {
                                const uint2 pk = make_uint2(pack2<F16>(x[0], x[1]), pack2<F16>(x[2], x[3]));
                                const int f = (q * NT + nt) * C::KSTEPS + 2 * i + w;
                                if constexpr (C::QS) {
                                    qsm[f * 32 + lane] = pk;
                                } else {
                                    qf[f][0] = pk.x;
                                    qf[f][1] = pk.y;
                                }
                                const float2 r0 = unpack2<F16>(pk.x), r1 = unpack2<F16>(pk.y);
                                x[0] -= r0.x; x[1] -= r0.y; x[2] -= r1.x; x[3] -= r1.y;
                            }
                        }
                    const float f0 = a.scale * a.k_scale * 1.4426950408889634f;
                    fac[nt][0] = f0 * __shfl_sync(0xffffffffu, pw, (2 * c) * 4);
                    fac[nt][1] = f0 * __shfl_sync(0xffffffffu, pw, (2 * c + 1) * 4);
                }
            };

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

            request_keys(tok0 + first * C::TT);
            build_query();
#pragma unroll 1
            for (int step = first; step < last; ++step) {
                const int t = tok0 + step * C::TT;
                request_values(t);
                // S^T = K q^T
                float s[C::R][NT][4];
#pragma unroll
                for (int r = 0; r < C::R; ++r)
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                        for (int i = 0; i < 4; ++i) s[r][nt][i] = 0.f;
#pragma unroll
                for (int i = 0; i < C::KCH; ++i)
#pragma unroll
                    for (int r = 0; r < C::R; ++r) {
                        constexpr int WORDS = C::ES == 1 ? 8 : 4;
                        uint32_t x[2][WORDS];
#pragma unroll
                        for (int h = 0; h < 2; ++h) {
                            const uint4 y = kr[r][h][i];
                            const uint32_t w[4] = {y.x, y.y, y.z, y.w};
#pragma unroll
                            for (int j = 0; j < 4; ++j) {
                                if constexpr (C::ES == 1) e4m3x4_to_f16x4(w[j], x[h][2 * j], x[h][2 * j + 1]);
                                else x[h][j] = w[j];
                            }
                        }
                        float part[WIDE ? NT : 1][4];  // (see the second product)
                        if constexpr (WIDE) {
#pragma unroll
                            for (int e = 0; e < NT * 4; ++e) part[e / 4][e % 4] = 0.f;
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
                                    mma<F16>(WIDE ? part[WIDE ? nt : 0] : s[r][nt],
                                             x[0][2 * w], x[1][2 * w], x[0][2 * w + 1], x[1][2 * w + 1], qq.x, qq.y);
                                }
                        if constexpr (WIDE) {
#pragma unroll
                            for (int e = 0; e < NT * 4; ++e) s[r][e / 4][e % 4] += part[e / 4][e % 4];
                        }
                    }

                if (step + 1 < last) request_keys(t + C::TT);

                // softmax weights against the running maximum
#pragma unroll
                for (int r = 0; r < C::R; ++r)
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                        for (int i = 0; i < 4; ++i) s[r][nt][i] *= fac[nt][i & 1];
                if (t < from || t + C::TT > len || __any_sync(0xffffffffu, holes)) {
#pragma unroll
                    for (int r = 0; r < C::R; ++r)
#pragma unroll
                        for (int h = 0; h < 2; ++h) {
                            const int tok = t + 16 * r + g + 8 * h;
                            bool on = tok >= from && tok < len;
                            if (on && holes) on = (uint32_t)ld_in(bt + p.by_page.div(tok)) < p.n_pages;
                            if (!on) {
#pragma unroll
                                for (int nt = 0; nt < NT; ++nt) s[r][nt][2 * h] = s[r][nt][2 * h + 1] = -INFINITY;
                            }
                        }
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
                            if constexpr (F16) {
#pragma unroll
                                for (int q = 0; q < C::NP; ++q) {
                                    const uint32_t pk = pack2<F16>(x, y);
                                    pb[r][nt][q][h] = transpose8x8(pk);
                                    const float2 z = unpack2<F16>(pk);
                                    x -= z.x;
                                    y -= z.y;
                                }
                            } else {
                                // bf16 terms by cutting, 8 bits each, exactly: a weight's
                                // upper half is its first term.  Both halves change
                                // lanes, and the rest is cut up there.
                                const uint32_t a = __float_as_uint(x), e = __float_as_uint(y);
                                const uint32_t hi = transpose8x8(__byte_perm(a, e, 0x7632));
                                const uint32_t lo = transpose8x8(__byte_perm(a, e, 0x5410));
                                pb[r][nt][0][h] = hi;
                                x = __uint_as_float(__byte_perm(lo, hi, 0x5410)) - __uint_as_float(hi << 16);
                                y = __uint_as_float(__byte_perm(lo, hi, 0x7632)) - __uint_as_float(hi & 0xFFFF0000u);
#pragma unroll
                                for (int q = 1; q < C::NP; ++q) {
                                    pb[r][nt][q][h] = __byte_perm(__float_as_uint(x), __float_as_uint(y), 0x7632);
                                    x -= __uint_as_float(__float_as_uint(x) & 0xFFFF0000u);
                                    y -= __uint_as_float(__float_as_uint(y) & 0xFFFF0000u);
                                }
                            }
                        }
                    }

                // O^T += V^T P^T.  The tensor cores cut a sum's last bits off, and do so
                // with O's own each time they add to it.  Over many steps that shows (fp32
                // outputs of 24 x 8192 tokens: 3.3e-6; bf16 caches, 64 ragged requests:
                // other last places in 0.2% of the outputs), so fp32 queries and bf16
                // caches take a step's products by a rounded add, fp32 ones of each tile.
#pragma unroll
                for (int r0 = 0; r0 < C::R; r0 += C::SUM ? C::SUM : C::R)
#pragma unroll
                    for (int i = 0; i < C::VCH; ++i) {
                        // (two words together, so that an accumulator's terms do not
                        // follow one another)
                        constexpr int PER = C::ES == 1 ? 2 : 1;  // pairs of dimensions a word
#pragma unroll
                        for (int j = 0; j < C::VB / 4; j += 2) {
                            float part[C::SUM ? 2 * PER : 1][NT][4];
                            if constexpr (C::SUM > 0) {
#pragma unroll
                                for (int x = 0; x < 2 * PER * NT * 4; ++x) part[x / (NT * 4)][x / 4 % NT][x % 4] = 0.f;
                            }
#pragma unroll
                            for (int r = r0; r < r0 + (C::SUM ? C::SUM : C::R); ++r) {
                                uint32_t am[2 * PER][4];
#pragma unroll
                                for (int jj = 0; jj < 2; ++jj) {
                                    const uint32_t w0 = vr[r][0][i][j + jj], w1 = vr[r][1][i][j + jj],
                                                   w2 = vr[r][2][i][j + jj], w3 = vr[r][3][i][j + jj];
                                    uint32_t(&m)[4] = am[jj * PER];
                                    if constexpr (C::ES == 1) {  // a dimension's codes of two tokens side by side
                                        uint32_t(&m1)[4] = am[jj * PER + PER - 1];
                                        e4m3x4_to_f16x4(__byte_perm(w0, w1, 0x5140), m[0], m[1]);
                                        e4m3x4_to_f16x4(__byte_perm(w2, w3, 0x5140), m[2], m[3]);
                                        e4m3x4_to_f16x4(__byte_perm(w0, w1, 0x7362), m1[0], m1[1]);
                                        e4m3x4_to_f16x4(__byte_perm(w2, w3, 0x7362), m1[2], m1[3]);
                                    } else {
                                        m[0] = __byte_perm(w0, w1, 0x5410);
                                        m[1] = __byte_perm(w0, w1, 0x7632);
                                        m[2] = __byte_perm(w2, w3, 0x5410);
                                        m[3] = __byte_perm(w2, w3, 0x7632);
                                    }
                                }
#pragma unroll
                                for (int q = 0; q < C::NP; ++q)
#pragma unroll
                                    for (int e = 0; e < 2 * PER; ++e)
#pragma unroll
                                        for (int nt = 0; nt < NT; ++nt)
                                            mma<F16>(C::SUM ? part[C::SUM ? e : 0][nt]
                                                            : o[nt][i * (C::VE / 2) + j * PER + e],
                                                     am[e][0], am[e][1], am[e][2], am[e][3], pb[r][nt][q][0],
                                                     pb[r][nt][q][1]);
                            }
                            if constexpr (C::SUM > 0) {
#pragma unroll
                                for (int x = 0; x < 2 * PER * NT * 4; ++x)
                                    o[x / 4 % NT][i * (C::VE / 2) + j * PER + x / (NT * 4)][x % 4] +=
                                        part[x / (NT * 4)][x / 4 % NT][x % 4];
                            }
                        }
                    }
            }
            __syncwarp();

            // The segment's end, or the run's.  The whole segment goes to the
            // output, a piece of it to the block's join.
            const bool whole = sb >= wb && se <= we, before = sb < wb;
            float *pc = my_piece + (before ? 0 : C::PIECE);
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
            if (whole) {
#pragma unroll 1
                for (int e = lane; e < C::ROWS * (DMAX / 4); e += 32)
                    join_pieces<C::ROWS, DMAX, 1>(p, [&](int) { return pc; }, 1, b, hg, e / (DMAX / 4),
                                               4 * (e % (DMAX / 4)), nullptr);
                __syncwarp();
            } else if (lane == 0 && (!before || warp == 0)) {
                // the first warp of the block that has a piece lists the segment
                Shared &sh = shared[atomicAdd(&n_shared, 1)];
                sh.b = b;
                sh.hg = hg;
                sh.warp = warp;
                sh.n = (min(se, hi) - 1 - lo) / per_w - warp + 1;
                sh.before = sb < lo ? (int)blockIdx.x - sb / per : 0;
                // (no boundary inside a long segment moved, so the blocks are per apart)
                sh.more = sb >= lo && se <= hi ? 0 : (se - 1) / per - sb / per;
            }
        }
        u = min(se, we);
        if (u < we) {
            if (++hg == HG) {
                hg = 0;
                do {
                    ++b;
                    seen(a, b, from, len);
                } while (len <= from);
                steps = (len - 1) / C::TT - from / C::TT + 1;
            }
            sb = se + kSegCost;
        }
    }
    __syncthreads();

    // The warps' pieces of each shared segment, in order: into the output, or,
    // if other blocks have pieces too, into the block's own (its second place if
    // the segment starts here, the first otherwise).
    const int ns = n_shared;
    constexpr int CELLS = C::ROWS * (DMAX / 4);
#pragma unroll 1
    for (int e = tid; e < ns * CELLS; e += C::THREADS) {
        const Shared &sh = shared[e / CELLS];
        const int row = e % CELLS / (DMAX / 4), d = 4 * (e % (DMAX / 4));
        float *to = sh.more ? p.part + (size_t)(2 * blockIdx.x + (sh.before ? 0 : 1)) * C::PIECE : nullptr;
        // the first warp's piece began in its run, unless the segment did in another block
        const float *of = pieces + (2 * sh.warp + (sh.before ? 0 : 1)) * C::PIECE;
        const float *rest = pieces + 2 * sh.warp * C::PIECE;
        join_pieces<C::ROWS, DMAX, 8>(p, [&](int i) { return i == 0 ? of : rest + 2 * i * C::PIECE; }, sh.n, sh.b, sh.hg,
                                   row, d, to);
    }
    bool open = false;
    for (int k = 0; k < ns; ++k) open |= shared[k].more != 0;
    if (!open) return;

    // Segments shared with other blocks: the last block to arrive joins them.
    __syncthreads();
    if (tid < ns && shared[tid].more) {
        const Shared &sh = shared[tid];
        int *cnt = p.arrived + sh.b * HG + sh.hg;
        // release: the block's pieces (the barrier orders the other threads' before
        // this); acquire: those of the blocks that came before
        int arrived;
        asm volatile("atom.add.acq_rel.gpu.global.s32 %0, [%1], 1;" : "=r"(arrived) : "l"(cnt) : "memory");
        if (arrived == sh.more) {
            *cnt = 0;  // for the next launch
            last_of[sh.before ? 0 : 1] = tid;
        }
    }
    __syncthreads();
    for (int k = 0; k < 2; ++k) {
        if (last_of[k] < 0) continue;
        // Maxima and sums come first, in one round trip, as weights into shared
        // memory (the warps' pieces have been read); then the sums of O, kBatch
        // pieces in flight (51 pieces of 16 x 128: 12 us by eights).
        const Shared sh = shared[last_of[k]];
        constexpr int kBatch = C::THREADS <= 256 ? 24 : 16;
        const int n = sh.more + 1, c0 = blockIdx.x - sh.before;
        auto piece = [&](int i) { return p.part + (size_t)(2 * (c0 + i) + (i == 0 ? 1 : 0)) * C::PIECE; };
        float *wm = reinterpret_cast<float *>(smem), *ws = wm + n * C::ROWS;
        for (int e = tid; e < n * C::ROWS; e += C::THREADS) {
            const float *q = piece(e / C::ROWS) + C::ROWS * DMAX + e % C::ROWS;
            wm[e] = __ldcg(q);
            ws[e] = __ldcg(q + C::ROWS);
        }
        __syncthreads();
        const int kvh = sh.hg / p.n_groups, h0 = kvh * p.group + (sh.hg - kvh * p.n_groups) * C::ROWS;
        const int heads = min(C::ROWS, (kvh + 1) * p.group - h0);
#pragma unroll 1
        for (int e = tid; e < heads * (DMAX / 4); e += C::THREADS) {
            const int row = e / (DMAX / 4), d = 4 * (e - row * (DMAX / 4));
            if (d >= p.v_dim) continue;
            float top = kFloor, sum = 0.f, x[4] = {0.f, 0.f, 0.f, 0.f};
            for (int i = 0; i < n; ++i) top = fmaxf(top, wm[i * C::ROWS + row]);
#pragma unroll 1
            for (int i0 = 0; i0 < n; i0 += kBatch) {
                float4 v[kBatch];
#pragma unroll
                for (int i = 0; i < kBatch; ++i)
                    if (i0 + i < n) v[i] = __ldcg(reinterpret_cast<const float4 *>(piece(i0 + i) + row * DMAX + d));
#pragma unroll
                for (int i = 0; i < kBatch; ++i) {
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
            store_out(p, sh.b * a.out_stride_b + (h0 + row) * a.out_stride_h + d, x);
            if (d == 0 && a.lse)
                a.lse[(int64_t)sh.b * p.n_heads + h0 + row] =
                    none ? -INFINITY : (top + log2f(sum)) * 0.6931471805599453f;
        }
        __syncthreads();
    }
}

// Host: the kernel's function, its shared memory and its block for one form.
struct Form {
    void (*fn)(Params);
    size_t smem;
    int threads, rows, piece;
};
template <int CT, int DMAX, int NT, bool WIDE>
Form form_of() {
    using C = Cfg<CT, DMAX, NT, WIDE>;
    return Form{attn_decode_kernel<CT, DMAX, NT, WIDE>, C::kSmem, C::THREADS, C::ROWS, C::PIECE};
}
// dmax 64, 128 or 256; groups of more than 8 heads take two tiles (not at 256,
// whose sums would not fit the registers).  A key head with more query heads than
// that is a segment for each 16 (8) of them, and its rows are read again for each,
// at another time and by other SMs: 64 x 4096 tokens bf16, 256 heads on 8 key heads
// of 128 388 us, 128 heads 203; 64 heads on 4 key heads of 256 335, 32 heads 173.
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
