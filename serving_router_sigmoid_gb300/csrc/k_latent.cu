// k_latent.cu -- attention of one new token per request over a paged cache of
// latent rows that all heads share (moe_latent_decode):
//   s_hj = scale q_h . c_j,  out_h = sum_j e^(s_hj) c_j[0 .. latent) / sum_j e^(s_hj)
//
// A row of the cache (1152 bytes at 512 + 64 in 16 bits) serves 64 heads twice, as
// key and as value: 139 kflop, 121 a byte, which the legacy tensor pipe cannot do
// at HBM speed and tcgen05 can.  Both products take the same image of the rows in
// shared memory, 64 tokens by chunks of 64 dimensions with the 128-byte swizzle:
//   S [heads x tokens] = Q K^T: queries on M (64), tokens on N, K-major operands;
//   O^T [latent x heads] += V^T P^T: 128 latent dimensions on M, where the image is
//   an MN-major operand, the heads on N.  O (512 x 64 fp32) takes half of the
//   tensor memory; with the heads on M of both it would take all of it.
// A thread then holds whole rows of logits (a quarter, four lanes a row), O is
// scaled by columns, and the weights P go through shared memory as operand B.
//
// Per tile of 64 tokens the tensor core works 36 x 32 + 16 x 48 = 1920 cycles (the
// second product is bound by its operands' 128 bytes a cycle); HBM brings a tile in
// 3300 cycles a SM (16-bit) or 1650 (E4M3).
//
// - Work is split by cost: the tiles of all requests, and kSegCost more for each
//   request, form one line; each block takes an equal run, found from the lengths
//   by itself.  More than 64 heads form groups; the blocks of a run's groups are
//   neighbours and read the same rows at the same time, once from HBM.
// - Eight producer warps copy rows (cp.async, any page size and stride), or load
//   E4M3 codes and widen them, into two stages; one warp issues the MMAs: S of tile
//   i + 1 before O of tile i, so that the softmax of one runs under the products of
//   the other; four warps do the softmax and write the results.
// - The maximum moves only when a logit passes it by 2^kLazy; then O is scaled in
//   tensor memory.  Weights are rounded to the operand type (their sum is not), for
//   f16 times 2^7, so that its subnormals begin at 2^-31 of the maximum.
// - A request that several blocks share leaves its pieces (O, m, l) in the handle's
//   workspace; a second small launch joins them in order, so results do not depend
//   on timing.
#include "tc_dev.cuh"

namespace moe {
namespace {

using namespace tc;

__device__ int32_t g_err;  // flags since the last read

constexpr int kTile = 64;             // tokens
constexpr int kHeads = 64;            // of a group, at most
constexpr int kChunks = 9;            // of 64 dimensions: 512 + 64
constexpr uint32_t kChunk = kTile * 128;
constexpr uint32_t kStageB = kChunks * kChunk;
constexpr int kStages = 2;
constexpr int kProd = 8;              // producer warps
constexpr int kThreads = 32 * (4 + 1 + kProd);
constexpr uint32_t kOffQ = 0, kOffK = kStageB, kOffP = kOffK + kStages * kStageB;
constexpr size_t kSmem = kOffP + kHeads * 128 + 1024;
constexpr uint32_t kColS = 256;       // tensor memory: O 4 x 64 columns, then S twice
constexpr int kSegCost = 2;           // what a request costs besides its tiles, in tiles
constexpr float kLazy = 8.f;
constexpr float kFloor = -3.4028235e38f;  // maximum before any token: no logit lies below
constexpr float kLog2e = 1.4426950408889634f;

struct Params {
    MoeLatentArgs a;
    int heads, latent, dim;
    int groups, per_group, n;         // head groups, heads of one, the same as columns (a multiple of 16)
    int runs;
    float factor;                     // scale * k_scale * log2(e)
    FastDiv by_page;
    int64_t c_page, c_tok;            // bytes
    uint32_t n_pages;
    float *part;                      // [2 * blocks] pieces
    int4 *rec;                        // [blocks]: the request that begins and does not end in the block's run
};

__host__ __device__ inline int64_t piece_floats(int latent) { return (int64_t)kHeads * latent + 2 * kHeads; }

struct Shared {
    uint64_t full[kStages], empty[kStages], valid_full[kStages], q_full, q_empty, s_full[2], p_ready, pv_done, o_full, o_empty, drain;
    uint32_t valid[kStages][2];
    uint32_t tmem;
    int abort;
    int b0, s0;                       // the request where the run begins, and where that one begins on the line
    int sums[kThreads / 32];
    float factor[kHeads];
};

__device__ __forceinline__ int len_of(const MoeLatentArgs &a, int b) {
    return min(ld_in(a.seq_len + b), a.max_pages * a.page_size);
}
__device__ __forceinline__ int tiles_of(int len) { return len > 0 ? (len + kTile - 1) / kTile : 0; }

// The tiles of a run, request by request.
struct Walk {
    int b, s, hi, n;      // request, its begin on the line, end of the run, requests
    int len, tiles, t, te;
    __device__ __forceinline__ bool settle(const MoeLatentArgs &a, int lo) {
        for (;;) {
            if (b >= n || s >= hi) return false;
            len = len_of(a, b);
            tiles = tiles_of(len);
            if (tiles) {
                t = max(0, lo - s - kSegCost);
                te = min(tiles, hi - s - kSegCost);
                if (t < te) return true;
                s += kSegCost + tiles;
            }
            ++b;
        }
    }
    __device__ __forceinline__ bool start(const MoeLatentArgs &a, const Shared &sm, int lo, int hi_) {
        b = sm.b0;
        s = sm.s0;
        hi = hi_;
        n = a.n_requests;
        return lo < hi && settle(a, lo);
    }
    // the next tile; first: it opens another request
    __device__ __forceinline__ bool next(const MoeLatentArgs &a, bool &first) {
        first = false;
        if (++t < te) return true;
        first = true;
        s += kSegCost + tiles;
        ++b;
        return settle(a, 0);
    }
};

__device__ __forceinline__ float ex2(float x) {
    float r;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
    return r;
}
__device__ __forceinline__ void cp16(uint32_t dst, const void *src, bool live) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(live ? 16 : 0) : "memory");
}
__device__ __forceinline__ void cp_arrive(uint64_t *b) {  // once this thread's copies so far have landed
    asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(su32(b)) : "memory");
}
// two E4M3 codes -> two elements of the query's type (exact)
template <bool BF>
__device__ __forceinline__ uint32_t widen(uint32_t codes) {
    uint32_t h;
    asm("{ .reg .b16 a; cvt.u16.u32 a, %1; cvt.rn.f16x2.e4m3x2 %0, a; }" : "=r"(h) : "r"(codes));
    if (!BF) return h;
    const float2 f = half_pair(h, __half());
    return pack_pair(f.x, f.y, __nv_bfloat16());
}
template <bool BF>
__device__ __forceinline__ uint4 widen8(uint32_t a, uint32_t b) {
    return make_uint4(widen<BF>(a & 0xffff), widen<BF>(a >> 16), widen<BF>(b & 0xffff), widen<BF>(b >> 16));
}
// 16 lanes by 64 columns as matrix fragments: v[4 j ..] = rows lane / 4 and + 8, columns 8 j + 2 (lane % 4) and + 1
__device__ __forceinline__ void tmem_ld_rows(uint32_t at, uint32_t (&v)[32]) {
    asm volatile("tcgen05.ld.sync.aligned.16x256b.x8.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,%17,%18,%19,"
                 "%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];"
                 : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3]), "=r"(v[4]), "=r"(v[5]), "=r"(v[6]), "=r"(v[7]), "=r"(v[8]),
                   "=r"(v[9]), "=r"(v[10]), "=r"(v[11]), "=r"(v[12]), "=r"(v[13]), "=r"(v[14]), "=r"(v[15]), "=r"(v[16]),
                   "=r"(v[17]), "=r"(v[18]), "=r"(v[19]), "=r"(v[20]), "=r"(v[21]), "=r"(v[22]), "=r"(v[23]), "=r"(v[24]),
                   "=r"(v[25]), "=r"(v[26]), "=r"(v[27]), "=r"(v[28]), "=r"(v[29]), "=r"(v[30]), "=r"(v[31])
                 : "r"(at));
}
__device__ __forceinline__ bool soft_or(bool p) {
    uint32_t r;
    asm volatile("{\n .reg .pred pi, po;\n setp.ne.u32 pi, %1, 0;\n bar.red.or.pred po, 1, 128, pi;\n selp.u32 %0, 1, 0, po;\n}"
                 : "=r"(r) : "r"((uint32_t)p) : "memory");
    return r != 0;
}

template <bool BF, bool E4>
__global__ void __launch_bounds__(kThreads, 1) latent_decode_kernel(const __grid_constant__ Params p) {
    using T = typename Elem<BF ? MOE_BF16 : MOE_F16>::type;
    extern __shared__ uint8_t raw[];
    __shared__ Shared sm;
    uint8_t *dyn = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(raw) + 1023) & ~uintptr_t(1023));
    const uint32_t sbase = su32(dyn);
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const MoeLatentArgs &a = p.a;
    volatile int *abort = &sm.abort;

    if (tid == 0) {
        for (int i = 0; i < kStages; ++i) {
            mb_init(&sm.full[i], E4 ? kProd : 32 * kProd);
            mb_init(&sm.valid_full[i], kProd);
            mb_init(&sm.empty[i], 1);
            mb_init(&sm.s_full[i], 1);
        }
        mb_init(&sm.q_full, 32 * kProd);
        mb_init(&sm.q_empty, 1);
        mb_init(&sm.p_ready, 4);
        mb_init(&sm.pv_done, 1);
        mb_init(&sm.o_full, 1);
        mb_init(&sm.o_empty, 4);
        mb_init(&sm.drain, 1);
        sm.abort = 0;
        mb_init_done();
    }
    if (warp == 4) tmem_alloc(&sm.tmem, 512);
    after_previous();

    // the line of all tiles, and this block's run of it
    const int group = blockIdx.x % p.groups, run = blockIdx.x / p.groups;
    const int per = (a.n_requests + kThreads - 1) / kThreads;
    const int c0 = min(tid * per, a.n_requests), c1 = min(c0 + per, a.n_requests);
    int mine = 0;
    for (int b = c0; b < c1; ++b) {
        const int t = tiles_of(len_of(a, b));
        mine += t ? t + kSegCost : 0;
    }
    int before = mine;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
        const int v = __shfl_up_sync(0xffffffffu, before, d);
        if (lane >= d) before += v;
    }
    if (lane == 31) sm.sums[warp] = before;
    tc_before_sync();
    __syncthreads();
    tc_after_sync();
    const uint32_t tmem = sm.tmem;
    int total = 0;
    before -= mine;
#pragma unroll
    for (int w = 0; w < kThreads / 32; ++w) {
        if (w < warp) before += sm.sums[w];
        total += sm.sums[w];
    }
    const int lo = (int)((int64_t)total * run / p.runs), hi = (int)((int64_t)total * (run + 1) / p.runs);
    if (lo < hi && before <= lo && lo < before + mine) {
        int b = c0, s = before;
        for (;; ++b) {
            const int t = tiles_of(len_of(a, b)), c = t ? t + kSegCost : 0;
            if (lo < s + c) break;
            s += c;
        }
        sm.b0 = b;
        sm.s0 = s;
    }
    __syncthreads();

    Walk w;
    bool more = w.start(a, sm, lo, hi);
    const int h0 = group * p.per_group, nh = min(p.per_group, p.heads - h0);  // this group's heads

    if (warp >= 5) {
        // -------------------------------------------------------- producers
        const int pw = warp - 5, sub = lane & 7;
        const int row = 8 * pw + (lane >> 3);                  // and row + 4
        const uint8_t *cache = static_cast<const uint8_t *>(a.cache);
        const int pieces = p.dim / (E4 ? 16 : 8);              // of 16 bytes
        const uint8_t *src[2];
        const auto find = [&](int i) -> const uint8_t * {      // row i of the tile at w, or none
            const int t = w.t * kTile + row + 4 * i;
            if (t >= w.len) return nullptr;
            const uint32_t col = p.by_page.div((uint32_t)t);
            const uint32_t id = (uint32_t)ld_in(a.block_table + w.b * a.table_stride + col);
            if (id >= p.n_pages) return nullptr;
            return cache + (int64_t)id * p.c_page + (int64_t)(t - col * a.page_size) * p.c_tok;
        };
        constexpr int kLoads = E4 ? 5 : 9;
        if (more) {
            src[0] = find(0);
            src[1] = find(1);
        }
        bool first = true;
        Ring r;
        uint32_t q_phase = 0;
        while (more) {
            if (first) {
                // the queries of another request, once the products with the last ones are done
                if (__any_sync(0xffffffffu, !mb_wait(&sm.q_empty, q_phase ^ 1, abort, &g_err))) break;
                q_phase ^= 1;
                const T *q = static_cast<const T *>(a.q) + w.b * a.q_stride_b;
                const int qp = p.dim / 8;
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    const int h = row + 4 * i;
                    const bool has = h < nh;
                    const T *qr = q + (has ? (int64_t)(h0 + h) * a.q_stride_h : 0);
#pragma unroll
                    for (int j = 0; j < kChunks; ++j)
                        if (8 * j + sub < qp)
                            cp16(sbase + kOffQ + (uint32_t)j * kChunk + sw_off(h, sub), qr + 8 * (8 * j + sub), has);
                }
                cp_arrive(&sm.q_full);
            }
            uint4 code[2][E4 ? kLoads : 1];
            if constexpr (E4) {
#pragma unroll
                for (int i = 0; i < 2; ++i)
#pragma unroll
                    for (int j = 0; j < kLoads; ++j) {
                        code[i][j] = make_uint4(0, 0, 0, 0);
                        if (src[i] && 8 * j + sub < pieces) code[i][j] = ld_once16(src[i] + 16 * (8 * j + sub));
                    }
            }
            const uint8_t *now[2] = {src[0], src[1]};
            more = w.next(a, first);
            if (more) {  // table entries of the next tile, under this one's copies
                src[0] = find(0);
                src[1] = find(1);
            }
            if (__any_sync(0xffffffffu, !mb_wait(&sm.empty[r.slot], r.phase ^ 1, abort, &g_err))) break;
            const uint32_t at = sbase + kOffK + (uint32_t)r.slot * kStageB;
            if constexpr (E4) {
                uint8_t *tile = dyn + kOffK + (uint32_t)r.slot * kStageB;
#pragma unroll
                for (int i = 0; i < 2; ++i)
#pragma unroll
                    for (int j = 0; j < kLoads; ++j) {
                        const int c = 8 * j + sub;
                        if (c >= pieces) continue;
                        uint8_t *d = tile + (uint32_t)(c >> 2) * kChunk;
                        *reinterpret_cast<uint4 *>(d + sw_off(row + 4 * i, 2 * (c & 3))) = widen8<BF>(code[i][j].x, code[i][j].y);
                        *reinterpret_cast<uint4 *>(d + sw_off(row + 4 * i, 2 * (c & 3) + 1)) = widen8<BF>(code[i][j].z, code[i][j].w);
                    }
                fence_async_smem();
                __syncwarp();
                if (lane == 0) mb_arrive(&sm.full[r.slot]);
            } else {
#pragma unroll
                for (int i = 0; i < 2; ++i)
#pragma unroll
                    for (int j = 0; j < kLoads; ++j)
                        if (8 * j + sub < pieces)
                            cp16(at + (uint32_t)j * kChunk + sw_off(row + 4 * i, sub), now[i] ? now[i] + 16 * (8 * j + sub) : cache,
                                 now[i] != nullptr);
                cp_arrive(&sm.full[r.slot]);
            }
            // which of the warp's 8 tokens are seen
            const uint32_t b0 = __ballot_sync(0xffffffffu, sub == 0 && now[0]), b1 = __ballot_sync(0xffffffffu, sub == 0 && now[1]);
            if (lane == 0) {
                uint32_t m = 0;
#pragma unroll
                for (int k = 0; k < 4; ++k) m |= (b0 >> (8 * k) & 1) << k | (b1 >> (8 * k) & 1) << (4 + k);
                reinterpret_cast<volatile uint8_t *>(sm.valid[r.slot])[pw] = (uint8_t)m;
                mb_arrive(&sm.valid_full[r.slot]);
            }
            r.next(kStages);
        }
        asm volatile("cp.async.wait_all;" ::: "memory");
    } else if (warp == 4) {
        // -------------------------------------------------------------- MMA
        const uint32_t fmt = BF ? 1 : 0;
        const uint32_t id_s = idesc(fmt, 0, 0, 64, kTile), id_o = idesc(fmt, 1, 0, 128, p.n);
        const uint64_t dq = desc(sbase + kOffQ, 16, 1024), dk = desc(sbase + kOffK, 16, 1024);
        const uint64_t dv = desc(sbase + kOffK, kChunk, 1024), dp = desc(sbase + kOffP, 16, 1024);
        const int full_chunks = p.dim / 64, rest = p.dim % 64 / 16, mts = (p.latent + 127) / 128;
        const bool lead = elect();
        Ring r;                           // stage of the tile whose S comes next
        Ring ro;                          // stage of the tile whose O comes next
        uint32_t qf = 0, pr = 0, oe = 0, i = 0;
        bool first = true, ok = more;
        bool pend = false, pend_first = false;
        const auto second = [&]() -> bool {  // O += V^T P^T of the pending tile
            if (!mb_wait(&sm.p_ready, pr, abort, &g_err)) return false;
            pr ^= 1;
            if (pend_first) {
                if (!mb_wait(&sm.o_empty, oe ^ 1, abort, &g_err)) return false;
                oe ^= 1;
            }
            tc_after_sync();
            if (lead) {
                const uint64_t v = dv + (uint64_t)(ro.slot * (kStageB >> 4));
                for (int m = 0; m < mts; ++m)
#pragma unroll
                    for (int k = 0; k < 4; ++k)
                        mma_f16(tmem + 64 * m, v + (uint64_t)(m * (2 * kChunk >> 4) + k * (2048 >> 4)), dp + 2 * k, id_o,
                                !(pend_first && k == 0));
                mma_commit(&sm.empty[ro.slot]);
                mma_commit(&sm.pv_done);
            }
            __syncwarp();
            ro.next(kStages);
            pend = false;
            return true;
        };
        while (ok && more) {
            if (first) {
                if (pend) {
                    if (!(ok = second())) break;
                    if (lead) mma_commit(&sm.o_full);
                    __syncwarp();
                }
                if (!(ok = mb_wait(&sm.q_full, qf, abort, &g_err))) break;
                qf ^= 1;
            }
            if (!(ok = mb_wait(&sm.full[r.slot], r.phase, abort, &g_err))) break;
            fence_async_smem();  // the copies landed by the generic proxy
            tc_after_sync();
            const bool last = w.t + 1 == w.te;
            if (lead) {
                const uint64_t k = dk + (uint64_t)(r.slot * (kStageB >> 4));
                const uint32_t d = tmem + kColS + (i & 1) * kTile;
                for (int c = 0; c < full_chunks; ++c)
#pragma unroll
                    for (int j = 0; j < 4; ++j)
                        mma_f16(d, dq + (uint64_t)(c * (kChunk >> 4) + 2 * j), k + (uint64_t)(c * (kChunk >> 4) + 2 * j), id_s,
                                c + j != 0);
                for (int j = 0; j < rest; ++j)
                    mma_f16(d, dq + (uint64_t)(full_chunks * (kChunk >> 4) + 2 * j),
                            k + (uint64_t)(full_chunks * (kChunk >> 4) + 2 * j), id_s, 1);
                mma_commit(&sm.s_full[i & 1]);
                if (last) mma_commit(&sm.q_empty);
            }
            __syncwarp();
            r.next(kStages);
            ++i;
            if (pend && !(ok = second())) break;
            pend = true;
            pend_first = first;
            more = w.next(a, first);
        }
        if (ok && pend) {
            ok = second();
            if (ok && lead) mma_commit(&sm.o_full);
            __syncwarp();
        }
        if (*abort && lead) {  // what was issued ends before the tensor memory is freed
            mma_commit(&sm.drain);
            const unsigned long long t = global_ns();
            while (!mb_try(&sm.drain, 0) && global_ns() - t < kWaitNs) {}
        }
        __syncwarp();
    } else {
        // ---------------------------------------------------------- softmax
        constexpr float kOff = BF ? 0.f : 7.f;
        const uint32_t quad = (uint32_t)(warp * 32) << 16;
        const int hr = 16 * warp + (lane >> 2);            // and hr + 8: this thread's heads
        const bool has[2] = {hr < nh, hr + 8 < nh};
        T *out = static_cast<T *>(a.out);

        // requests without a token
        for (int b = run; b < a.n_requests; b += p.runs) {
            if (len_of(a, b) > 0) continue;
            for (int h = 0; h < nh; ++h) {
                for (int d = tid; d < p.latent; d += 128)
                    from_f32(0.f, out[b * a.out_stride_b + (h0 + h) * a.out_stride_h + d]);
                if (a.lse && tid == 0) a.lse[(int64_t)b * p.heads + h0 + h] = -INFINITY;
            }
        }
        if (tid == 0) p.rec[blockIdx.x].x = -1;

        Ring r;
        uint32_t i = 0, pv = 0, of = 0;
        bool first = true, ok = true;
        float m[2], l[2];
        while (more && ok) {
            if (first) {
                m[0] = m[1] = kFloor;
                l[0] = l[1] = 0.f;
            }
            ok = mb_wait(&sm.valid_full[r.slot], r.phase, abort, &g_err) &&
                 mb_wait(&sm.s_full[i & 1], (i >> 1) & 1, abort, &g_err);
            if (soft_or(!ok)) { ok = false; break; }
            tc_after_sync();
            uint32_t v[32];
            tmem_ld_rows(tmem + quad + kColS + (i & 1) * kTile, v);
            const uint32_t seen[2] = {*(volatile uint32_t *)&sm.valid[r.slot][0], *(volatile uint32_t *)&sm.valid[r.slot][1]};
            tmem_wait_ld();
            float top[2] = {kFloor, kFloor};
            const bool whole = (seen[0] & seen[1]) == 0xffffffffu;
#pragma unroll
            for (int j = 0; j < 32; ++j) {
                float t = __uint_as_float(v[j]) * p.factor;
                const int col = 8 * (j >> 2) + (j & 1);    // and 2 (lane % 4)
                if (!whole && !(seen[col >> 5] >> ((col & 31) + 2 * (lane & 3)) & 1)) t = -INFINITY;
                v[j] = __float_as_uint(t);
                top[j >> 1 & 1] = fmaxf(top[j >> 1 & 1], t);
            }
#pragma unroll
            for (int k = 0; k < 2; ++k) {
                top[k] = fmaxf(top[k], __shfl_xor_sync(0xffffffffu, top[k], 1));
                top[k] = fmaxf(top[k], __shfl_xor_sync(0xffffffffu, top[k], 2));
            }
            bool waited = i == 0;
            if (first) {
                m[0] = top[0];
                m[1] = top[1];
            } else if (soft_or((has[0] && top[0] > m[0] + kLazy) || (has[1] && top[1] > m[1] + kLazy))) {
                // O of the tiles before is complete, then scaled by its columns
#pragma unroll
                for (int k = 0; k < 2; ++k) {
                    const float to = fmaxf(m[k], top[k]), f = ex2(m[k] - to);
                    m[k] = to;
                    l[k] *= f;
                    if ((lane & 3) == 0) sm.factor[hr + 8 * k] = f;
                }
                ok = mb_wait(&sm.pv_done, pv, abort, &g_err);
                waited = true;
                if (soft_or(!ok)) { ok = false; break; }
                tc_after_sync();
                for (int c = 0; c < (p.latent + 127) / 128 * 64; c += 16) {
                    if ((c & 63) >= p.n) continue;
                    uint32_t o[16];
                    tmem_ld(tmem + quad + c, o);
                    tmem_wait_ld();
#pragma unroll
                    for (int j = 0; j < 16; ++j) o[j] = __float_as_uint(__uint_as_float(o[j]) * sm.factor[(c & 63) + j]);
                    tmem_st(tmem + quad + c, o);
                }
                tmem_wait_st();
            }
            uint32_t w2[16];
#pragma unroll
            for (int j = 0; j < 16; ++j) {
                const int k = j & 1;
                const float x = ex2(__uint_as_float(v[2 * j]) - m[k] + kOff), y = ex2(__uint_as_float(v[2 * j + 1]) - m[k] + kOff);
                l[k] += x + y;
                w2[j] = pack_pair(x, y, T());
            }
            if (!waited) ok = mb_wait(&sm.pv_done, pv, abort, &g_err);  // the weights' place is free
            if (i) pv ^= 1;
            uint8_t *pt = dyn + kOffP;
#pragma unroll
            for (int j = 0; j < 16; ++j)
                *reinterpret_cast<uint32_t *>(pt + sw_off(hr + 8 * (j & 1), j >> 1) + 4 * (lane & 3)) = w2[j];
            fence_async_smem();
            tc_before_sync();
            __syncwarp();
            if (lane == 0) mb_arrive(&sm.p_ready);
            r.next(kStages);
            ++i;

            const int b = w.b, s = w.s, tiles = w.tiles;
            if (w.t + 1 == w.te) {  // the last tile of this request in the run
                const bool from0 = max(0, lo - s - kSegCost) == 0, ends = w.te == tiles;
#pragma unroll
                for (int k = 0; k < 2; ++k) {
                    l[k] += __shfl_xor_sync(0xffffffffu, l[k], 1);
                    l[k] += __shfl_xor_sync(0xffffffffu, l[k], 2);
                }
                ok = mb_wait(&sm.o_full, of, abort, &g_err) && ok;
                of ^= 1;
                if (from0 && ends) {
                    if ((lane & 3) == 0)
#pragma unroll
                        for (int k = 0; k < 2; ++k) {
                            sm.factor[hr + 8 * k] = l[k] > 0.f ? a.k_scale / l[k] : 0.f;
                            if (has[k] && a.lse)
                                a.lse[(int64_t)b * p.heads + h0 + hr + 8 * k] =
                                    l[k] > 0.f ? (m[k] - kOff) / kLog2e + logf(l[k]) : -INFINITY;
                        }
                    if (soft_or(!ok)) { ok = false; break; }
                    tc_after_sync();
                    for (int c = 0; c < (p.latent + 127) / 128 * 64; c += 16) {
                        if ((c & 63) >= p.n) continue;
                        uint32_t o[16];
                        tmem_ld(tmem + quad + c, o);
                        tmem_wait_ld();
                        const int d = (c >> 6) * 128 + 32 * warp + lane;
                        if (d >= p.latent) continue;
                        T *to = out + b * a.out_stride_b + (h0 + (c & 63)) * a.out_stride_h + d;
#pragma unroll
                        for (int j = 0; j < 16; ++j)
                            if ((c & 63) + j < nh) from_f32(__uint_as_float(o[j]) * sm.factor[(c & 63) + j], to[j * a.out_stride_h]);
                    }
                } else {
                    float *piece = p.part + (2 * (int64_t)blockIdx.x + (from0 ? 1 : 0)) * piece_floats(p.latent);
                    if ((lane & 3) == 0)
#pragma unroll
                        for (int k = 0; k < 2; ++k) {
                            piece[(int64_t)kHeads * p.latent + hr + 8 * k] = m[k];
                            piece[(int64_t)kHeads * p.latent + kHeads + hr + 8 * k] = l[k];
                        }
                    if (from0 && tid == 0) {
                        // the runs that hold tiles of it: this one to the one of its last tile
                        const int64_t end = s + kSegCost + tiles;
                        p.rec[blockIdx.x] = make_int4(b, run, (int)((end * p.runs - 1) / total), total);
                    }
                    if (soft_or(!ok)) { ok = false; break; }
                    tc_after_sync();
                    for (int c = 0; c < (p.latent + 127) / 128 * 64; c += 16) {
                        if ((c & 63) >= p.n) continue;
                        uint32_t o[16];
                        tmem_ld(tmem + quad + c, o);
                        tmem_wait_ld();
                        const int d = (c >> 6) * 128 + 32 * warp + lane;
                        if (d >= p.latent) continue;
#pragma unroll
                        for (int j = 0; j < 16; ++j) piece[(int64_t)((c & 63) + j) * p.latent + d] = __uint_as_float(o[j]);
                    }
                }
                tc_before_sync();
                __syncwarp();
                if (lane == 0) mb_arrive(&sm.o_empty);
            }
            more = w.next(a, first);
        }
    }

    tc_before_sync();
    __syncthreads();
    tc_after_sync();
    if (warp == 4) tmem_free(tmem, 512);
}

// Joins the pieces of the requests that several runs share: a block a (record,
// head), four groups of 128 threads over the runs, then over the groups.
template <typename T>
__global__ void __launch_bounds__(512) latent_join_kernel(const __grid_constant__ Params p) {
    after_previous();
    __shared__ float wt[512];
    __shared__ float4 sums[4][128];
    __shared__ float red[2];
    const MoeLatentArgs &a = p.a;
    const int block = blockIdx.x, h = blockIdx.y, tid = threadIdx.x;
    const int4 rec = p.rec[block];
    if (rec.x < 0) return;
    const int group = block % p.groups, h0 = group * p.per_group;
    if (h >= min(p.per_group, p.heads - h0)) return;
    const int n = rec.z - rec.y + 1;
    const int64_t floats = piece_floats(p.latent);
    const auto piece = [&](int i) { return p.part + (2 * ((int64_t)(rec.y + i) * p.groups + group) + (i == 0)) * floats; };
    const auto holds = [&](int i) {  // a run may be empty
        const int r = rec.y + i;
        return (int)((int64_t)rec.w * r / p.runs) < (int)((int64_t)rec.w * (r + 1) / p.runs);
    };
    const int64_t at = (int64_t)kHeads * p.latent + h;
    if (tid < 32) {
        float m = kFloor, l = 0.f;
        for (int i = tid; i < n; i += 32)
            if (holds(i)) m = fmaxf(m, piece(i)[at]);
#pragma unroll
        for (int d = 16; d; d >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, d));
        for (int i = tid; i < n; i += 32) {
            const float f = holds(i) ? ex2(piece(i)[at] - m) : 0.f;
            wt[i] = f;
            l += f > 0.f ? f * piece(i)[at + kHeads] : 0.f;
        }
#pragma unroll
        for (int d = 16; d; d >>= 1) l += __shfl_xor_sync(0xffffffffu, l, d);
        if (tid == 0) {
            red[0] = l;
            red[1] = m;
        }
    }
    __syncthreads();
    const int part = tid >> 7, d = (tid & 127) * 4;
    float4 s = make_float4(0.f, 0.f, 0.f, 0.f);
    if (d < p.latent) {
#pragma unroll 4
        for (int i = part; i < n; i += 4) {
            const float f = wt[i];
            if (f == 0.f) continue;
            const float4 v = *reinterpret_cast<const float4 *>(piece(i) + (int64_t)h * p.latent + d);
            s.x += f * v.x; s.y += f * v.y; s.z += f * v.z; s.w += f * v.w;
        }
    }
    sums[part][tid & 127] = s;
    __syncthreads();
    if (part || d >= p.latent) return;
    const float l = red[0], f = l > 0.f ? a.k_scale / l : 0.f;
#pragma unroll
    for (int k = 1; k < 4; ++k) {
        const float4 v = sums[k][tid & 127];
        s.x += v.x; s.y += v.y; s.z += v.z; s.w += v.w;
    }
    T *out = static_cast<T *>(a.out) + rec.x * a.out_stride_b + (h0 + h) * a.out_stride_h + d;
    from_f32(s.x * f, out[0]);
    from_f32(s.y * f, out[1]);
    from_f32(s.z * f, out[2]);
    from_f32(s.w * f, out[3]);
    constexpr float kOff = sizeof(T) == 2 && std::is_same<T, __half>::value ? 7.f : 0.f;
    if (tid == 0 && a.lse)
        a.lse[(int64_t)rec.x * p.heads + h0 + h] = l > 0.f ? (red[1] - kOff) / kLog2e + logf(l) : -INFINITY;
}

int groups_of(int heads) { return (heads + kHeads - 1) / kHeads; }
int runs_of(int heads, int sms) { return sms / groups_of(heads) > 0 ? sms / groups_of(heads) : 1; }

template <bool BF, bool E4>
const void *kernel() { return reinterpret_cast<const void *>(latent_decode_kernel<BF, E4>); }

}  // namespace

cudaError_t latent_prepare(const MoeLatentDesc &d, int num_sms, size_t *bytes) {
    for (const void *fn : {kernel<false, false>(), kernel<false, true>(), kernel<true, false>(), kernel<true, true>()}) {
        const cudaError_t e = cudaFuncSetAttribute(fn, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)kSmem);
        if (e != cudaSuccess) return e;
    }
    const int64_t blocks = (int64_t)groups_of(d.n_heads) * runs_of(d.n_heads, num_sms);
    *bytes = (size_t)blocks * (2 * (size_t)piece_floats(d.latent_dim) * 4 + sizeof(int4));
    return cudaSuccess;
}

cudaError_t launch_latent_decode(const LatentHandle &h, const MoeLatentArgs &a, cudaStream_t s) {
    Params p = {};
    const int64_t ce = (int64_t)dtype_bytes(a.cache_type);
    p.a = a;
    p.heads = h.d.n_heads;
    p.latent = h.d.latent_dim;
    p.dim = h.d.latent_dim + h.d.rope_dim;
    p.groups = groups_of(p.heads);
    p.per_group = (p.heads + p.groups - 1) / p.groups;
    p.n = (p.per_group + 15) / 16 * 16;
    p.runs = runs_of(p.heads, h.num_sms);
    p.factor = a.scale * a.k_scale * kLog2e;
    p.by_page = FastDiv((uint32_t)a.page_size);
    p.c_page = a.c_stride_page * ce;
    p.c_tok = a.c_stride_tok * ce;
    p.n_pages = (uint32_t)a.n_pages;
    p.part = h.part;
    const int blocks = p.groups * p.runs;
    p.rec = reinterpret_cast<int4 *>(h.part + 2 * blocks * piece_floats(p.latent));
    const bool bf = a.act_type == MOE_BF16, e4 = a.cache_type == MOE_E4M3;
    const void *fn = bf ? (e4 ? kernel<true, true>() : kernel<true, false>()) : (e4 ? kernel<false, true>() : kernel<false, false>());
    void *args[] = {&p};
    cudaError_t e = launch_after(fn, blocks, kThreads, kSmem, s, args);
    if (e != cudaSuccess) return e;
    cudaLaunchAttribute at[1];
    at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[0].val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t c = {};
    c.gridDim = dim3((unsigned)blocks, (unsigned)p.per_group);
    c.blockDim = dim3(512);
    c.stream = s;
    c.attrs = at;
    c.numAttrs = 1;
    return cudaLaunchKernelExC(&c, reinterpret_cast<const void *>(bf ? latent_join_kernel<__nv_bfloat16> : latent_join_kernel<__half>),
                               args);
}

cudaError_t latent_decode_flags(int32_t *out) {
    const int32_t zero = 0;
    cudaError_t e = cudaMemcpyFromSymbol(out, g_err, 4);
    if (e == cudaSuccess && *out) e = cudaMemcpyToSymbol(g_err, &zero, 4);
    return e;
}

}  // namespace moe
