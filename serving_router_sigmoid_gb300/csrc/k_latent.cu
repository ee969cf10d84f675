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
// 3300 cycles a SM (16-bit) or 1650 (E4M3) where each SM reads rows of its own, in half of
// that where two groups of heads read them together.  Measured: a tile in 4100 (16-bit), since
// two stages beside 72 KB of queries leave the chain load, S, softmax, O little to
// overlap; 32-token tiles in four stages were slower (fixed costs an MMA and a
// barrier).  64 requests of up to 16384 tokens, 128 heads: 121 us (2.3 TB/s of rows
// read once from HBM and twice from L2); 2 of 131072 in E4M3, 64 heads: 83 us.
// Prefetches to L2 two or three tiles ahead changed nothing (TMA) or cost 3 to 20%
// (16-bit rows by prefetch instructions).
//
// - Work is split by cost: the tiles of all requests, and kSegCost more for each
//   request, form one line; each block takes an equal run, found from the lengths
//   by itself.  More than 64 heads form groups; the blocks of a run's groups are
//   neighbours and read the same rows at the same time, once from HBM.
// - Eight producer warps copy rows (cp.async, any page size and stride), issue TMA
//   copies of them (a warp a part: 127 against 128 us), or load E4M3 codes and widen
//   them, into two stages of three parts; S starts on a part when it is there, and a
//   part is given back by itself.  One warp issues the products S, another
//   the products O (one that issued both in turn let each wait for the other's
//   barriers: 139 against 136 us); four warps do the softmax and write the results.
// - The maximum moves only when a logit passes it by 2^kLazy; then O is scaled in
//   tensor memory.  Weights are rounded to the operand type (their sum is not), for
//   f16 times 2^7, so that its subnormals begin at 2^-31 of the maximum.  With bf16 the
//   result is off by 0.0021 in the norm where its own rounding alone makes 0.0017; for a
//   second term of the weights there is no room beside queries and stages.
// - A request that several blocks share leaves its pieces (O, m, l) in the handle's
//   workspace; a second small launch joins them in order, so results do not depend
//   on timing.  Pieces lie as [8 heads][latent][8], so that 32 lanes write and read
//   1 KB in a row (256-byte steps took 20 us more for 2 requests of 30000 tokens).
#include <type_traits>

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
constexpr int kParts = 3;             // of a stage: four chunks, which come and are given back together
constexpr int kProd = 8;              // producer warps
constexpr int kThreads = 32 * (4 + 2 + kProd);  // softmax, two that issue MMAs, producers
constexpr uint32_t kOffQ = 0, kOffK = kStageB, kOffP = kOffK + kStages * kStageB;
constexpr size_t kSmem = kOffP + kHeads * 128 + 1024;
constexpr uint32_t kColS = 256;       // tensor memory: O 4 x 64 columns, then S twice
// What a request costs besides its tiles, in tiles.  Measured with 1 2 3 4: 64 requests of up to
// 16384 tokens, 128 heads 135.5 123.8 120.4 121.5 us, 300 of 300 63.4 55.3 56.4 53.4, 200 of 3000
// 128.0 127.5 125.3 125.1, 2000 of 100 177 174 171 171
constexpr int kSegCost = 3;
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
    int box;                          // rows of a TMA box: the largest power of two to 64 that divides a page; used from 32 on
    int out32;                        // rows of out start on 32 bytes
    int64_t c_page, c_tok;            // bytes
    uint32_t n_pages;
    float *part;                      // [2 * blocks] pieces
    int2 *rec;                        // [requests * groups]: first and last run of a request that several hold, else x < 0
};

__host__ __device__ inline int64_t piece_floats(int latent) { return (int64_t)kHeads * latent + 2 * kHeads; }

struct Shared {
    uint64_t full[kStages][kParts], empty[kStages][kParts], valid_full[kStages], q_full, q_empty, s_full[2], s_empty[2], p_ready, pv_done, o_full, o_empty, drain[2];
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
__device__ __forceinline__ void soft_bar() { asm volatile("bar.sync 1, 128;" ::: "memory"); }
__device__ __forceinline__ void prod_bar() { asm volatile("bar.sync 2, 256;" ::: "memory"); }
__device__ __forceinline__ bool soft_or(bool p) {
    uint32_t r;
    asm volatile("{\n .reg .pred pi, po;\n setp.ne.u32 pi, %1, 0;\n bar.red.or.pred po, 1, 128, pi;\n selp.u32 %0, 1, 0, po;\n}"
                 : "=r"(r) : "r"((uint32_t)p) : "memory");
    return r != 0;
}

// How rows come: by TMA (pages of whole runs of 32 tokens; a request's last, ragged
// tile row by row), row by row (any page size and stride), or as E4M3 codes.
constexpr int kByRow = 0, kByTma = 1, kByCode = 2;

template <bool BF, int LOAD>
__global__ void __launch_bounds__(kThreads, 1) latent_decode_kernel(const __grid_constant__ CUtensorMap cmap, const __grid_constant__ Params p) {
    constexpr bool E4 = LOAD == kByCode;
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
            for (int j = 0; j < kParts; ++j) {
                mb_init(&sm.full[i][j], LOAD == kByRow ? 32 * kProd : LOAD == kByCode ? kProd : 1);
                mb_init(&sm.empty[i][j], 1);
            }
            mb_init(&sm.valid_full[i], LOAD == kByTma ? 1 : kProd);
            mb_init(&sm.s_full[i], 1);
            mb_init(&sm.s_empty[i], 4);
        }
        mb_init(&sm.q_full, 32 * kProd);
        mb_init(&sm.q_empty, 1);
        mb_init(&sm.p_ready, 4);
        mb_init(&sm.pv_done, 1);
        mb_init(&sm.o_full, 1);
        mb_init(&sm.o_empty, 4);
        mb_init(&sm.drain[0], 1);
        mb_init(&sm.drain[1], 1);
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
    const int runs = min(max(total, 1), p.runs);  // none is empty
    const int lo = run < runs ? (int)((int64_t)total * run / runs) : total;
    const int hi = run < runs ? (int)((int64_t)total * (run + 1) / runs) : total;
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

    if (warp >= 6) {
        // -------------------------------------------------------- producers
        const int pw = warp - 6, sub = lane & 7;
        const int row = 8 * pw + (lane >> 3);                  // and row + 4
        const uint8_t *cache = static_cast<const uint8_t *>(a.cache);
        const int pieces = p.dim / (E4 ? 16 : 8);              // of 16 bytes
        struct Next {                                          // a tile to bring
            const uint8_t *row[2];                             // this thread's rows, or none
            int b, page, off;                                  // by TMA: page and row of the group `lane`
            bool first, have, whole;
        };
        const int gshift = LOAD == kByTma ? 31 - __clz(p.box) : 3;  // log2 of the rows of a group
        bool opens = true;
        const auto fetch = [&]() {
            Next x;
            x.have = more;
            if (!more) return x;
            x.whole = LOAD == kByTma && (w.t + 1) * kTile <= w.len;
            if (x.whole) {
                const int t = w.t * kTile + (lane << gshift);
                x.page = -1;
                if (lane << gshift < kTile) {
                    const uint32_t col = p.by_page.div((uint32_t)t);
                    x.page = ld_in(a.block_table + w.b * a.table_stride + col);
                    x.off = t - (int)(col * a.page_size);
                }
            } else {
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    const int t = w.t * kTile + row + 4 * i;
                    const uint32_t col = p.by_page.div((uint32_t)t);
                    const uint32_t id = t < w.len ? (uint32_t)ld_in(a.block_table + w.b * a.table_stride + col) : ~0u;
                    x.row[i] = id < p.n_pages ? cache + (int64_t)id * p.c_page + (int64_t)(t - col * a.page_size) * p.c_tok : nullptr;
                }
            }
            x.b = w.b;
            x.first = opens;
            more = w.next(a, opens);
            return x;
        };
        const int parts = (p.dim + 255) / 256, chunks = (p.dim + 63) / 64;
        Next now = fetch(), nxt = fetch();
        Ring r;
        uint32_t q_phase = 0;
        constexpr int kCodes = E4 ? (kChunks + 1) / 2 : 1;
        uint4 code[2][kCodes];
        const auto load = [&](const Next &x, int j) {          // codes of two chunks, 8 pieces of 16 bytes a row
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                code[i][j] = make_uint4(0, 0, 0, 0);
                if (x.have && x.row[i] && 8 * j + sub < pieces) code[i][j] = ld_once16(x.row[i] + 16 * (8 * j + sub));
            }
        };
        if constexpr (E4)
#pragma unroll
            for (int j = 0; j < kCodes; ++j) load(now, j);
        const auto queries = [&](int b) {                      // of another request
            const T *q = static_cast<const T *>(a.q) + b * a.q_stride_b;
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
        };
        const auto copy_part = [&](uint32_t at, int j) {       // this thread's pieces of a part
#pragma unroll
            for (int c = 4 * j; c < 4 * j + 4; ++c)
#pragma unroll
                for (int i = 0; i < 2; ++i)
                    if (8 * c + sub < pieces)
                        cp16(sbase + at + (uint32_t)c * kChunk + sw_off(row + 4 * i, sub),
                             now.row[i] ? now.row[i] + 16 * (8 * c + sub) : cache, now.row[i] != nullptr);
        };
        const auto seen = [&]() {                              // which of the warp's 8 tokens are
            const uint32_t b0 = __ballot_sync(0xffffffffu, sub == 0 && now.row[0]), b1 = __ballot_sync(0xffffffffu, sub == 0 && now.row[1]);
            uint32_t m = 0;
#pragma unroll
            for (int k = 0; k < 4; ++k) m |= (b0 >> (8 * k) & 1) << k | (b1 >> (8 * k) & 1) << (4 + k);
            if (lane == 0) reinterpret_cast<volatile uint8_t *>(sm.valid[r.slot])[pw] = (uint8_t)m;
        };
        bool ok = true;
        if constexpr (LOAD == kByTma) {
            // a warp a part waits and issues; all copy where it goes row by row.  Nobody leaves early: all warps
            // meet at every barrier, whatever was given up
            int issued[kStages] = {-1, -1};
            for (; now.have; now = nxt, nxt = fetch()) {
                if (now.first) {
                    if (pw == 0) ok = mb_wait(&sm.q_empty, q_phase ^ 1, abort, &g_err) && ok;
                    q_phase ^= 1;
                    prod_bar();
                    queries(now.b);
                }
                const uint32_t at = kOffK + (uint32_t)r.slot * kStageB;
                if (now.whole) {
                    const int groups = kTile >> gshift;
                    uint32_t lives = 0;
                    for (int g = 0; g < groups; ++g)
                        if ((uint32_t)__shfl_sync(0xffffffffu, now.page, g) < p.n_pages) lives |= 1u << g;
                    if (pw < parts) {
                        // a part a warp; lane: a group of rows of a chunk, 32 of them at most; a page that is none reads as zeros
                        const int n = min(4, chunks - 4 * pw), g = lane & (groups - 1), c = 4 * pw + lane / groups;
                        const int id = __shfl_sync(0xffffffffu, now.page, g), off = __shfl_sync(0xffffffffu, now.off, g);
                        ok = __all_sync(0xffffffffu, ok && mb_wait(&sm.empty[r.slot][pw], r.phase ^ 1, abort, &g_err));
                        if (ok) {
                            if (lane == 0) mb_expect_tx(&sm.full[r.slot][pw], (uint32_t)n * kChunk);
                            __syncwarp();
                            if (lane < n * groups)
                                tma_3d(sbase + at + (uint32_t)c * kChunk + (uint32_t)(g << gshift) * 128u, &cmap, 64 * c,
                                       lives >> g & 1 ? off : 0, lives >> g & 1 ? id : (int)p.n_pages, &sm.full[r.slot][pw]);
                            issued[r.slot] = (int)r.phase;
                        }
                        __syncwarp();
                    }
                    if (pw == 0) {  // part 0 was free: the softmax has read what was there
                        if (lane < 8) reinterpret_cast<volatile uint8_t *>(sm.valid[r.slot])[lane] = lives >> (8 * lane >> gshift) & 1 ? 0xff : 0;
                        __syncwarp();
                        if (lane == 0) mb_arrive(&sm.valid_full[r.slot]);
                    }
                } else {
                    // the last tile of a request, row by row
                    if (pw == 0)
                        for (int j = 0; j < parts; ++j) ok = mb_wait(&sm.empty[r.slot][j], r.phase ^ 1, abort, &g_err) && ok;
                    prod_bar();
#pragma unroll
                    for (int j = 0; j < kParts; ++j) copy_part(at, j);
                    seen();
                    asm volatile("cp.async.wait_all;" ::: "memory");
                    fence_async_smem();
                    prod_bar();
                    if (pw == 0 && lane < parts) mb_arrive(&sm.full[r.slot][lane]);
                    if (pw == 0 && lane == 0) mb_arrive(&sm.valid_full[r.slot]);
                }
                r.next(kStages);
            }
            if (pw < parts && *abort) {  // copies in flight land before the block ends
                const long long t = clock64();
                for (int i = 0; i < kStages; ++i)
                    while (issued[i] >= 0 && !mb_test(&sm.full[i][pw], (uint32_t)issued[i]) && clock64() - t < kWaitClk) {}
            }
        } else {
            for (; now.have && ok; now = nxt, nxt = fetch()) {
                if (now.first) {  // once the products with the last queries are done
                    ok = __all_sync(0xffffffffu, mb_wait(&sm.q_empty, q_phase ^ 1, abort, &g_err));
                    q_phase ^= 1;
                    if (ok) queries(now.b);
                }
                const uint32_t at = kOffK + (uint32_t)r.slot * kStageB;
#pragma unroll
                for (int k = 0; k < kParts; ++k) {
                    const int j = (k + kParts - 1) % kParts;
                    if (j >= parts) continue;
                    ok = __all_sync(0xffffffffu, ok && mb_wait(&sm.empty[r.slot][j], r.phase ^ 1, abort, &g_err));
                    if constexpr (E4) {
                        // lanes of both chunks store to different banks: the upper ones their second 8 codes first
                        const bool f = sub >> 2;
#pragma unroll
                        for (int h = 2 * j; h < 2 * j + 2 && h < kCodes; ++h) {
                            uint8_t *tile = dyn + at + (uint32_t)(2 * h + (sub >> 2)) * kChunk;
                            if (8 * h + sub < pieces)
#pragma unroll
                                for (int i = 0; i < 2; ++i) {
                                    const uint4 w = code[i][h];
                                    const int c = 2 * (sub & 3);
                                    *reinterpret_cast<uint4 *>(tile + sw_off(row + 4 * i, c + f)) = widen8<BF>(f ? w.z : w.x, f ? w.w : w.y);
                                    *reinterpret_cast<uint4 *>(tile + sw_off(row + 4 * i, c + !f)) = widen8<BF>(f ? w.x : w.z, f ? w.y : w.w);
                                }
                        }
                    } else {
                        copy_part(at, j);
                        cp_arrive(&sm.full[r.slot][j]);
                    }
                }
                if constexpr (E4) {
                    // one fence a tile: it waits for the loads in flight too, so the next codes are asked for behind it
                    fence_async_smem();
                    __syncwarp();
                    if (lane < parts) mb_arrive(&sm.full[r.slot][lane]);
#pragma unroll
                    for (int j = 0; j < kCodes; ++j) load(nxt, j);
                }
                seen();  // read by the softmax before the second product, which frees the stage
                if (lane == 0) mb_arrive(&sm.valid_full[r.slot]);
                r.next(kStages);
            }
        }
        asm volatile("cp.async.wait_all;" ::: "memory");
    } else if (warp >= 4) {
        // -------------------------------------------------------------- MMA
        // One warp issues S, the other O, each as soon as what it needs is there.
        const uint32_t fmt = BF ? 1 : 0;
        const uint32_t id_s = idesc(fmt, 0, 0, 64, kTile), id_o = idesc(fmt, 1, 0, 128, p.n);
        const uint32_t dq = desc(sbase + kOffQ, 16), dk = desc(sbase + kOffK, 16);
        const uint32_t dv = desc(sbase + kOffK, kChunk), dp = desc(sbase + kOffP, 16);
        const int steps = p.dim / 16, parts = (steps + 15) / 16, mts = (p.latent + 127) / 128, own = (mts + 1) / 2;  // own: parts that O reads
        const auto part_of = [&](int k) { return parts < kParts ? k : (k + kParts - 1) % kParts; };  // what only S reads comes first
        const bool lead = elect();
        const auto wait = [&](uint64_t *bar, uint32_t phase) { return __all_sync(0xffffffffu, mb_wait(bar, phase, abort, &g_err)); };
        Ring r;
        uint32_t i = 0, flip = 0;
        bool first = true, ok = true;
        if (warp == 4) {
            // ---- S = Q K^T
            uint32_t qf = 0;
            while (ok && more) {
                if (first) {
                    if (!(ok = wait(&sm.q_full, qf))) break;
                    qf ^= 1;
                    fence_async_smem();  // copied by the generic proxy
                }
                const bool last = w.t + 1 == w.te;
                // the buffer of the tile before the last: its logits are read
                if (i >= 2) ok = wait(&sm.s_empty[i & 1], (i >> 1 & 1) ^ 1);
                const uint32_t slot = dk + (uint32_t)(r.slot * (int)(kStageB >> 4)), d = tmem + kColS + (i & 1) * kTile;
                for (int k = 0; k < parts && ok; ++k) {  // as they come
                    const int j = part_of(k);
                    if (!(ok = wait(&sm.full[r.slot][j], r.phase))) break;
                    if (LOAD == kByRow) fence_async_smem();  // the copies landed by the generic proxy
                    tc_after_sync();
                    if (lead) {
                        const int n = min(16, steps - 16 * j);
                        for (int c = 4 * j; c < 4 * j + n / 4; ++c)
#pragma unroll
                            for (int e = 0; e < 4; ++e)
                                mma_f16(d, dq + (uint32_t)(c * (int)(kChunk >> 4) + 2 * e), slot + (uint32_t)(c * (int)(kChunk >> 4) + 2 * e),
                                        id_s, k + (c - 4 * j) + e != 0);
                        for (int e = 0; e < n % 4; ++e)
                            mma_f16(d, dq + (uint32_t)(steps / 4 * (int)(kChunk >> 4) + 2 * e),
                                    slot + (uint32_t)(steps / 4 * (int)(kChunk >> 4) + 2 * e), id_s, k + n / 4 + e != 0);
                    }
                    __syncwarp();
                }
                if (!ok) break;
                if (lead) {
                    mma_commit(&sm.s_full[i & 1]);
                    for (int e = own; e < parts; ++e) mma_commit(&sm.empty[r.slot][e]);
                    if (last) mma_commit(&sm.q_empty);
                }
                __syncwarp();
                r.next(kStages);
                ++i;
                more = w.next(a, first);
            }
        } else {
            // ---- O += V^T P^T
            uint32_t oe = 0;
            while (ok && more) {
                const bool last = w.t + 1 == w.te;
                if (first) {
                    if (!(ok = wait(&sm.o_empty, oe ^ 1))) break;
                    oe ^= 1;
                }
                if (!(ok = wait(&sm.p_ready, flip))) break;
                flip ^= 1;
                tc_after_sync();
                if (lead) {
                    const uint32_t v = dv + (uint32_t)(r.slot * (int)(kStageB >> 4));
                    for (int m = 0; m < mts; ++m) {
#pragma unroll
                        for (int k = 0; k < 4; ++k)
                            mma_f16(tmem + 64 * m, v + (uint32_t)(m * (int)(2 * kChunk >> 4) + k * (2048 >> 4)), dp + 2 * k, id_o,
                                    !(first && k == 0));
                        if (m & 1 || m + 1 == mts) mma_commit(&sm.empty[r.slot][m >> 1]);
                    }
                    mma_commit(&sm.pv_done);
                    if (last) mma_commit(&sm.o_full);
                }
                __syncwarp();
                r.next(kStages);
                more = w.next(a, first);
            }
        }
        if (*abort) {  // what was issued ends before the tensor memory is freed
            if (lead) mma_commit(&sm.drain[warp - 4]);
            const long long t = clock64();
            while (!mb_try(&sm.drain[warp - 4], 0) && clock64() - t < kWaitClk) {}
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
            if (tid == 0) p.rec[(int64_t)b * p.groups + group].x = -1;
        }

        Ring r;
        uint32_t i = 0, pv = 0, of = 0;
        bool first = true;
        float m[2], l[2];
        // (a wait that was given up changes nothing here: every thread takes every barrier)
        while (more) {
            if (first) {
                m[0] = m[1] = kFloor;
                l[0] = l[1] = 0.f;
            }
            mb_wait(&sm.valid_full[r.slot], r.phase, abort, &g_err);
            mb_wait(&sm.s_full[i & 1], (i >> 1) & 1, abort, &g_err);
            tc_after_sync();
            uint32_t v[32];
            tmem_ld_rows(tmem + quad + kColS + (i & 1) * kTile, v);
            const uint32_t seen[2] = {*(volatile uint32_t *)&sm.valid[r.slot][0], *(volatile uint32_t *)&sm.valid[r.slot][1]};
            tmem_wait_ld();
            tc_before_sync();
            __syncwarp();
            if (lane == 0) mb_arrive(&sm.s_empty[i & 1]);
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
                mb_wait(&sm.pv_done, pv, abort, &g_err);
                waited = true;
                soft_bar();
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
            if (!waited) mb_wait(&sm.pv_done, pv, abort, &g_err);  // the weights' place is free
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
                mb_wait(&sm.o_full, of, abort, &g_err);
                of ^= 1;
                // the runs that hold tiles of it: this one to the one of its last tile (the first writes)
                if (from0 && tid == 0)
                    p.rec[(int64_t)b * p.groups + group] =
                        make_int2(ends ? -1 : run, (int)(((int64_t)(s + kSegCost + tiles) * runs - 1) / total));
                if (from0 && ends) {
                    if ((lane & 3) == 0)
#pragma unroll
                        for (int k = 0; k < 2; ++k) {
                            sm.factor[hr + 8 * k] = l[k] > 0.f ? a.k_scale / l[k] : 0.f;
                            if (has[k] && a.lse)
                                a.lse[(int64_t)b * p.heads + h0 + hr + 8 * k] =
                                    l[k] > 0.f ? (m[k] - kOff) / kLog2e + logf(l[k]) : -INFINITY;
                        }
                    soft_bar();
                    tc_after_sync();
                    for (int c = 0; c < (p.latent + 127) / 128 * 64; c += 16) {
                        if ((c & 63) >= p.n) continue;
                        uint32_t o[16];
                        tmem_ld(tmem + quad + c, o);
                        tmem_wait_ld();
                        // 16 heads by 32 dimensions, turned in the weights' place: a lane takes half a head's row
                        float *turn = reinterpret_cast<float *>(dyn + kOffP) + 512 * warp;
#pragma unroll
                        for (int j = 0; j < 16; ++j)
                            turn[32 * j + (lane ^ 4 * (j & 7))] = __uint_as_float(o[j]) * sm.factor[(c & 63) + j];
                        __syncwarp();
                        const int h = (c & 63) + (lane >> 1), d = (c >> 6) * 128 + 32 * warp + 16 * (lane & 1);
                        float x[16];
#pragma unroll
                        for (int k = 0; k < 4; ++k)
                            *reinterpret_cast<float4 *>(x + 4 * k) = *reinterpret_cast<const float4 *>(
                                turn + 32 * (lane >> 1) + ((16 * (lane & 1) + 4 * k) ^ 4 * (lane >> 1 & 7)));
                        __syncwarp();
                        if (h >= nh || d >= p.latent) continue;
                        T *to = out + b * a.out_stride_b + (h0 + h) * a.out_stride_h + d;
                        if (p.out32) {
                            uint32_t y[8];
#pragma unroll
                            for (int k = 0; k < 8; ++k) y[k] = pack_pair(x[2 * k], x[2 * k + 1], T());
                            st32(to, y);
                        } else {
#pragma unroll
                            for (int k = 0; k < 16; ++k) from_f32(x[k], to[k]);
                        }
                    }
                } else {
                    float *piece = p.part + (2 * (int64_t)blockIdx.x + (from0 ? 1 : 0)) * piece_floats(p.latent);
                    if ((lane & 3) == 0)
#pragma unroll
                        for (int k = 0; k < 2; ++k) {
                            piece[(int64_t)kHeads * p.latent + hr + 8 * k] = m[k];
                            piece[(int64_t)kHeads * p.latent + kHeads + hr + 8 * k] = l[k];
                        }
                    tc_after_sync();
                    for (int c = 0; c < (p.latent + 127) / 128 * 64; c += 16) {
                        if ((c & 63) >= p.n) continue;
                        uint32_t o[16];
                        tmem_ld(tmem + quad + c, o);
                        tmem_wait_ld();
                        const int d = (c >> 6) * 128 + 32 * warp + lane;
                        if (d >= p.latent) continue;
                        uint32_t *to = reinterpret_cast<uint32_t *>(piece) + (c & 63) * p.latent + 8 * d;  // by 8 heads
#pragma unroll
                        for (int k = 0; k < 2; ++k) {
                            const uint32_t y[8] = {o[8 * k], o[8 * k + 1], o[8 * k + 2], o[8 * k + 3], o[8 * k + 4], o[8 * k + 5], o[8 * k + 6], o[8 * k + 7]};
                            st32(to + 8 * k * p.latent, y);
                        }
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

// Joins the pieces of the requests that several runs share.  A block takes 32
// latent dimensions of a request and head group, or several times 32 in turn, a lane one
// of them for 8 heads (32 contiguous bytes a piece); W of its 8 warps take 8 heads, each
// a part of the runs.
constexpr int kMaxRuns = 152;
constexpr int kBatch = 6;  // pieces that a lane loads at once
template <typename T, int W>
__global__ void __launch_bounds__(256) latent_join_kernel(const __grid_constant__ Params p) {
    after_previous();
    __shared__ __align__(16) float wt[8 / W][kMaxRuns][8];
    __shared__ float sums[8][8][32];
    const MoeLatentArgs &a = p.a;
    const int group = blockIdx.x % p.groups, b = blockIdx.x / p.groups, tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int2 rec = p.rec[blockIdx.x];
    if (rec.x < 0) return;
    const int h0 = group * p.per_group, nh = min(p.per_group, p.heads - h0);
    const int oct = blockIdx.z * (8 / W) + warp / W, part = warp % W, n = rec.y - rec.x + 1;
    const int64_t floats = piece_floats(p.latent);
    const float *pieces = p.part + (2 * ((int64_t)rec.x * p.groups + group)) * floats;  // of run i: 2 i groups further; the first is a second piece
    const auto piece = [&](int i) { return pieces + (2 * (int64_t)i * p.groups + (i == 0)) * floats; };
    float top = kFloor, l = 0.f;
    float (*const w)[8] = wt[warp / W];
    // maxima and sums of the pieces, (run, head) pairs over the W warps' threads
    const int team = 32 * W, me = 32 * part + lane, pairs = 8 * oct < nh ? 8 * n : 0;
    const int64_t at = (int64_t)kHeads * p.latent + 8 * oct + (lane & 7);
    for (int i0 = me; i0 < pairs; i0 += 5 * team) {
        float m[5];
#pragma unroll
        for (int k = 0; k < 5; ++k) {
            const int i = (i0 + k * team) >> 3;
            m[k] = i < n ? piece(i)[at] : -INFINITY;
        }
#pragma unroll
        for (int k = 0; k < 5; ++k) {
            if (i0 + k * team < pairs) w[(i0 + k * team) >> 3][lane & 7] = m[k];
            top = fmaxf(top, m[k]);
        }
    }
    top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 8));
    top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 16));
    if (W > 1) {
        if (lane < 8) sums[0][warp][lane] = top;
        __syncthreads();
#pragma unroll
        for (int q = 0; q < W; ++q) top = fmaxf(top, sums[0][warp - part + q][lane & 7]);
    }
    for (int i0 = me; i0 < pairs; i0 += 5 * team) {
        float v[5];
#pragma unroll
        for (int k = 0; k < 5; ++k) {
            const int i = (i0 + k * team) >> 3;
            v[k] = i < n ? piece(i)[at + kHeads] : 0.f;
        }
#pragma unroll
        for (int k = 0; k < 5; ++k) {
            const int i = (i0 + k * team) >> 3;
            if (i >= n) continue;
            const float f = ex2(w[i][lane & 7] - top);
            w[i][lane & 7] = f;
            l += f * v[k];
        }
    }
    l += __shfl_xor_sync(0xffffffffu, l, 8);
    l += __shfl_xor_sync(0xffffffffu, l, 16);
    if (W > 1) {
        if (lane < 8) sums[1][warp][lane] = l;
        __syncthreads();
        l = 0.f;
#pragma unroll
        for (int q = 0; q < W; ++q) l += sums[1][warp - part + q][lane & 7];
        __syncthreads();
    } else {
        __syncwarp();
    }
    constexpr float kOff = std::is_same<T, __half>::value ? 7.f : 0.f;
    for (int d = 32 * blockIdx.y + lane; d < p.latent; d += 32 * gridDim.y) {
        float s[8] = {};
        for (int i0 = part; i0 < n && 8 * oct < nh; i0 += kBatch * W) {
            float4 v[kBatch][2];
#pragma unroll
            for (int k = 0; k < kBatch; ++k) {  // all in flight at once
                if (i0 + k * W >= n) continue;
                const float4 *at = reinterpret_cast<const float4 *>(piece(i0 + k * W) + 8 * (oct * p.latent + d));
                v[k][0] = at[0];
                v[k][1] = at[1];
            }
#pragma unroll
            for (int k = 0; k < kBatch; ++k) {
                const int i = i0 + k * W;
                if (i >= n) continue;
                const float4 f0 = *reinterpret_cast<const float4 *>(w[i]), f1 = *reinterpret_cast<const float4 *>(w[i] + 4);
                s[0] += f0.x * v[k][0].x; s[1] += f0.y * v[k][0].y; s[2] += f0.z * v[k][0].z; s[3] += f0.w * v[k][0].w;
                s[4] += f1.x * v[k][1].x; s[5] += f1.y * v[k][1].y; s[6] += f1.z * v[k][1].z; s[7] += f1.w * v[k][1].w;
            }
        }
        if (W > 1) {
#pragma unroll
            for (int j = 0; j < 8; ++j) sums[warp][j][lane] = s[j];
            __syncthreads();
            if (part == 0) {
#pragma unroll
                for (int q = 1; q < W; ++q)
#pragma unroll
                    for (int j = 0; j < 8; ++j) s[j] += sums[warp + q][j][lane];
            }
            __syncthreads();
            if (part) continue;
        }
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const float lj = __shfl_sync(0xffffffffu, l, j), mj = __shfl_sync(0xffffffffu, top, j);
            const int h = 8 * oct + j;
            if (h >= nh) continue;
            from_f32(lj > 0.f ? s[j] * (a.k_scale / lj) : 0.f,
                     static_cast<T *>(a.out)[b * a.out_stride_b + (h0 + h) * a.out_stride_h + d]);
            if (a.lse && d == 0) a.lse[(int64_t)b * p.heads + h0 + h] = lj > 0.f ? (mj - kOff) / kLog2e + logf(lj) : -INFINITY;
        }
    }
}

int groups_of(int heads) { return (heads + kHeads - 1) / kHeads; }
int runs_of(int heads, int sms) {
    const int n = sms / groups_of(heads);
    return n < 1 ? 1 : n > kMaxRuns ? kMaxRuns : n;
}

template <int LOAD>
const void *kernel(bool bf) {
    return bf ? reinterpret_cast<const void *>(latent_decode_kernel<true, LOAD>)
              : reinterpret_cast<const void *>(latent_decode_kernel<false, LOAD>);
}

template <typename T>
cudaError_t launch_join(Params &p, cudaStream_t s) {
    const int n = p.a.n_requests;
    // by the pieces a request has at most. Measured, decode and join of requests of up to
    // 3000 tokens, 64 heads, W = 1 2 4 8: 2 requests 20.1 17.0 15.5 14.7 us; 4: 29.0 21.2
    // 17.4 18.7; 8: 23.9 19.7 21.2 23.1; 18: 25.0 27.3 30.0 37.1
    const int W = 50 * n <= p.runs ? 8 : 25 * n <= p.runs ? 4 : 12 * n <= p.runs ? 2 : 1;
    // Blocks a request: by 32 columns; by 64 where those make more than three blocks an SM (30
    // requests of up to 3000 tokens 31.6 and, by 32, 32.6 us, 64 of 6000 with 128 heads 138 and
    // 142; 18 of 3000 29.2 and 24.8); four beyond the runs, where most have nothing to join (300
    // of 300: 55 us, with one block 76, 16 61), one for thousands (8192 of 40: 289, with four 317)
    const int by32 = p.latent / 32;
    const int columns = n > 16 * p.runs ? 1 : n > p.runs ? (by32 < 4 ? by32 : 4) : n * by32 > 3 * p.runs ? by32 / 2 : by32;
    const void *fn = W == 8 ? reinterpret_cast<const void *>(latent_join_kernel<T, 8>)
                     : W == 4 ? reinterpret_cast<const void *>(latent_join_kernel<T, 4>)
                     : W == 2 ? reinterpret_cast<const void *>(latent_join_kernel<T, 2>)
                              : reinterpret_cast<const void *>(latent_join_kernel<T, 1>);
    cudaLaunchAttribute at[1];
    at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[0].val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t c = {};
    c.gridDim = dim3((unsigned)(n * p.groups), (unsigned)columns,
                     (unsigned)((p.per_group + 7) / 8 * W + 7) / 8);
    c.blockDim = dim3(256);
    c.stream = s;
    c.attrs = at;
    c.numAttrs = 1;
    void *args[] = {&p};
    return cudaLaunchKernelExC(&c, fn, args);
}

}  // namespace

cudaError_t latent_prepare(const MoeLatentDesc &d, int num_sms, size_t *bytes) {
    for (const bool bf : {false, true})
        for (const void *fn : {kernel<kByRow>(bf), kernel<kByTma>(bf), kernel<kByCode>(bf)}) {
            const cudaError_t e = cudaFuncSetAttribute(fn, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)kSmem);
            if (e != cudaSuccess) return e;
        }
    const int64_t blocks = (int64_t)groups_of(d.n_heads) * runs_of(d.n_heads, num_sms);
    *bytes = (size_t)blocks * 2 * (size_t)piece_floats(d.latent_dim) * 4 + (size_t)d.max_requests * groups_of(d.n_heads) * sizeof(int2);
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
    p.out32 = reinterpret_cast<uintptr_t>(a.out) % 32 == 0 && a.out_stride_b % 16 == 0 && a.out_stride_h % 16 == 0;
    p.part = h.part;
    const int blocks = p.groups * p.runs;
    p.rec = reinterpret_cast<int2 *>(h.part + 2 * blocks * piece_floats(p.latent));
    const bool bf = a.act_type == MOE_BF16;
    for (p.box = kTile; p.box > 1 && a.page_size % p.box;) p.box /= 2;
    CUtensorMap cmap = {};
    const void *fn;
    if (a.cache_type == MOE_E4M3) {
        fn = kernel<kByCode>(bf);
    } else {
        // (rows that overlap have no map)
        const int64_t dims[3] = {p.dim, a.page_size, a.n_pages}, str[2] = {p.c_tok, a.n_pages > 1 ? p.c_page : p.c_tok * a.page_size};
        // Boxes of 8 rows and more keep the swizzle's atoms, small ones are slow. Measured, 64
        // requests, 128 heads, TMA and rows: pages of 8 tokens 190 and 148 us, 16: 147.6 and
        // 147.6, 32: 143.5 and 147.6, 64: 142 and 147.5
        const bool tma = p.box >= 32 && a.n_pages > 0 && p.c_tok >= 2 * p.dim && str[1] >= 2 * p.dim &&
                         encode_map(&cmap, bf ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16, 2, a.cache, 3, dims,
                                    str, p.box) == cudaSuccess;
        fn = tma ? kernel<kByTma>(bf) : kernel<kByRow>(bf);
    }
    void *args[] = {&cmap, &p};
    cudaError_t e = launch_after(fn, blocks, kThreads, kSmem, s, args);
    if (e != cudaSuccess) return e;
    return bf ? launch_join<__nv_bfloat16>(p, s) : launch_join<__half>(p, s);
}

cudaError_t latent_decode_flags(int32_t *out) {
    const int32_t zero = 0;
    cudaError_t e = cudaMemcpyFromSymbol(out, g_err, 4);
    if (e == cudaSuccess && *out) e = cudaMemcpyToSymbol(g_err, &zero, 4);
    return e;
}

}  // namespace moe
