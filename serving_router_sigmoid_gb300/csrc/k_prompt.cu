// k_prompt.cu -- attention of ragged prompts over keys and values expanded a
// head, the keys' rotary part shared by the heads (moe_latent_prompt):
//   s_ij = scale (qn_i . kn_j + qr_i . kr_j),  out_i = sum_j e^(s_ij) v_j / sum_j e^(s_ij)
//
// Both products run on tcgen05 with fp32 accumulators in tensor memory: S = Q K^T
// (128 queries by 128 keys) from shared memory, O += P V with the weights P in
// tensor memory (where S stood) and V an MN-major operand.  At 128 + 64 / 128
// dimensions a tile of keys is 768 + 512 cycles of the tensor core.
//
// - Narrow heads (values up to 128, keys up to 192 dimensions): a block holds 256
//   queries as two streams that share the keys; while one stream's softmax runs,
//   the tensor core works for the other (512 columns: S and O of both).  A warp a
//   stream issues its products (one for both: 112 against 95 us for 2048 tokens).  Wide
//   heads (to 256), and few blocks of 256 queries: 128 queries, S of two tiles in turn,
//   one O of 256 columns; one warp issues S, another PV, and both groups of softmax
//   warps work on one tile, half the columns each.
//   In both the order is S(0), S(1), PV(0), S(2), PV(1), ... over the steps, where
//   step k + 2 reuses the S buffer of step k.
// - A softmax thread holds a row (narrow) or half a row of logits in registers: no
//   shuffles.  The maximum moves only when a logit passes it by 2^kLazy; then the
//   row of O is scaled in tensor memory.  Weights are rounded to the operand type
//   (their sum is not), for f16 times 2^7, so that its subnormals begin at 2^-31.  The
//   result is off by 0.0021 (bf16) in the norm where its own rounding alone makes 0.0016;
//   a second term of the weights was measured: 0.0016, but 104 us for 91 (2048 tokens) and
//   183 for 157 (wide).
// - One warp brings tiles by TMA into a ring of 16 KB slots, several lanes at once: 128
//   keys by 64 dimensions, or as many rows of V as fit; tiles are handed on in halves
//   (narrow) or slots (wide).  What lies outside a tensor reads as
//   zeros; rows of V behind a request's last key, which belong to others, are set
//   to zero (a weight of 0 does not hide a NaN).
// - Blocks are persistent; work items (request, 256 or 128 queries, head) go to them
//   in turn and back, a request's last queries first: the longest come first where
//   the mask is causal.
//
// Measured: 2048 tokens, 64 heads of 128 + 64 / 128, causal: 91 us, 0.95 PFLOP/s (95 us where
// nothing is in L2); 1000 queries over 5000 keys, 32 heads of 192 + 64 / 256: 159 us, 0.93.  What bounds it is the
// chain of a step: some 300 to 440 cycles from a product's end to whoever waits for it, twice, and
// the softmax between (two steps of both streams 4560 cycles, their MMAs 2560).
#include <type_traits>

#include "tc_dev.cuh"

namespace moe {
namespace {

using namespace tc;

__device__ int32_t g_err;  // flags since the last read

constexpr uint32_t kSlot = 16384;
constexpr int kTiles = 8;         // narrow: tiles of keys or values in flight, at most
constexpr int kSlots = 14;        // slots of the ring, at most
// Wide: barriers of the slots' copies, in turn, one ring of them for keys and one for values,
// since each is waited for by another warp.  (One barrier a slot would have phases that a warp
// does not see: where the ring is shorter than a tile of keys and one of values, the
// copy before the awaited one may not have landed, and the parity is that of the one before.)
// More than slots, so none comes round before it was waited for.
constexpr int kTurns = 16;
// Tiles of values whose last rows are cleared, in flight at most (one an item).  The copies
// come to an item once S of the item before is complete; that S (wide, items of one
// tile) needs PV of the item two further back at most, by its two buffers.  So when an
// item's rows are cleared, those of the third one before have been waited for, and of
// three in flight none may share a barrier.
constexpr int kFixes = 4;
constexpr int kThreads = 352;     // 8 softmax warps, two that issue MMAs, one TMA warp
constexpr long long kStartClk = 20000;  // cycles that the second stream waits for the first to be ahead, at most
constexpr float kLazy = 8.f;
constexpr float kFloor = -3.4028235e38f;
constexpr float kLog2e = 1.4426950408889634f;
constexpr uint32_t kColO = 256;   // tensor memory: S twice 128 columns, then O

struct Params {
    MoePromptArgs a;
    float factor;                 // |scale| * log2(e)
    int negate;                   // scale < 0
    int nope_chunks, rope, chunks; // of 64 dimensions; chunks: with the rotary one
    int v_rows, v_boxes, v_slots; // rows of V in a slot, boxes of 64 dimensions, slots of 128 rows
    int slots;                    // of the ring
    int q_heads, k_heads, v_heads; // 0: one row for all heads
    int out32;
};

struct Shared {
    uint64_t full[kTurns], v_full[kTurns], empty[kSlots], q_full[2], q_empty[2], v_fixed[kFixes], s_full[2], p_ready[2][2], pv_done[2], o_full[2], o_empty[2], drain[2];
    uint32_t tmem;
    int abort;
    int began;                    // narrow: behind the last item whose first stream has weights
    float top[2][2][128];         // wide heads: the halves' row maxima, by the step's parity
};

// A work item: queries [q0, q0 + nq) of a request, its keys [k0, k0 + nk), and for
// each stream the tiles of 128 keys that its rows see.
struct Item {
    int head, q0, nq, k0, nk, last;   // last: the request's queries end `last` rows behind q0
    int tiles[2], n;
};

template <int NQ>
struct Cursor {
    int group = 0;                    // 32 requests from here on
    long long before = 0;             // blocks of queries before them
    // the it-th item of this block; the whole warp calls
    __device__ __forceinline__ bool item(const Params &p, int it, Item &x) {
        const MoePromptArgs &a = p.a;
        constexpr int kRows = 128 * NQ;
        const int G = gridDim.x, c = blockIdx.x, lane = threadIdx.x & 31;
        const long long idx = (long long)it * G + (it & 1 ? G - 1 - c : c);
        const long long unit = idx / a.n_heads;
        x.head = (int)(idx - unit * a.n_heads);
        for (; group < a.n_requests; group += 32) {
            const int b = group + lane;
            int q0 = 0, q1 = 0;
            if (b < a.n_requests) {
                q0 = max(ld_in(a.q_start + b), 0);
                q1 = min(ld_in(a.q_start + b + 1), a.n_queries);
            }
            const int blocks = q1 > q0 ? (q1 - q0 + kRows - 1) / kRows : 0;
            int sum = blocks;
#pragma unroll
            for (int d = 1; d < 32; d <<= 1) {
                const int v = __shfl_up_sync(0xffffffffu, sum, d);
                if (lane >= d) sum += v;
            }
            const int all = __shfl_sync(0xffffffffu, sum, 31);
            if (unit < before + all) {
                const int at = (int)(unit - before);
                const int from = __ffs(__ballot_sync(0xffffffffu, at < sum)) - 1;  // the lane of its request
                const int first = __shfl_sync(0xffffffffu, sum - blocks, from), nb = __shfl_sync(0xffffffffu, blocks, from);
                q0 = __shfl_sync(0xffffffffu, q0, from);
                q1 = __shfl_sync(0xffffffffu, q1, from);
                const int r = group + from;
                x.k0 = min(max(ld_in(a.kv_start + r), 0), a.n_keys);
                x.nk = max(min(ld_in(a.kv_start + r + 1), a.n_keys) - x.k0, 0);
                x.q0 = q0 + (nb - 1 - (at - first)) * kRows;
                x.last = q1 - x.q0;
                x.nq = min(x.last, kRows);
                x.n = 0;
#pragma unroll
                for (int g = 0; g < 2; ++g) {
                    const int rows = min(max(x.nq - 128 * g, 0), 128);
                    const int sees = rows ? seen(a, x, 128 * g + rows - 1) : 0;
                    x.tiles[g] = (sees + 127) / 128;
                    x.n = max(x.n, x.tiles[g]);
                }
                return true;
            }
            before += all;
        }
        return false;
    }
    // keys that row r of the item sees
    static __device__ __forceinline__ int seen(const MoePromptArgs &a, const Item &x, int r) {
        return a.causal ? max(min(x.nk - (x.last - r) + 1, x.nk), 0) : x.nk;
    }
};

// A position in the ring of slots.
struct Place {
    int slot = 0;
    uint32_t phase = 0;
    __device__ __forceinline__ void step(int n, int slots) {  // n <= slots
        if ((slot += n) >= slots) {
            slot -= slots;
            phase ^= 1;
        }
    }
};

__device__ __forceinline__ float ex2(float x) {
    float r;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
    return r;
}

__device__ __forceinline__ float max3(float a, float b, float c) {
    float r;
    asm("max.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
    return r;
}
// two fp32 operations an instruction, each rounded as by itself
__device__ __forceinline__ float2 fma2(float2 a, float b, float c) {
    unsigned long long x, y, z, r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(x) : "f"(a.x), "f"(a.y));
    asm("mov.b64 %0, {%1, %1};" : "=l"(y) : "f"(b));
    asm("mov.b64 %0, {%1, %1};" : "=l"(z) : "f"(c));
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(x), "l"(y), "l"(z));
    float2 o;
    asm("mov.b64 {%0, %1}, %2;" : "=f"(o.x), "=f"(o.y) : "l"(r));
    return o;
}
__device__ __forceinline__ float2 add2(float2 a, float2 b) {
    unsigned long long x, y, r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(x) : "f"(a.x), "f"(a.y));
    asm("mov.b64 %0, {%1, %2};" : "=l"(y) : "f"(b.x), "f"(b.y));
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(x), "l"(y));
    float2 o;
    asm("mov.b64 {%0, %1}, %2;" : "=f"(o.x), "=f"(o.y) : "l"(r));
    return o;
}

template <typename T, int NQ>
__global__ void __launch_bounds__(kThreads, 1)
    prompt_kernel(const __grid_constant__ CUtensorMap qmap, const __grid_constant__ CUtensorMap kmap,
                  const __grid_constant__ CUtensorMap rmap, const __grid_constant__ CUtensorMap vmap, const __grid_constant__ Params p) {
    constexpr bool BF = sizeof(T) == 2 && !std::is_same<T, __half>::value;
    extern __shared__ uint8_t raw[];
    __shared__ Shared sm;
    uint8_t *dyn = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(raw) + 1023) & ~uintptr_t(1023));
    const MoePromptArgs &a = p.a;
    const uint32_t ring = su32(dyn), qbase = ring + (uint32_t)p.slots * kSlot;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    volatile int *abort = &sm.abort;

    if (tid == 0) {
        for (int i = 0; i < kTurns; ++i) {  // narrow: one a tile, wide: one a copy
            mb_init(&sm.full[i], 1);
            mb_init(&sm.v_full[i], 1);
        }
        for (int i = 0; i < kSlots; ++i) mb_init(&sm.empty[i], NQ);  // narrow: one a tile, the streams; wide: one a slot
        for (int i = 0; i < kFixes; ++i) mb_init(&sm.v_fixed[i], 1);
        for (int i = 0; i < 2; ++i) {
            mb_init(&sm.q_full[i], 1);
            mb_init(&sm.q_empty[i], 1);
            mb_init(&sm.s_full[i], 1);
            for (int h = 0; h < 2; ++h) mb_init(&sm.p_ready[i][h], NQ == 2 ? 4 : 8);
            mb_init(&sm.pv_done[i], 1);
            mb_init(&sm.drain[i], 1);
            mb_init(&sm.o_full[i], 1);
            mb_init(&sm.o_empty[i], NQ == 2 ? 4 : 8);
        }
        sm.abort = 0;
        sm.began = 0;
        mb_init_done();
        tma_prefetch(&qmap);
        tma_prefetch(&kmap);
        tma_prefetch(&vmap);
    }
    if (warp == 8) tmem_alloc(&sm.tmem, 512);
    tc_before_sync();
    __syncthreads();
    tc_after_sync();
    const uint32_t tmem = sm.tmem;
    after_previous();

    Cursor<NQ> cur;
    Item x;

    if (warp == 10) {
        // ------------------------------------------------------------- TMA
        // Tiles take their slots in ring order and give them back in that order.
        const int nk = p.chunks, nv = p.v_slots;
        int slot = 0, room = p.slots;      // next slot, free ones
        uint32_t put = 0, got = 0;         // tiles brought, tiles whose slots are back
        uint32_t sizes = 0;                // of the tiles in flight, 4 bits each, the oldest lowest
        Place here;                        // wide: the next slot
        uint32_t kt = 0, vt = 0;           // and the copies of keys and of values so far
        uint32_t qp = 0, fixes = 0;
        bool ok = true;
        const auto take = [&](int n) {     // n free slots and a free pair of barriers
            while (ok && (room < n || put - got == kTiles)) {
                ok = __all_sync(0xffffffffu, mb_wait(&sm.empty[got % kTiles], got / kTiles & 1, abort, &g_err));
                room += (int)(sizes & 15);
                sizes >>= 4;
                ++got;
            }
            sizes |= (uint32_t)n << (4 * (put - got));
            room -= n;
        };
        for (int it = 0; ok && cur.item(p, it, x); ++it) {
            if (!x.n) continue;
            // a stream's queries, once its last product with the last ones is done
            const auto queries = [&](int g) {
                ok = __all_sync(0xffffffffu, ok && mb_wait(&sm.q_empty[g], qp ^ 1, abort, &g_err));
                if (ok && lane == 0) mb_expect_tx(&sm.q_full[g], (uint32_t)nk * kSlot);
                __syncwarp();
                if (ok && lane < nk) {
                    const int c = lane;
                    tma_3d(qbase + (uint32_t)(g * nk + c) * kSlot, &qmap, c < p.nope_chunks ? 64 * c : a.nope_dim, x.q0 + 128 * g,
                               p.q_heads * x.head, &sm.q_full[g]);
                }
                __syncwarp();
            };
            const uint32_t box = (uint32_t)p.v_rows * 128u;
            // rows of V behind the last key, as far as the last step of 16 goes, once they are there
            const auto clear = [&](int live, int begin) {
                const int n = (live + 15) / 16 * 16 - live;
                for (int i = lane; i < n * 8 * p.v_boxes; i += 32) {
                    const int c = i / (8 * n), r = live + i / 8 % n, part = r / p.v_rows;
                    const int at = begin + part < p.slots ? begin + part : begin + part - p.slots;
                    *reinterpret_cast<uint4 *>(dyn + (uint32_t)at * kSlot + (uint32_t)c * box + sw_off(r % p.v_rows, i & 7)) =
                        make_uint4(0, 0, 0, 0);
                }
                fence_async_smem();
                __syncwarp();
                if (lane == 0) mb_arrive(&sm.v_fixed[fixes % kFixes]);
                ++fixes;
            };
            // a slot's part of a tile: chunk c of the keys, or rows of the values
            const auto bring_k = [&](uint32_t at, int c, int j, uint64_t *full) {
                const int row = x.k0 + 128 * j;
                if (c < p.nope_chunks) tma_3d(at, &kmap, 64 * c, row, p.k_heads * x.head, full);
                else tma_2d(at, &rmap, 0, row, full);
            };
            const auto bring_v = [&](uint32_t at, int i, int c, int j, uint64_t *full) {
                tma_3d(at + (uint32_t)c * box, &vmap, 64 * c, x.k0 + 128 * j + i * p.v_rows, p.v_heads * x.head, full);
            };
            // Copies are issued by several lanes at once: a single thread gets 32 to 43
            // bytes a cycle from the TMA unit, four lanes or two warps 70.
            const auto keys = [&](int j) {
                if (NQ == 1) {
                    for (int c = 0; c < nk && ok; c += 2) {  // two slots at a time
                        const int n = min(2, nk - c);
                        Place mine = here;
                        if (lane & 1) mine.step(1, p.slots);
                        ok = __all_sync(0xffffffffu, lane >= n || mb_wait(&sm.empty[mine.slot], mine.phase ^ 1, abort, &g_err));
                        if (ok && lane < n) {
                            uint64_t *const full = &sm.full[(kt + lane) % kTurns];
                            mb_expect_tx(full, kSlot);
                            bring_k(ring + (uint32_t)mine.slot * kSlot, c + lane, j, full);
                        }
                        __syncwarp();
                        here.step(n, p.slots);
                        if (ok) kt += n;
                    }
                    return;
                }
                take(nk);
                if (!ok) return;
                uint64_t *const full = &sm.full[put % kTiles];
                if (lane == 0) mb_expect_tx(full, (uint32_t)nk * kSlot);
                __syncwarp();
                const int at = slot + lane < p.slots ? slot + lane : slot + lane - p.slots;
                if (lane < nk) bring_k(ring + (uint32_t)at * kSlot, lane, j, full);
                __syncwarp();
                slot = slot + nk < p.slots ? slot + nk : slot + nk - p.slots;
                ++put;
            };
            const auto values = [&](int j) {
                const int live = x.nk - 128 * j;   // rows of this request
                if (NQ == 1) {
                    const int begin = here.slot;
                    for (int i = 0; i < nv && ok; ++i, ++vt, here.step(1, p.slots)) {
                        uint64_t *const full = &sm.v_full[vt % kTurns];
                        if (!(ok = __all_sync(0xffffffffu, mb_wait(&sm.empty[here.slot], here.phase ^ 1, abort, &g_err)))) return;
                        if (lane == 0) mb_expect_tx(full, (uint32_t)p.v_boxes * box);
                        __syncwarp();
                        if (lane < p.v_boxes) bring_v(ring + (uint32_t)here.slot * kSlot, i, lane, j, full);
                        __syncwarp();
                    }
                    if (live < 128) {
                        for (uint32_t i = vt - nv; i != vt && ok; ++i)
                            ok = __all_sync(0xffffffffu, mb_wait(&sm.v_full[i % kTurns], i / kTurns & 1, abort, &g_err));
                        if (ok) clear(live, begin);
                    }
                    return;
                }
                take(nv);
                if (!ok) return;
                uint64_t *const full = &sm.full[put % kTiles];
                const int begin = slot, i = lane >> 2;  // four lanes a slot
                if (lane == 0) mb_expect_tx(full, (uint32_t)(nv * p.v_boxes) * box);
                __syncwarp();
                const int at = slot + i < p.slots ? slot + i : slot + i - p.slots;
                if (i < nv && (lane & 3) < p.v_boxes) bring_v(ring + (uint32_t)at * kSlot, i, lane & 3, j, full);
                __syncwarp();
                slot = slot + nv < p.slots ? slot + nv : slot + nv - p.slots;
                if (live < 128) {
                    ok = __all_sync(0xffffffffu, mb_wait(full, put / kTiles & 1, abort, &g_err));
                    if (ok) clear(live, begin);
                }
                ++put;
            };
            queries(0);
            for (int j = 0; j < x.n && ok; ++j) {
                keys(j);
                if (NQ == 2 && j == 0) queries(1);
                if (!ok) break;
                if (NQ == 2) values(j);
                else if (j) values(j - 1);
            }
            if (NQ == 1 && ok) values(x.n - 1);
            qp ^= 1;
        }
        if (*abort) {  // copies in flight land before the block ends
            const long long t = clock64();
            for (uint32_t i = kt > kTurns ? kt - kTurns : 0; i < kt; ++i)
                while (!mb_test(&sm.full[i % kTurns], i / kTurns & 1) && clock64() - t < kWaitClk) {}
            for (uint32_t i = vt > kTurns ? vt - kTurns : 0; i < vt; ++i)
                while (!mb_test(&sm.v_full[i % kTurns], i / kTurns & 1) && clock64() - t < kWaitClk) {}
            for (uint32_t i = put > kTiles ? put - kTiles : 0; i < put; ++i)
                while (!mb_test(&sm.full[i % kTiles], i / kTiles & 1) && clock64() - t < kWaitClk) {}
        }
    } else if (warp >= 8) {
        // -------------------------------------------------------------- MMA
        // Two warps issue (an issue takes 40 to 100 cycles, more than a short MMA), narrow:
        // one a stream, so that its S follows its PV without a word; wide: one the first
        // products, the other the second ones.
        const uint32_t fmt = BF ? 1 : 0;
        const uint32_t id_s = idesc(fmt, 0, 0, 128, 128), id_o = idesc(fmt, 0, 1, 128, a.v_dim);
        const uint32_t dq = desc(qbase, 16), dk = desc(ring, 16), dv = desc(ring, (uint32_t)p.v_rows * 128u);
        const int rest = (a.nope_dim % 64) / 16, rope_steps = a.rope_dim / 16, per = p.v_rows / 16, lper = 31 - __clz(per);
        const bool lead = elect();
        const int nk = p.chunks, nv = p.v_slots, slots = p.slots;
        const auto wait = [&](uint64_t *bar, uint32_t phase) { return __all_sync(0xffffffffu, mb_wait(bar, phase, abort, &g_err)); };
        const auto ahead = [&](int slot, int n) { return slot + n < slots ? slot + n : slot + n - slots; };
        // S of the keys at a slot, issued by one lane
        const auto product_s = [&](uint32_t d, uint32_t q, int at, int c0, int c1) {
#pragma unroll 1
            for (int c = c0; c < c1; ++c, q += kSlot >> 4) {
                const uint32_t k = dk + (uint32_t)(at * (int)(kSlot >> 4));
                const int n = c >= p.nope_chunks ? rope_steps : c + 1 == p.nope_chunks && rest ? rest : 4;
                if (n == 4) {
#pragma unroll
                    for (int e = 0; e < 4; ++e) mma_f16(d, q + 2 * e, k + 2 * e, id_s, c + e != 0);
                } else {
#pragma unroll 1
                    for (int e = 0; e < n; ++e) mma_f16(d, q + 2 * e, k + 2 * e, id_s, c + e != 0);
                }
                if (++at == slots) at = 0;
            }
        };
        // O += P V for steps [e0, e1) of 16 keys; the second 64 weights stand 64 columns on
        const auto product_o = [&](uint32_t d, uint32_t w, int at, int e0, int e1, bool starts) {
            w += e0 < 4 ? 8 * e0 : 64 + 8 * (e0 - 4);
            at = ahead(at, e0 >> lper);
            int left = per - (e0 & (per - 1));
            uint32_t v = dv + (uint32_t)(at * (int)(kSlot >> 4)) + (uint32_t)(e0 & (per - 1)) * (2048 >> 4);
#pragma unroll 1
            for (int e = e0; e < e1; e += 2) {      // a slot holds an even number of steps
                mma_f16_ta(d, w, v, id_o, !(starts && e == 0));
                if (e + 1 < e1) mma_f16_ta(d, w + 8, v + (2048 >> 4), id_o, 1);
                w += e == 2 ? 48 : 16;
                v += 2 * (2048 >> 4);
                if ((left -= 2) == 0) {
                    if (++at == slots) at = 0;
                    v = dv + (uint32_t)(at * (int)(kSlot >> 4));
                    left = per;
                }
            }
        };
        // Tiles come, narrow: K0 V0 K1 V1 ..., wide: K0 K1 V0 K2 V1 ..., as they are first used.
        int slot = 0;                      // of the next item's first keys
        uint32_t tile = 0;                 // the same as a tile, counted as they come
        uint32_t uses[2] = {0, 0};         // of the S buffers, the last bit
        uint32_t step = 0, fixes = 0, qf = 0;
        bool ok = true;
        const bool firsts = warp == 8;
        if (NQ == 2) {
            const int g = warp - 8;
            uint32_t oe = 0;
            const uint32_t sd = tmem + 128 * g, od = tmem + kColO + 128 * g, q = dq + (uint32_t)(g * nk * (int)(kSlot >> 4));
            for (int it = 0; ok && cur.item(p, it, x); ++it) {
                if (!x.n) continue;
                const int mine = x.tiles[g], other = x.tiles[g ^ 1];
                if (!(ok = wait(&sm.q_full[g], qf))) break;
                qf ^= 1;
                // S of tile j, issued by one lane; its keys are free when both streams have read them
                const auto first = [&](int j) {
                    const uint32_t t = tile + 2 * j;
                    product_s(sd, q, slot, 0, nk);
                    mma_commit(&sm.s_full[g]);
                    mma_commit(&sm.empty[t % kTiles]);
                    if (j + 1 == mine) mma_commit(&sm.q_empty[g]);
                };
                const auto keys = [&](int j) { return wait(&sm.full[(tile + 2 * j) % kTiles], (tile + 2 * j) / kTiles & 1); };
                // The second stream starts when the first has weights: the products of one then
                // run under the softmax of the other (8 heads of 8192 tokens 157 us, without it 172;
                // 20 x 300, 16 heads 41.9 and 39.8; 64 heads of 2048 91 either way).  This is for
                // speed alone, and the first stream may be tiles or an item further by now: so it is a
                // count, compared, and given up after a while (a barrier's parity would come round).
                if (g == 1 && mine && other) {
                    const long long t = clock64();
                    while (*(volatile int *)&sm.began <= it && !*abort && clock64() - t < kStartClk) {}
                    __syncwarp();
                }
                if (mine) {
                    if (!(ok = keys(0))) break;
                    tc_after_sync();
                    if (lead) first(0);
                    __syncwarp();
                } else if (lead) mma_commit(&sm.q_empty[g]);
                for (int j = 0; j < x.n; ++j) {
                    const int live = x.nk - 128 * j, vs = ahead(slot, nk);
                    const uint32_t fix = fixes, t = tile + 2 * j + 1;
                    if (live < 128) ++fixes;
                    if (j < mine) {
                        const int steps = (min(live, 128) + 15) / 16;
                        ok = wait(&sm.full[t % kTiles], t / kTiles & 1) && (live >= 128 || wait(&sm.v_fixed[fix % kFixes], fix / kFixes & 1)) &&
                             (j || wait(&sm.o_empty[g], oe ^ 1)) && wait(&sm.p_ready[g][0], uses[0]);
                        if (!ok) break;
                        if (!j) oe ^= 1;
                        tc_after_sync();
                        if (lead) {
                            product_o(od, sd, vs, 0, min(steps, 4), j == 0);
                            mma_commit(&sm.pv_done[g]);
                        }
                        __syncwarp();
                        const bool more = j + 1 < mine;
                        if (!(ok = wait(&sm.p_ready[g][1], uses[0]))) break;
                        uses[0] ^= 1;
                        tc_after_sync();
                        slot = ahead(slot, nk + nv);
                        if (lead) {
                            product_o(od, sd, vs, 4, steps, false);
                            mma_commit(&sm.empty[t % kTiles]);
                            if (!more) mma_commit(&sm.o_full[g]);
                        }
                        __syncwarp();
                        if (more) {
                            if (!(ok = keys(j + 1))) break;
                            tc_after_sync();
                            if (lead) first(j + 1);
                            __syncwarp();
                        }
                    } else {
                        // A tile for the other stream alone is waited for and given back all the same: a
                        // phase of its barrier that goes by unseen could be taken for a later one
                        if (!(ok = wait(&sm.full[(t - 1) % kTiles], (t - 1) / kTiles & 1) &&
                                   wait(&sm.full[t % kTiles], t / kTiles & 1)))
                            break;
                        if (lead) {
                            mb_arrive(&sm.empty[(t - 1) % kTiles]);
                            mb_arrive(&sm.empty[t % kTiles]);
                        }
                        __syncwarp();
                        slot = ahead(slot, nk + nv);
                    }
                }
                tile += 2 * x.n;
            }
        } else if (firsts) {
            // ---- S = Q K^T, a slot of keys after the other
            Place at;
            uint32_t began = 0, kt = 0;
            for (int it = 0; ok && cur.item(p, it, x); ++it) {
                if (!x.n) continue;
                if (!(ok = wait(&sm.q_full[0], qf))) break;
                qf ^= 1;
                for (int j = 0; j < x.n && ok; ++j) {
                    const int b = (int)(step++ & 1);
                    // the weights of the step before in this buffer have been read
                    if (began >> b & 1 && !(ok = wait(&sm.pv_done[b], uses[b] ^ 1))) break;
                    began |= 1u << b;
                    uses[b] ^= 1;
                    uint32_t q = dq;
                    for (int c = 0; c < nk; ++c, ++kt, q += kSlot >> 4, at.step(1, slots)) {
                        if (!(ok = wait(&sm.full[kt % kTurns], kt / kTurns & 1))) break;
                        tc_after_sync();
                        if (lead) {
                            product_s(tmem + 128 * b, q, at.slot, c, c + 1);
                            mma_commit(&sm.empty[at.slot]);
                            if (c + 1 == nk) mma_commit(&sm.s_full[b]);
                        }
                        __syncwarp();
                    }
                    if (j) at.step(nv, slots);
                }
                if (ok && lead) mma_commit(&sm.q_empty[0]);
                __syncwarp();
                at.step(nv, slots);        // the last values stand before the next keys
            }
        } else {
            // ---- O += P V
            Place at;
            uint32_t oe = 0, vt = 0;
            for (int it = 0; ok && cur.item(p, it, x); ++it) {
                if (!x.n) continue;
                at.step(nk, slots);
                if (x.n > 1) at.step(nk, slots);
                for (int j = 0; j < x.n && ok; ++j) {
                    const int live = x.nk - 128 * j, steps = (min(live, 128) + 15) / 16, b = (int)(step++ & 1);
                    if (live < 128) {
                        if (!(ok = wait(&sm.v_fixed[fixes % kFixes], fixes / kFixes & 1))) break;
                        ++fixes;
                    }
                    if (!(ok = (j || wait(&sm.o_empty[0], oe ^ 1)) && wait(&sm.p_ready[b][0], uses[b]))) break;
                    uses[b] ^= 1;
                    if (!j) oe ^= 1;
                    for (int i = 0; i < nv; ++i, ++vt, at.step(1, slots)) {
                        if (!(ok = wait(&sm.v_full[vt % kTurns], vt / kTurns & 1))) break;
                        tc_after_sync();
                        if (lead) {
                            product_o(tmem + kColO, tmem + 128 * b, ahead(at.slot, slots - i), per * i, min(steps, per * (i + 1)), j == 0);
                            mma_commit(&sm.empty[at.slot]);
                            if (i + 1 == nv) {
                                mma_commit(&sm.pv_done[b]);
                                if (j + 1 == x.n) mma_commit(&sm.o_full[0]);
                            }
                        }
                        __syncwarp();
                    }
                    if (j + 2 < x.n) at.step(nk, slots);
                }
            }
        }
        if (*abort) {  // what was issued ends before the tensor memory is freed
            if (lead) mma_commit(&sm.drain[warp - 8]);
            const long long t = clock64();
            while (!mb_test(&sm.drain[warp - 8], 0) && clock64() - t < kWaitClk) {}
        }
        __syncwarp();
    } else {
        // ---------------------------------------------------------- softmax
        constexpr float kOff = BF ? 0.f : 7.f;
        const int g = warp >> 2, row = tid & 127;      // stream (narrow) or half of the columns (wide)
        const uint32_t quad = (uint32_t)((warp & 3) * 32) << 16;
        T *out = static_cast<T *>(a.out);
        uint32_t sf[2] = {0, 0}, pd[2] = {0, 0}, of = 0, step = 0;
        const int o = NQ == 2 ? g : 0;
        for (int it = 0; cur.item(p, it, x); ++it) {
            const int q = NQ == 2 ? 128 * g + row : row;   // of the item
            const bool mine = q < x.nq;
            const int tiles = NQ == 2 ? x.tiles[g] : x.n;
            const int sees = mine ? Cursor<NQ>::seen(a, x, q) : 0;
            // tiles that every row of this warp sees whole need no mask
            const int lead_row = q & ~31;
            const int whole = lead_row + 31 < x.nq ? Cursor<NQ>::seen(a, x, lead_row) / 128 : 0;
            float m = kFloor, l = 0.f;                 // the maximum in units of the logits
            // Steps of 64 logits a thread: narrow, the halves of a tile one after the other,
            // each handed on by itself; wide, this group's half.
            const int halves = NQ == 2 ? 2 : 1;
#pragma unroll 1
            for (int j = 0; j < tiles * halves; ++j) {
                const int half = NQ == 2 ? j & 1 : g, b = NQ == 2 ? g : (int)(step & 1), ph = NQ == 2 ? half : 0;
                if (NQ == 1 || !half) {
                    mb_wait(&sm.s_full[b], sf[b], abort, &g_err);
                    sf[b] ^= 1;
                    tc_after_sync();
                }
                const uint32_t at = tmem + quad + 128 * b + 64 * half;               // this thread's columns
                const int tile = NQ == 2 ? j >> 1 : j, sees_here = sees - 128 * tile - 64 * half;  // those that count
                const bool masked = tile >= whole;
                uint32_t s[2][32];
                tmem_ld(at, s[0]);
                tmem_ld(at + 32, s[1]);
                tmem_wait_ld();
                if (p.negate) {
#pragma unroll
                    for (int c = 0; c < 64; ++c) s[c >> 5][c & 31] ^= 0x80000000u;
                }
                if (masked) {
#pragma unroll
                    for (int c = 0; c < 64; ++c)
                        if (c >= sees_here) s[c >> 5][c & 31] = 0xff800000u;
                }
                float t4[4] = {kFloor, kFloor, kFloor, kFloor};
#pragma unroll
                for (int c = 0; c < 64; c += 2)
                    t4[c >> 1 & 3] = max3(t4[c >> 1 & 3], __uint_as_float(s[c >> 5][c & 31]), __uint_as_float(s[c >> 5][(c & 31) + 1]));
                float top = fmaxf(max3(t4[0], t4[1], t4[2]), t4[3]);
                if (NQ == 1) {                         // the row's other half
                    sm.top[step & 1][g][row] = top;
                    asm volatile("bar.sync 1, 256;" ::: "memory");
                    top = fmaxf(top, sm.top[step & 1][g ^ 1][row]);
                }
                if (j == 0) {
                    m = top;
                } else if (__any_sync(0xffffffffu, top * p.factor > m * p.factor + kLazy)) {
                    const float to = fmaxf(m, top), f = ex2((m - to) * p.factor);
                    m = to;
                    l *= f;
                    // O of the steps before is complete, then its rows are scaled
                    // (narrow: S of this tile came after all of the tile before)
                    if (NQ == 2 && half) mb_wait(&sm.pv_done[g], pd[0], abort, &g_err);
                    if (NQ == 1) mb_wait(&sm.pv_done[b ^ 1], pd[b ^ 1] ^ 1, abort, &g_err);
                    tc_after_sync();
                    const int c0 = NQ == 2 ? 0 : 16 * g, c1 = a.v_dim, dc = NQ == 2 ? 16 : 32;
                    for (int c = c0; c < c1; c += dc) {
                        uint32_t v[16];
                        tmem_ld(tmem + quad + kColO + 128 * o + c, v);
                        tmem_wait_ld();
#pragma unroll
                        for (int k = 0; k < 16; ++k) v[k] = __float_as_uint(__uint_as_float(v[k]) * f);
                        tmem_st(tmem + quad + kColO + 128 * o + c, v);
                    }
                }
                if (NQ == 1) pd[b] ^= 1;
                else if (half) pd[0] ^= 1;
                const float mf = kOff - m * p.factor;
                float2 l2 = make_float2(0.f, 0.f);
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    uint32_t w[16];
#pragma unroll
                    for (int c = 0; c < 32; c += 2) {
                        float2 e = fma2(make_float2(__uint_as_float(s[h][c]), __uint_as_float(s[h][c + 1])), p.factor, mf);
                        e.x = ex2(e.x);
                        e.y = ex2(e.y);
                        if (masked) {                  // not by the logit: nothing is known of factor and m
                            e.x = 32 * h + c < sees_here ? e.x : 0.f;
                            e.y = 32 * h + c + 1 < sees_here ? e.y : 0.f;
                        }
                        l2 = add2(l2, e);
                        w[c >> 1] = pack_pair(e.x, e.y, T());
                    }
                    tmem_st(at + 16 * h, w);           // over logits that were read
                }
                l += l2.x + l2.y;
                tmem_wait_st();
                tc_before_sync();
                __syncwarp();
                if (lane == 0) mb_arrive(&sm.p_ready[b][ph]);
                if (NQ == 2 && j == 0 && tid == 0) *(volatile int *)&sm.began = it + 1;
                if (NQ == 1 || half) ++step;
            }
            if (NQ == 1) {                             // the row's whole sum
                sm.top[step & 1][g][row] = l;
                asm volatile("bar.sync 1, 256;" ::: "memory");
                l += sm.top[step & 1][g ^ 1][row];
                asm volatile("bar.sync 1, 256;" ::: "memory");
            }
            const float inv = l > 0.f ? 1.f / l : 0.f;
            T *to = out + (int64_t)(x.q0 + q) * a.out_stride_t + (int64_t)x.head * a.out_stride_h;
            if (tiles) {
                mb_wait(&sm.o_full[o], of, abort, &g_err);
                of ^= 1;
                tc_after_sync();
            }
            const int c0 = NQ == 2 ? 0 : 16 * g, dc = NQ == 2 ? 16 : 32;
            for (int c = c0; c < a.v_dim; c += dc) {
                uint32_t v[16], y[8];
                if (tiles) {
                    tmem_ld(tmem + quad + kColO + 128 * o + c, v);
                    tmem_wait_ld();
                }
                if (!mine) continue;
#pragma unroll
                for (int k = 0; k < 8; ++k)
                    y[k] = tiles ? pack_pair(__uint_as_float(v[2 * k]) * inv, __uint_as_float(v[2 * k + 1]) * inv, T()) : 0u;
                if (l == 0.f)
#pragma unroll
                    for (int k = 0; k < 8; ++k) y[k] = 0u;
                if (p.out32) {
                    st32(to + c, y);
                } else {
#pragma unroll
                    for (int k = 0; k < 16; ++k) reinterpret_cast<uint16_t *>(to)[c + k] = (uint16_t)(y[k >> 1] >> (16 * (k & 1)));
                }
            }
            if (mine && a.lse && (NQ == 2 || g == 0))
                a.lse[(int64_t)(x.q0 + q) * a.n_heads + x.head] = l > 0.f ? (m * p.factor - kOff) / kLog2e + logf(l) : -INFINITY;
            if (tiles) {
                tc_before_sync();
                __syncwarp();
                if (lane == 0) mb_arrive(&sm.o_empty[o]);
            }
        }
    }

    tc_before_sync();
    __syncthreads();
    tc_after_sync();
    if (warp == 8) tmem_free(tmem, 512);
}

template <typename T, int NQ>
cudaError_t launch(const MoePromptArgs &a, Params &p, int dev, int sms, cudaStream_t s) {
    const int v_pad = (a.v_dim + 63) / 64;
    p.v_boxes = v_pad;
    p.v_rows = v_pad == 1 ? 128 : v_pad == 2 ? 64 : 32;
    p.v_slots = 128 / p.v_rows;
    p.slots = (int)((227 * 1024 - 1024 - sizeof(Shared) - 64) / kSlot) - NQ * p.chunks;
    static_assert((227 * 1024 - 1024 - sizeof(Shared) - 64) / kSlot <= kSlots && kSlots <= kTurns, "barriers of the ring");
    const CUtensorMapDataType type = std::is_same<T, __half>::value ? CU_TENSOR_MAP_DATA_TYPE_FLOAT16 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16;
    CUtensorMap maps[4] = {};
    const auto map = [&](int i, const void *base, int dim, int rows, int64_t st, int64_t sh, int &heads, int box) {
        const bool one = a.n_heads == 1 || sh == 0;
        heads = one ? 0 : 1;
        const int64_t row = (2 * dim + 15) / 16 * 16;
        const int64_t d[3] = {dim, rows, one ? 1 : a.n_heads}, str[2] = {rows > 1 ? 2 * st : row, one ? row : 2 * sh};
        return encode_map(&maps[i], type, 2, base, 3, d, str, box);
    };
    cudaError_t e = map(0, a.q, a.nope_dim + a.rope_dim, a.n_queries, a.q_stride_t, a.q_stride_h, p.q_heads, 128);
    // without keys nothing is loaded: any valid map will do
    if (e == cudaSuccess) e = a.n_keys ? map(1, a.k, a.nope_dim, a.n_keys, a.k_stride_t, a.k_stride_h, p.k_heads, 128) : (maps[1] = maps[0], cudaSuccess);
    if (e == cudaSuccess) e = a.n_keys ? map(3, a.v, a.v_dim, a.n_keys, a.v_stride_t, a.v_stride_h, p.v_heads, p.v_rows) : (maps[3] = maps[0], cudaSuccess);
    if (e == cudaSuccess && a.rope_dim && a.n_keys) {
        const int64_t d[3] = {a.rope_dim, a.n_keys, 1}, str[2] = {a.n_keys > 1 ? 2 * a.kr_stride_t : 128, 0};
        e = encode_map(&maps[2], type, 2, a.k_rope, 2, d, str, 128);
    } else {
        maps[2] = maps[0];
    }
    if (e != cudaSuccess) return e;
    const size_t smem = (size_t)(p.slots + NQ * p.chunks) * kSlot + 1024;
    auto fn = prompt_kernel<T, NQ>;
    static SmemOnce once;
    if ((e = once.allow(reinterpret_cast<const void *>(fn), dev, 227 * 1024 - sizeof(Shared) - 64)) != cudaSuccess) return e;
    // no more blocks than there can be items
    const int64_t most = ((int64_t)a.n_queries / (128 * NQ) + a.n_requests) * a.n_heads;
    void *args[] = {&maps[0], &maps[1], &maps[2], &maps[3], &p};
    return launch_after(reinterpret_cast<const void *>(fn), (int)(most < sms ? most : sms), kThreads, smem, s, args);
}

}  // namespace

cudaError_t launch_latent_prompt(const MoePromptArgs &a, cudaStream_t s) {
    int dev = 0, sms = 0;
    cudaError_t e = current_sms(&dev, &sms);
    if (e != cudaSuccess) return e;
    Params p = {};
    p.a = a;
    p.factor = (a.scale < 0 ? -a.scale : a.scale) * kLog2e;
    p.negate = a.scale < 0;
    p.nope_chunks = (a.nope_dim + 63) / 64;
    p.chunks = p.nope_chunks + (a.rope_dim > 0);
    p.out32 = reinterpret_cast<uintptr_t>(a.out) % 32 == 0 && a.out_stride_t % 16 == 0 && a.out_stride_h % 16 == 0;
    // Two streams where heads are narrow enough, blocks of 256 queries give every SM
    // work, and requests hold more than 128 queries on average: a shorter one leaves the
    // second stream without a tile.  Measured, heads of 128 + 64 / 128, two streams and one:
    // 2048 queries, 16 heads (128 blocks) 42.7 and 28.7 us, 32 heads 46.2 and 53.8, 64 heads
    // 91.5 and 104.6; 5 x 250, 16 heads 11.1 and 8.6; requests of 40 queries, 100 with 16 heads
    // 44.5 and 43.5, with 64 heads 170 and 163; 40 of 100 behind 900 others 96.8 and 80.8; 20
    // of 128, 64 heads 44.0 and 42.0; 40 of 160, 16 heads 41.9 and 42.4; 20 of 256, 64 heads 73.9
    // and 82.2; 100 of 20 and one of 1000, 16 heads 61.6 and 57.6; 40 of up to 500 (302 on
    // average), 16 heads 73.8 and 75.7, 64 heads (240) 209 and 204
    const bool narrow = a.v_dim <= 128 && p.chunks <= 3 && (a.n_queries + 255ll) / 256 * a.n_heads >= sms &&
                        a.n_queries > 128ll * a.n_requests;
    if (a.act_type == MOE_F16) return narrow ? launch<__half, 2>(a, p, dev, sms, s) : launch<__half, 1>(a, p, dev, sms, s);
    return narrow ? launch<__nv_bfloat16, 2>(a, p, dev, sms, s) : launch<__nv_bfloat16, 1>(a, p, dev, sms, s);
}

cudaError_t latent_prompt_flags(int32_t *out) {
    const int32_t zero = 0;
    cudaError_t e = cudaMemcpyFromSymbol(out, g_err, 4);
    if (e == cudaSuccess && *out) e = cudaMemcpyToSymbol(g_err, &zero, 4);
    return e;
}

}  // namespace moe
