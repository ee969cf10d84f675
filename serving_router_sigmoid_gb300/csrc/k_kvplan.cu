// k_kvplan.cu -- page allocation, positions and cache slots of a batch's new
// tokens, from the lengths on the GPU (moe_kv_plan).
//
// With have = ceil(past / P) and need = ceil((past + new) / P), both at most the
// entries of a table row (a page that no row can hold stays on the free list),
// take = need - have and off the exclusive prefix sum of take over the requests:
//   table[b, have + j] = free[head + off[b] + j]           (j < take[b])
//   token i of request b: pos = past + i, slot = table[b, pos / P] * P + pos % P
//
// Bytes are few (12 a token, 16 a request), so the launch and the dependent
// round trips (lengths, free list, stores) are what it costs.  One launch:
// every block forms both prefix sums for itself in shared memory (8 bytes a
// request, from L2 after the first block), which costs less than a second
// launch or a hand-over between blocks, and then takes its share of the tokens
// and pages; a new token's page comes from the free list itself, never from a
// table entry that another block may be writing.  8 requests of one token: 4.0
// us; 512 requests with 360k tokens (4.5 MB written): 6.2 us.  Each 512 requests are
// a round of loads and scan that waits for the one before: 1500 requests of one
// token 8.4 us, 8192 18.9.
#include "attn_args.cuh"

namespace moe {
namespace {

constexpr int kThreads = 512;
constexpr int kTok = 4;  // consecutive tokens of a thread: 16-byte stores of positions

// Exclusive prefix sums of two ints over the block, and their totals.
__device__ __forceinline__ void block_scan2(int &a, int &b, int &ta, int &tb, int2 *wsum) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    int x = a, y = b;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int u = __shfl_up_sync(0xffffffffu, x, o), v = __shfl_up_sync(0xffffffffu, y, o);
        if (lane >= o) { x += u; y += v; }
    }
    __syncthreads();  // the previous round's wsum has been read
    if (lane == 31) wsum[warp] = make_int2(x, y);
    __syncthreads();
    int bx = 0, by = 0;
    ta = tb = 0;
#pragma unroll
    for (int w = 0; w < kThreads / 32; ++w) {
        const int2 s = wsum[w];
        if (w < warp) { bx += s.x; by += s.y; }
        ta += s.x; tb += s.y;
    }
    a = bx + x - a;
    b = by + y - b;
}

// Largest i in [0, n) with v[i] <= x (v ascending, v[0] <= x).
__device__ __forceinline__ int last_le(const int *v, int n, int x) {
    int lo = 0, hi = n;
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (v[mid] <= x) lo = mid; else hi = mid;
    }
    return lo;
}

__global__ void __launch_bounds__(kThreads) kv_plan_kernel(KvPlanArgs a, FastDiv by_page) {
    after_previous();
    extern __shared__ int sh[];
    int *start = sh, *off = sh + a.n_req + 1;  // [n_req + 1] each
    __shared__ int2 wsum[kThreads / 32];
    __shared__ int s_flags, s_longest;
    const int tid = threadIdx.x;
    const bool first = blockIdx.x == 0;
    if (tid == 0) s_flags = 0, s_longest = 0;
    int n_new = 0, n_take = 0;
    int flags = 0, longest = 0;
    for (int base = 0; base < a.n_req; base += kThreads) {
        const int b = base + tid;
        int past = 0, fresh = 0;
        if (b < a.n_req) {
            past = ld_in(a.past + b);
            fresh = ld_in(a.fresh + b);
            if (past < 0 || fresh < 0) flags |= MOE_PLAN_NEGATIVE;
            past = max(past, 0);
            fresh = max(fresh, 0);
        }
        const int need = (int)by_page.div((uint32_t)(past + fresh) + a.page - 1);
        const int have = (int)by_page.div((uint32_t)past + a.page - 1);
        const int take = min(need, a.max_pages) - min(have, a.max_pages);
        if (need > a.max_pages) flags |= MOE_PLAN_ROW_FULL;
        longest = max(longest, past + fresh);
        int s = fresh, o = take, ts, to;
        block_scan2(s, o, ts, to, wsum);
        if (b < a.n_req) {
            start[b] = n_new + s;
            off[b] = n_take + o;
            if (first) {
                a.q_start[b] = n_new + s;
                a.seq_len[b] = past + fresh;
            }
        }
        n_new += ts;
        n_take += to;
    }
    if (tid == 0) start[a.n_req] = n_new, off[a.n_req] = n_take;
    int head = ld_in(a.free_head);
    if (head < 0) flags |= MOE_PLAN_NEGATIVE, head = 0;
    const int avail = max(a.n_free - head, 0);
    if (first) {
        if (flags) atomicOr(&s_flags, flags);
        atomicMax(&s_longest, longest);
    }
    __syncthreads();
    if (first && tid == 0) {
        int f = s_flags;
        if (n_take > avail) f |= MOE_PLAN_NO_PAGES;
        if (n_new > a.max_new) f |= MOE_PLAN_NO_ROOM;
        a.q_start[a.n_req] = n_new;
        a.info[0] = n_new;
        a.info[1] = head + min(n_take, avail);
        a.info[2] = f;
        a.info[3] = s_longest;
    }
    const int nthr = gridDim.x * kThreads, me = blockIdx.x * kThreads + tid;
    // the new pages' table entries
    for (int64_t j = me; j < n_take; j += nthr) {
        const int i = (int)j;
        const int b = last_le(off, a.n_req, i);
        const int col = (int)by_page.div((uint32_t)max(ld_in(a.past + b), 0) + a.page - 1) + i - off[b];
        if (col >= 0 && col < a.max_pages)
            a.table[b * a.table_stride + col] = i < avail ? ld_in(a.free_pages + head + i) : -1;
    }
    // positions and slots
    const bool vec = (reinterpret_cast<uintptr_t>(a.positions) & 15u) == 0 &&
                     (reinterpret_cast<uintptr_t>(a.slots) & 15u) == 0;
    for (int64_t t0 = (int64_t)me * kTok; t0 < a.max_new; t0 += (int64_t)nthr * kTok) {
        int pos[kTok];
        long long slot[kTok];
        int b = -1, past = 0, have = 0;
#pragma unroll
        for (int i = 0; i < kTok; ++i) {
            const int t = (int)t0 + i;
            pos[i] = 0;
            slot[i] = -1;
            if (t0 + i >= a.max_new || t >= n_new) continue;
            if (b < 0 || t >= start[b + 1]) {
                b = last_le(start, a.n_req, t);
                past = max(ld_in(a.past + b), 0);
                have = (int)by_page.div((uint32_t)past + a.page - 1);
            }
            const int p = past + t - start[b];
            const int col = (int)by_page.div((uint32_t)p);
            pos[i] = p;
            int page = -1;
            if (col >= 0 && col < a.max_pages) {
                if (col < have) {
                    page = a.table[b * a.table_stride + col];
                } else {
                    const int f = off[b] + col - have;
                    if (f >= 0 && f < avail) page = ld_in(a.free_pages + head + f);
                }
            }
            if (page >= 0) slot[i] = (long long)page * a.page + (p - col * a.page);
        }
        if (vec && t0 + kTok <= a.max_new) {
            *reinterpret_cast<int4 *>(a.positions + t0) = make_int4(pos[0], pos[1], pos[2], pos[3]);
            *reinterpret_cast<longlong2 *>(a.slots + t0) = make_longlong2(slot[0], slot[1]);
            *reinterpret_cast<longlong2 *>(a.slots + t0 + 2) = make_longlong2(slot[2], slot[3]);
        } else {
#pragma unroll
            for (int i = 0; i < kTok; ++i)
                if (t0 + i < a.max_new) a.positions[t0 + i] = pos[i], a.slots[t0 + i] = slot[i];
        }
    }
}

}  // namespace

cudaError_t launch_kv_plan(const KvPlanArgs &a, cudaStream_t s) {
    const size_t smem = 2 * sizeof(int) * ((size_t)a.n_req + 1);
    if (smem > 47 * 1024) {
        const cudaError_t ce = cudaFuncSetAttribute(kv_plan_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                                    2 * sizeof(int) * (MOE_MAX_REQUESTS + 1));
        if (ce != cudaSuccess) return ce;
    }
    const int64_t per = (int64_t)kThreads * kTok;
    int64_t grid = (a.max_new + per - 1) / per;
    grid = grid < 1 ? 1 : grid > 304 ? 304 : grid;
    FastDiv by_page((uint32_t)a.page);
    void *args[] = {const_cast<KvPlanArgs *>(&a), &by_page};
    return launch_after(reinterpret_cast<const void *>(kv_plan_kernel), (int)grid, kThreads, smem, s, args);
}

}  // namespace moe
