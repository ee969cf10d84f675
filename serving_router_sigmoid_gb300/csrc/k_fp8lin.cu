// k_fp8lin.cu -- product of E4M3 activations and an E4M3 matrix, both with fp32
// scales of 128-blocks (moe_fp8_linear), on the fifth-generation tensor cores:
//   out[t, o] = sum_b xs[t, b] ws[o / 128, b] sum_{i in b} x8[t, i] w8[o, i]
//
// A block of 128 inputs is one stage: 128 bytes of each row of both operands by
// TMA (128-byte swizzle) and four tcgen05.mma of 32 bytes of K into a fresh fp32
// accumulator in tensor memory, which the epilogue warps read, scale and add to
// sums in registers while the next block's MMAs run into the other accumulator.
// The scales are fp32, not powers of two, so the tensor cores cannot apply them.
//
// Two orientations:
//  - Few tokens (up to 32): 128 matrix rows on the MMA's M side, the tokens (16 or
//    32) on N.  The matrix streams once; HBM bounds it, and at the smallest the
//    launch.  A stage is 18 or 20 KB, five or six of them let two blocks share an SM.
//    Measured: 1 token, 6144 -> 2048 (12.6 MB) 7.5 us (6.7 with the matrix in L2); 8
//    tokens, 2048 -> 12288 (25 MB) 9.0 (7.4).
//  - More: 128 tokens on M, 128 or 256 matrix rows on N: a thread's sums belong to
//    one token, whose scale is one register, and the matrix scale is one number a
//    block of 128 rows: one FMA an element.  Every accumulator is read from tensor
//    memory once a block of inputs, by up to 16 warps (8 with twice the sums took 117
//    us where these take 112).  Measured: 2048 tokens, 8192 -> 6144: 112 us, 1.84
//    PFLOP/s.  About 750 cycles a block of inputs where the MMAs need 512: operands
//    leave shared memory at 128 bytes a cycle and the reads of the accumulators take
//    tensor-memory cycles from the MMAs.
// Where the tiles do not fill the SMs, a cluster of up to 8 blocks shares a tile's
// contraction; each leaves its sums in its own shared memory and adds up a part of
// the tile from all of them, in rank order, so results do not depend on timing and
// no workspace is needed.
#include <algorithm>

#include "tc_dev.cuh"

namespace moe {
namespace {

using namespace tc;

__device__ int32_t g_err;  // flags since the last read

constexpr int kMaxSplit = 8;  // blocks of a cluster: the portable size

struct Params {
    int n_tokens, n_in, n_out, nb;
    const float *xs, *ws;
    void *out;
    int64_t out_stride;
    int out32;       // rows of out start on 32 bytes
    int tiles_t, tiles_o, split;
};

// TOKM: tokens on M; BN: rows on N.
template <bool TOKM, int BN>
struct Cfg {
    // Epilogue warps, with 64 sums a thread at most: 16 of them read 256 columns of tensor
    // memory in half the time that 8 with 128 sums took (each read is waited for).
    static constexpr int kEpi = TOKM ? BN / 16 : 4;
    static constexpr int kThreads = 128 + 32 * kEpi;
    static constexpr int kCols = TOKM ? 64 : BN;  // of a thread
    static constexpr uint32_t kA = 128 * 128, kB = BN * 128, kStage = kA + kB;
    static constexpr int kStages = TOKM ? (BN == 256 ? 4 : 6) : BN == 16 ? 6 : 5;
    static constexpr uint32_t kTmem = 2 * BN < 32 ? 32 : 2 * BN;  // a power of two
    static constexpr int kAcc = BN;                               // columns of an accumulator
    static constexpr size_t kSmem = kStages * kStage + 1024;
    // the sums of a tile for the cluster: rows of tokens with 4 floats more each (TOKM), else columns of 128
    static constexpr int kPitch = TOKM ? BN + 4 : 128;
    static constexpr size_t kPart = (size_t)(TOKM ? 128 : BN) * kPitch * 4;
    static_assert(kPart <= kStages * kStage, "the sums take the stages' place");
    static_assert(TOKM || BN <= 32, "columns of Shared::sc");
};

struct Shared {
    uint64_t full[8], empty[8], acc_full[2], acc_empty[2], drain;
    uint32_t tmem;
    int abort;
    // few tokens: the scales of a block's columns, by the accumulator they belong to.  Accumulators take
    // turns across tiles too, so a row is written two barriers after the one behind which it was read
    float sc[2][32];
};

template <typename T>
__device__ __forceinline__ void put(T *p, float v) { from_f32(v, *p); }

// N fp32 sums of one row to consecutive outputs.
template <typename T, int N>
__device__ __forceinline__ void put_row(T *p, const float (&v)[N], int n, bool wide) {
    constexpr int kPer = 32 / sizeof(T);
    if (wide && n == N) {
#pragma unroll
        for (int i = 0; i < N; i += kPer) {
            uint32_t w[8];
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                if constexpr (sizeof(T) == 4) w[j] = __float_as_uint(v[i + j]);
                else w[j] = pack_pair(v[i + 2 * j], v[i + 2 * j + 1], T());
            }
            st32(p + i, w);
        }
    } else {
#pragma unroll
        for (int i = 0; i < N; ++i)
            if (i < n) put(p + i, v[i]);
    }
}

// sum[0], sum[1] += (x, y) s: two fp32 FMAs in one instruction, each rounded as by itself
__device__ __forceinline__ void fma2(float *sum, uint32_t x, uint32_t y, float s) {
    asm("{\n .reg .b64 a, b, c;\n mov.b64 a, {%2, %3};\n mov.b64 b, {%4, %4};\n mov.b64 c, {%0, %1};\n fma.rn.f32x2 c, a, b, c;\n"
        " mov.b64 {%0, %1}, c;\n}"
        : "+f"(sum[0]), "+f"(sum[1]) : "r"(x), "r"(y), "f"(s));
}

__device__ __forceinline__ uint32_t map_rank(uint32_t at, int rank) {
    uint32_t r;
    asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(at), "r"(rank));
    return r;
}
__device__ __forceinline__ float4 ld_cluster(uint32_t at) {
    float4 v;
    asm volatile("ld.shared::cluster.v4.f32 {%0,%1,%2,%3}, [%4];" : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w) : "r"(at));
    return v;
}
template <bool TOKM, int BN, typename T>
__global__ void __launch_bounds__(Cfg<TOKM, BN>::kThreads, TOKM ? 1 : 2)
    fp8_linear_kernel(const __grid_constant__ CUtensorMap amap, const __grid_constant__ CUtensorMap bmap, const Params p) {
    using C = Cfg<TOKM, BN>;
    extern __shared__ uint8_t raw[];
    __shared__ Shared sm;
    uint8_t *dyn = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(raw) + 1023) & ~uintptr_t(1023));
    const uint32_t sbase = su32(dyn);
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    volatile int *abort = &sm.abort;

    if (tid == 0) {
        for (int i = 0; i < C::kStages; ++i) {
            mb_init(&sm.full[i], 1);
            mb_init(&sm.empty[i], 1);
        }
        for (int i = 0; i < 2; ++i) {
            mb_init(&sm.acc_full[i], 1);
            mb_init(&sm.acc_empty[i], C::kEpi);
        }
        mb_init(&sm.drain, 1);
        sm.abort = 0;
        mb_init_done();
        tma_prefetch(&amap);
        tma_prefetch(&bmap);
    }
    if (warp == 1) tmem_alloc(&sm.tmem, C::kTmem);
    tc_before_sync();
    __syncthreads();
    tc_after_sync();
    const uint32_t tmem = sm.tmem;
    after_previous();

    // tile: 128 rows of A (mt) by BN rows of B (nt); blocks of K [k0, k1) for this rank
    const int rank = p.split > 1 ? (int)(blockIdx.x % p.split) : 0;
    const int first = (int)(blockIdx.x / p.split), step = (int)(gridDim.x / p.split);
    const int k0 = (int)((int64_t)p.nb * rank / p.split), k1 = (int)((int64_t)p.nb * (rank + 1) / p.split);
    const int n_tiles = p.tiles_t * p.tiles_o;
    const auto tile_at = [&](int i, int &t0, int &o0) {  // tiles of the same matrix rows follow one another
        const int o = i / p.tiles_t, t = i - o * p.tiles_t;
        t0 = t * (TOKM ? 128 : BN);
        o0 = o * (TOKM ? BN : 128);
    };

    if (warp == 0) {
        // ------------------------------------------------------------- TMA
        // A stage is brought by kParts lanes in one instruction, 64 rows of A or what a
        // box of B holds each; the first stages all together.
        constexpr int kBoxB = BN < 128 ? BN : 128, kParts = 2 + BN / kBoxB;
        const auto bring = [&](int part, int slot, int k, int a0, int b0) {
            const uint32_t at = sbase + (uint32_t)slot * C::kStage;
            if (part < 2) tma_2d(at + (uint32_t)part * (C::kA / 2), &amap, k * 128, a0 + 64 * part, &sm.full[slot]);
            else tma_2d(at + C::kA + (uint32_t)(part - 2) * (kBoxB * 128), &bmap, k * 128, b0 + (part - 2) * kBoxB, &sm.full[slot]);
        };
        Ring r;
        int issued = 0;
        bool ok = true;
        for (int i = first; i < n_tiles && ok; i += step) {
            int t0, o0;
            tile_at(i, t0, o0);
            const int a0 = TOKM ? t0 : o0, b0 = TOKM ? o0 : t0;
            int k = k0;
            if (!issued) {
                const int n = min(C::kStages, k1 - k0), slot = lane / kParts;
                static_assert(C::kStages * kParts <= 32, "a lane a part");
                if (lane < n) mb_expect_tx(&sm.full[lane], C::kStage);
                __syncwarp();
                if (slot < n) bring(lane - slot * kParts, slot, k + slot, a0, b0);
                __syncwarp();
                issued = n;
                k += n;
                r.slot = n - 1;
                r.next(C::kStages);
            }
            for (; k < k1; ++k) {
                ok = __all_sync(0xffffffffu, mb_wait(&sm.empty[r.slot], r.phase ^ 1, abort, &g_err));
                if (!ok) break;
                if (lane == 0) mb_expect_tx(&sm.full[r.slot], C::kStage);
                __syncwarp();
                if (lane < kParts) bring(lane, r.slot, k, a0, b0);
                __syncwarp();
                ++issued;
                r.next(C::kStages);
            }
        }
        if (*abort) {  // copies in flight land before the block ends
            const long long t = clock64();
            for (int i = issued > C::kStages ? issued - C::kStages : 0; i < issued; ++i)
                while (!mb_try(&sm.full[i % C::kStages], (uint32_t)((i / C::kStages) & 1)) && clock64() - t < kWaitClk) {}
        }
    } else if (warp == 1) {
        // ------------------------------------------------------------- MMA
        const uint32_t id = idesc(0, 0, 0, 128, BN);
        const uint32_t da = desc(sbase, 16), db = desc(sbase + C::kA, 16);
        const bool lead = elect();
        Ring r, acc;
        bool ok = true;
        for (int i = first; i < n_tiles && ok; i += step)
            for (int k = k0; k < k1; ++k) {
                ok = __all_sync(0xffffffffu, mb_wait(&sm.acc_empty[acc.slot], acc.phase ^ 1, abort, &g_err) &&
                                                 mb_wait(&sm.full[r.slot], r.phase, abort, &g_err));
                if (!ok) break;
                tc_after_sync();
                const uint32_t off = (uint32_t)(r.slot * (int)(C::kStage >> 4)), d = tmem + (uint32_t)(acc.slot * C::kAcc);
                if (lead) {
#pragma unroll
                    for (int j = 0; j < 4; ++j) mma_f8(d, da + off + 2 * j, db + off + 2 * j, id, j != 0);
                    mma_commit(&sm.empty[r.slot]);
                    mma_commit(&sm.acc_full[acc.slot]);
                }
                __syncwarp();
                r.next(C::kStages);
                acc.next(2);
            }
        if (!ok) {  // what was issued ends before the tensor memory is freed
            if (lead) mma_commit(&sm.drain);
            const long long t = clock64();
            while (!mb_try(&sm.drain, 0) && clock64() - t < kWaitClk) {}
        }
        __syncwarp();
    } else if (warp >= 4) {
        // -------------------------------------------------------- epilogue
        const int quad = warp & 3, half = (warp - 4) >> 2;
        const int row = quad * 32 + lane;                  // of A, the thread's
        const uint32_t ta = tmem + ((uint32_t)(quad * 32) << 16) + (uint32_t)(half * C::kCols);
        Ring acc;
        bool ok = true;
        for (int i = first; i < n_tiles && ok; i += step) {
            int t0, o0;
            tile_at(i, t0, o0);
            float sum[C::kCols];
#pragma unroll
            for (int c = 0; c < C::kCols; ++c) sum[c] = 0.f;
            // the scale of this thread's token (TOKM) or of token t0 + (thread index), and that of the matrix block
            const int tok = TOKM ? t0 + row : t0 + (tid & 127);
            const int ob = (o0 + (TOKM ? half * C::kCols : 0)) >> 7;
            const bool has = tok < p.n_tokens && (TOKM || (tid & 127) < BN);
            const float *xs = p.xs + (int64_t)(has ? tok : 0) * p.nb;
            const float *ws = p.ws + (int64_t)(ob * 128 < p.n_out ? ob : 0) * p.nb;
            float nx = k0 < k1 && has ? ld_in(xs + k0) : 0.f, nw = k0 < k1 ? ld_in(ws + k0) : 0.f;
            for (int k = k0; k < k1; ++k) {
                const float s = nx * nw;
                if (k + 1 < k1) {
                    nx = has ? ld_in(xs + k + 1) : 0.f;
                    nw = ld_in(ws + k + 1);
                }
                if (!TOKM) {
                    if ((tid & 127) < BN) sm.sc[acc.slot][tid & 127] = s;
                    asm volatile("bar.sync 1, 128;" ::: "memory");
                }
                if (!mb_wait(&sm.acc_full[acc.slot], acc.phase, abort, &g_err)) ok = false;
                if (__any_sync(0xffffffffu, !ok)) {
                    ok = false;
                    if (TOKM) break;
                }
                tc_after_sync();
                const uint32_t at = ta + (uint32_t)(acc.slot * C::kAcc);
                if constexpr (TOKM) {
#pragma unroll
                    for (int c = 0; c < C::kCols; c += 16) {
                        uint32_t v[16];
                        tmem_ld(at + c, v);
                        tmem_wait_ld();
#pragma unroll
                        for (int j = 0; j < 16; j += 2) fma2(sum + c + j, v[j], v[j + 1], s);
                    }
                } else {
#pragma unroll
                    for (int c = 0; c < C::kCols; c += 16) {
                        uint32_t v[16];
                        tmem_ld(at + c, v);
                        tmem_wait_ld();
#pragma unroll
                        for (int j = 0; j < 16; ++j) sum[c + j] = fmaf(__uint_as_float(v[j]), sm.sc[acc.slot][c + j], sum[c + j]);
                    }
                }
                tc_before_sync();
                __syncwarp();
                if (lane == 0) mb_arrive(&sm.acc_empty[acc.slot]);
                acc.next(2);
            }
            if (p.split == 1) {
                T *out = static_cast<T *>(p.out);
                if (TOKM) {
                    const int c0 = o0 + half * C::kCols;
                    if (tok < p.n_tokens && c0 < p.n_out)
                        put_row(out + (int64_t)tok * p.out_stride + c0, sum, min(C::kCols, p.n_out - c0), p.out32);
                } else if (o0 + row < p.n_out) {
#pragma unroll
                    for (int c = 0; c < C::kCols; ++c)
                        if (t0 + c < p.n_tokens) put(out + (int64_t)(t0 + c) * p.out_stride + o0 + row, sum[c]);
                }
            } else if (ok) {
                // every MMA of this block is done, so the stages are free
                float *part = reinterpret_cast<float *>(dyn);
                if (TOKM) {
#pragma unroll
                    for (int c = 0; c < C::kCols; c += 4)
                        *reinterpret_cast<float4 *>(part + row * C::kPitch + half * C::kCols + c) =
                            make_float4(sum[c], sum[c + 1], sum[c + 2], sum[c + 3]);
                } else {
#pragma unroll
                    for (int c = 0; c < C::kCols; ++c) part[c * C::kPitch + row] = sum[c];
                }
            }
        }
    }

    tc_before_sync();
    __syncthreads();
    tc_after_sync();
    if (warp == 1) tmem_free(tmem, C::kTmem);
    if (p.split > 1) {
        // one tile a cluster; the ranks take turns of 4 neighbouring sums
        cluster_sync();
        int t0, o0;
        tile_at(first, t0, o0);
        T *out = static_cast<T *>(p.out);
        constexpr int kRows = TOKM ? 128 : BN, kPer = TOKM ? BN / 4 : 32;
        for (int i = rank * C::kThreads + tid; i < kRows * kPer; i += p.split * C::kThreads) {
            const int r = i / kPer, c = (i - r * kPer) * 4;
            const int t = t0 + r, o = o0 + c;
            if (t >= p.n_tokens || o >= p.n_out) continue;
            const uint32_t at = sbase + (uint32_t)(r * C::kPitch + c) * 4;
            float s[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
            for (int k = 0; k < 8; ++k) {
                if (k >= p.split) break;
                const float4 v = ld_cluster(map_rank(at, k));
                s[0] += v.x; s[1] += v.y; s[2] += v.z; s[3] += v.w;
            }
#pragma unroll
            for (int j = 0; j < 4; ++j)
                if (o + j < p.n_out) put(out + (int64_t)t * p.out_stride + o + j, s[j]);
        }
        cluster_sync();  // nobody's shared memory goes while others read it
    }
}

template <bool TOKM, int BN, typename T>
cudaError_t launch(const MoeFp8LinearArgs &a, Params p, int dev, int sms, cudaStream_t s) {
    using C = Cfg<TOKM, BN>;
    const int slots = (TOKM ? 1 : 2) * sms;  // blocks that run at once
    p.tiles_t = (a.n_tokens + (TOKM ? 127 : BN - 1)) / (TOKM ? 128 : BN);
    p.tiles_o = (a.n_out + (TOKM ? BN - 1 : 127)) / (TOKM ? BN : 128);
    const int64_t tiles = (int64_t)p.tiles_t * p.tiles_o;
    if (tiles > INT32_MAX / 16) return cudaErrorInvalidValue;
    CUtensorMap tok, mat;
    const int64_t td[3] = {a.n_in, a.n_tokens, 1}, md[3] = {a.n_in, a.n_out, 1};
    const int64_t in16 = (a.n_in + 15) / 16 * 16;
    const int64_t ts[2] = {a.n_tokens > 1 ? a.x_stride : in16, 0}, ms[2] = {a.n_out > 1 ? a.w_stride : in16, 0};
    cudaError_t e = encode_map(&tok, CU_TENSOR_MAP_DATA_TYPE_UINT8, 1, a.x8, 2, td, ts, TOKM ? 64 : BN);
    if (e == cudaSuccess) e = encode_map(&mat, CU_TENSOR_MAP_DATA_TYPE_UINT8, 1, a.w8, 2, md, ms, TOKM ? 128 : 64);
    if (e != cudaSuccess) return e;
    auto fn = fp8_linear_kernel<TOKM, BN, T>;
    static SmemOnce once;
    if ((e = once.allow(reinterpret_cast<const void *>(fn), dev, C::kSmem)) != cudaSuccess) return e;
    cudaLaunchAttribute at[2];
    at[0].id = cudaLaunchAttributeClusterDimension;
    at[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[1].val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t c = {};
    c.blockDim = dim3(C::kThreads);
    c.dynamicSmemBytes = C::kSmem;
    c.stream = s;
    c.attrs = at;
    // As many blocks a tile as find room at once: clusters lie within a GPC, so that of
    // 152 SMs 15 clusters of 8 have one a block; a 16th makes two turns (128 tokens, 6144 ->
    // 2048: 14 us, with 6 blocks a tile 9.4).
    static std::atomic<int> room[kDevices][kMaxSplit + 1];  // clusters of so many blocks, one a SM
    const int per_sm = slots / sms;
    int split = (int)std::min<int64_t>(std::min(kMaxSplit, p.nb), std::max<int64_t>(slots / tiles, 1));
    for (; split > 1; --split) {
        int n = dev < kDevices ? room[dev][split].load(std::memory_order_relaxed) : 0;
        if (n == 0) {
            at[0].val.clusterDim = {(unsigned)split, 1, 1};
            c.gridDim = dim3((unsigned)split);
            c.numAttrs = 1;
            if ((e = cudaOccupancyMaxActiveClusters(&n, fn, &c)) != cudaSuccess) return e;
            n = std::max(std::min(n, sms / split), 1);
            if (dev < kDevices) room[dev][split].store(n, std::memory_order_relaxed);
        }
        if ((int64_t)n * per_sm >= tiles) break;
    }
    p.split = split;
    at[0].val.clusterDim = {(unsigned)split, 1, 1};
    c.gridDim = dim3((unsigned)(split > 1 ? tiles * split : std::min<int64_t>(tiles, slots)));
    c.numAttrs = 2;
    return cudaLaunchKernelEx(&c, fn, TOKM ? tok : mat, TOKM ? mat : tok, p);
}

template <typename T>
cudaError_t pick(const MoeFp8LinearArgs &a, const Params &p, int dev, int sms, cudaStream_t s) {
    // Measured, matrix rows on M and tokens on M: 32 tokens, 6144 -> 2048 7.2 and 7.6 us;
    // 64 tokens, 6144 -> 2048 9.0 and 8.2, 2048 -> 12288 9.6 and 8.4, 8192 -> 6144 17.4 and 14.8
    if (a.n_tokens <= 16) return launch<false, 16, T>(a, p, dev, sms, s);
    if (a.n_tokens <= 32) return launch<false, 32, T>(a, p, dev, sms, s);
    // A tile of 256 rows takes 1.5 times as long as one of 128. Measured, 128 and 256 rows:
    // 300 tokens, 6144 -> 576 9.4 and 12.5 us; 512, 6144 -> 6144 37.1 and 29.1; 1024 54.7 and
    // 55.7; 2048, 8192 -> 6144 141.6 and 111.7
    const int64_t t = (a.n_tokens + 127) / 128, narrow = t * ((a.n_out + 127) / 128), wide = t * ((a.n_out + 255) / 256);
    return 3 * ((wide + sms - 1) / sms) <= 2 * ((narrow + sms - 1) / sms) ? launch<true, 256, T>(a, p, dev, sms, s)
                                                                          : launch<true, 128, T>(a, p, dev, sms, s);
}

}  // namespace

cudaError_t launch_fp8_linear(const MoeFp8LinearArgs &a, cudaStream_t s) {
    int dev = 0, sms = 0;
    cudaError_t e = current_sms(&dev, &sms);
    if (e != cudaSuccess) return e;
    Params p = {};
    p.n_tokens = a.n_tokens;
    p.n_in = a.n_in;
    p.n_out = a.n_out;
    p.nb = (a.n_in + 127) / 128;
    p.xs = a.x_scale;
    p.ws = a.w_scale;
    p.out = a.out;
    p.out_stride = a.out_stride;
    p.out32 = reinterpret_cast<uintptr_t>(a.out) % 32 == 0 && a.out_stride * (int64_t)dtype_bytes(a.out_type) % 32 == 0;
    switch (a.out_type) {
        case MOE_F32: return pick<float>(a, p, dev, sms, s);
        case MOE_F16: return pick<__half>(a, p, dev, sms, s);
        default: return pick<__nv_bfloat16>(a, p, dev, sms, s);
    }
}

cudaError_t fp8_linear_flags(int32_t *out) {
    const int32_t zero = 0;
    cudaError_t e = cudaMemcpyFromSymbol(out, g_err, 4);
    if (e == cudaSuccess && *out) e = cudaMemcpyToSymbol(g_err, &zero, 4);
    return e;
}

}  // namespace moe
