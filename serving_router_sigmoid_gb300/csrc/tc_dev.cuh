// tc_dev.cuh -- mbarriers, TMA and tcgen05 as used by the FP8 product and the
// latent attention: thin wrappers of the PTX, bounded waits, descriptors.
//
// A tcgen05.mma costs the tensor core N/2 cycles (M = 128, 32 bytes of K a row),
// at least what its operands take from shared memory at 128 bytes a cycle, if its
// issuer keeps up.  Measured: M = 128: N = 256 128 cycles, 128 64, 64 48, 16 39; M
// = 64: N = 64 32; A in tensor memory, N = 64: 32.  An issuer takes some 36 cycles an
// instruction where one branch that one lane takes holds a whole loop of them, up
// to 90 where it holds one.  A commit takes 50; from a commit to a thread that waits
// for its barrier 300 to 440 pass.
#pragma once

#include <atomic>
#include <cuda.h>

#include "latent_args.cuh"

namespace moe {
namespace tc {

__device__ __forceinline__ uint32_t su32(const void *p) { return (uint32_t)__cvta_generic_to_shared(p); }

// One lane of a converged warp.
__device__ __forceinline__ bool elect() {
    uint32_t p;
    asm volatile("{\n .reg .pred p;\n elect.sync _|p, 0xffffffff;\n selp.u32 %0, 1, 0, p;\n}" : "=r"(p));
    return p != 0;
}

// ---------------------------------------------------------------- mbarriers
__device__ __forceinline__ void mb_init(uint64_t *b, int n) {
    asm volatile("mbarrier.init.shared::cta.b64 [%0], %1;" ::"r"(su32(b)), "r"(n));
}
__device__ __forceinline__ void mb_init_done() { asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory"); }
__device__ __forceinline__ void mb_arrive(uint64_t *b) {
    asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(su32(b)) : "memory");
}
__device__ __forceinline__ void mb_expect_tx(uint64_t *b, uint32_t bytes) {
    asm volatile("mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;" ::"r"(su32(b)), "r"(bytes) : "memory");
}
__device__ __forceinline__ bool mb_try(uint64_t *b, uint32_t parity) {
    uint32_t ok;
    asm volatile("{\n .reg .pred p;\n mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\n selp.u32 %0, 1, 0, p;\n}"
                 : "=r"(ok) : "r"(su32(b)), "r"(parity) : "memory");
    return ok != 0;
}
__device__ __forceinline__ bool mb_test(uint64_t *b, uint32_t parity) {  // without waiting
    uint32_t ok;
    asm volatile("{\n .reg .pred p;\n mbarrier.test_wait.parity.shared::cta.b64 p, [%1], %2;\n selp.u32 %0, 1, 0, p;\n}"
                 : "=r"(ok) : "r"(su32(b)), "r"(parity) : "memory");
    return ok != 0;
}
// The same with a hint to sleep in the barrier unit (up to 0.1 ms): a dozen warps
// that spin slow down the one that issues MMAs.
__device__ __forceinline__ bool mb_try_sleep(uint64_t *b, uint32_t parity) {
    uint32_t ok;
    asm volatile("{\n .reg .pred p;\n mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2, %3;\n selp.u32 %0, 1, 0, p;\n}"
                 : "=r"(ok) : "r"(su32(b)), "r"(parity), "r"(100000u) : "memory");
    return ok != 0;
}
// Waits are bounded: a second or more, in cycles (%globaltimer costs about a
// microsecond to read).
constexpr long long kWaitClk = 2'100'000'000ll;
// Bounded wait for the phase with this parity; false on time-out or once another
// thread of the block has given up.  The block then ends with its results
// undefined and `err` set.
static __device__ __noinline__ bool mb_wait_slow(uint64_t *b, uint32_t parity, volatile int *abort, int32_t *err) {
    const long long t0 = clock64();
    for (;;) {
        if (mb_try_sleep(b, parity)) return true;
        if (*abort) return false;
        if (clock64() - t0 > kWaitClk) {
            *abort = 1;
            atomicOr(err, kErrSyncTimeout);
            return false;
        }
    }
}
__device__ __forceinline__ bool mb_wait(uint64_t *b, uint32_t parity, volatile int *abort, int32_t *err) {
    return mb_test(b, parity) || mb_wait_slow(b, parity, abort, err);
}
// Slot and parity of a ring.
struct Ring {
    int slot = 0;
    uint32_t phase = 0;
    __device__ __forceinline__ void next(int n) {
        if (++slot == n) { slot = 0; phase ^= 1; }
    }
};

// ------------------------------------------------------------------- fences
__device__ __forceinline__ void fence_async_smem() { asm volatile("fence.proxy.async.shared::cta;" ::: "memory"); }
__device__ __forceinline__ void tc_before_sync() { asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void tc_after_sync() { asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory"); }

// --------------------------------------------------------------- TMA loads
__device__ __forceinline__ void tma_2d(uint32_t dst, const CUtensorMap *map, int c0, int c1, uint64_t *bar) {
    asm volatile("cp.async.bulk.tensor.2d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3}], [%4];" ::"r"(dst),
                 "l"(reinterpret_cast<uint64_t>(map)), "r"(c0), "r"(c1), "r"(su32(bar))
                 : "memory");
}
__device__ __forceinline__ void tma_3d(uint32_t dst, const CUtensorMap *map, int c0, int c1, int c2, uint64_t *bar) {
    asm volatile("cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4}], [%5];" ::"r"(dst),
                 "l"(reinterpret_cast<uint64_t>(map)), "r"(c0), "r"(c1), "r"(c2), "r"(su32(bar))
                 : "memory");
}
// One thread that issues copies of 16 KB one after another gets 32 to 43 bytes a
// cycle, whatever the map; four lanes of a warp in one instruction, or two warps,
// get 70 to 80 (measured on all SMs, out of L2).
__device__ __forceinline__ void tma_prefetch(const CUtensorMap *map) {
    asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(map)) : "memory");
}

// ------------------------------------------------------------ tensor memory
// A whole warp allocates, and the same warp frees.
__device__ __forceinline__ void tmem_alloc(uint32_t *where, uint32_t cols) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(su32(where)), "r"(cols) : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;");
}
__device__ __forceinline__ void tmem_free(uint32_t at, uint32_t cols) {
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(at), "r"(cols));
}
#define MOE_TC_LD(N, LIST, ...)                                                                             \
    asm volatile("tcgen05.ld.sync.aligned.32x32b.x" #N ".b32 {" LIST "}, [%" #N "];" : __VA_ARGS__ : "r"(at))
__device__ __forceinline__ void tmem_ld(uint32_t at, uint32_t (&v)[16]) {
    MOE_TC_LD(16, "%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15", "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3]),
              "=r"(v[4]), "=r"(v[5]), "=r"(v[6]), "=r"(v[7]), "=r"(v[8]), "=r"(v[9]), "=r"(v[10]), "=r"(v[11]), "=r"(v[12]),
              "=r"(v[13]), "=r"(v[14]), "=r"(v[15]));
}
__device__ __forceinline__ void tmem_ld(uint32_t at, uint32_t (&v)[32]) {
    MOE_TC_LD(32, "%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31",
              "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3]), "=r"(v[4]), "=r"(v[5]), "=r"(v[6]), "=r"(v[7]), "=r"(v[8]),
              "=r"(v[9]), "=r"(v[10]), "=r"(v[11]), "=r"(v[12]), "=r"(v[13]), "=r"(v[14]), "=r"(v[15]), "=r"(v[16]),
              "=r"(v[17]), "=r"(v[18]), "=r"(v[19]), "=r"(v[20]), "=r"(v[21]), "=r"(v[22]), "=r"(v[23]), "=r"(v[24]),
              "=r"(v[25]), "=r"(v[26]), "=r"(v[27]), "=r"(v[28]), "=r"(v[29]), "=r"(v[30]), "=r"(v[31]));
}
#undef MOE_TC_LD
__device__ __forceinline__ void tmem_st(uint32_t at, const uint32_t (&v)[16]) {
    asm volatile("tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};" ::"r"(at),
                 "r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7]), "r"(v[8]), "r"(v[9]),
                 "r"(v[10]), "r"(v[11]), "r"(v[12]), "r"(v[13]), "r"(v[14]), "r"(v[15]));
}
__device__ __forceinline__ void tmem_wait_ld() { asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory"); }
__device__ __forceinline__ void tmem_wait_st() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

// -------------------------------------------------------------------- MMAs
// Shared-memory descriptor with the 128-byte swizzle (atoms of 8 rows of 128
// bytes, 1024-byte aligned).  K-major operands: sbo = distance of 8-row groups,
// lbo unused, and 32 bytes of K step the address by 32 (the descriptor by 2).  MN-major operands (a row
// of the tile holds 64 elements of M or N at one K): lbo = distance of the blocks
// of 64 elements, sbo = distance of groups of 8 K, and 16 K step the address by 2048.  Here sbo is 1024.
// Only the address and lbo vary: the lower half, without carries into the upper.
constexpr uint32_t kDescHi = (1024u >> 4) | (1u << 14) | (2u << 29);  // sbo 1024, 128-byte swizzle
__device__ __forceinline__ uint32_t desc(uint32_t at, uint32_t lbo) { return ((at & 0x3FFFF) >> 4) | ((lbo >> 4) << 16); }
// Byte offset of 16-byte piece c of row r in such a tile.
__device__ __forceinline__ uint32_t sw_off(int r, int c) {
    return (uint32_t)((r >> 3) * 1024 + (r & 7) * 128 + ((c ^ (r & 7)) << 4));
}
// fp32 accumulators; fmt 0: f16 or E4M3, 1: bf16; a_mn, b_mn: MN-major operands.
__host__ __device__ constexpr uint32_t idesc(int fmt, int a_mn, int b_mn, int m, int n) {
    return (1u << 4) | ((uint32_t)fmt << 7) | ((uint32_t)fmt << 10) | ((uint32_t)a_mn << 15) | ((uint32_t)b_mn << 16) |
           ((uint32_t)(n >> 3) << 17) | ((uint32_t)(m >> 4) << 24);
}
// D (+)= A B^T.  One thread issues: inside `if (lead)`, lead from elect().
#define MOE_TC_MMA(NAME, KIND, A, AREG)                                                                       \
    __device__ __forceinline__ void NAME(uint32_t d, uint32_t a, uint32_t b, uint32_t id, uint32_t acc) {     \
        asm volatile("{\n .reg .pred p;\n .reg .b64 x, y;\n setp.ne.u32 p, %5, 0;\n" AREG                    \
                     " mov.b64 y, {%2, %4};\n tcgen05.mma.cta_group::1.kind::" KIND " [%0], " A ", y, %3, p;\n}" ::"r"(d), \
                     "r"(a), "r"(b), "r"(id), "n"(kDescHi), "r"(acc));                                        \
    }
MOE_TC_MMA(mma_f16, "f16", "x", " mov.b64 x, {%1, %4};\n")
MOE_TC_MMA(mma_f16_ta, "f16", "[%1]", "")  // A in tensor memory
MOE_TC_MMA(mma_f8, "f8f6f4", "x", " mov.b64 x, {%1, %4};\n")
#undef MOE_TC_MMA
// The barrier's arrival once all MMAs of this thread so far are done.
__device__ __forceinline__ void mma_commit(uint64_t *b) {
    asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(su32(b)) : "memory");
}

__device__ __forceinline__ void cluster_sync() {
    asm volatile("barrier.cluster.arrive.release;\nbarrier.cluster.wait.acquire;" ::: "memory");
}

// ------------------------------------------------------------------ stores
__device__ __forceinline__ void st32(void *p, const uint32_t (&v)[8]) {  // 32-byte aligned
    asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(p), "r"(v[0]), "r"(v[1]), "r"(v[2]),
                 "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7])
                 : "memory");
}

// ------------------------------------------------- host: devices, kernels
constexpr int kDevices = 64;

// The current device and its SMs (asked for once a device).
inline cudaError_t current_sms(int *dev, int *sms) {
    static std::atomic<int> known[kDevices];
    cudaError_t e = cudaGetDevice(dev);
    if (e != cudaSuccess) return e;
    if (*dev < kDevices && (*sms = known[*dev].load(std::memory_order_relaxed)) > 0) return cudaSuccess;
    e = cudaDeviceGetAttribute(sms, cudaDevAttrMultiProcessorCount, *dev);
    if (e == cudaSuccess && *dev < kDevices) known[*dev].store(*sms, std::memory_order_relaxed);
    return e;
}
// A kernel's dynamic shared memory, allowed once a device.
struct SmemOnce {
    std::atomic<bool> done[kDevices] = {};
    cudaError_t allow(const void *fn, int dev, size_t bytes) {
        if (dev < kDevices && done[dev].load(std::memory_order_relaxed)) return cudaSuccess;
        const cudaError_t e = cudaFuncSetAttribute(fn, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)bytes);
        if (e == cudaSuccess && dev < kDevices) done[dev].store(true, std::memory_order_relaxed);
        return e;
    }
};

// -------------------------------------------------------------- host: maps
using EncodeFn = CUresult (*)(CUtensorMap *, CUtensorMapDataType, cuuint32_t, void *, const cuuint64_t *, const cuuint64_t *,
                              const cuuint32_t *, const cuuint32_t *, CUtensorMapInterleave, CUtensorMapSwizzle,
                              CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

// A map of rows of `cols` elements with the 128-byte swizzle; boxes of 128 bytes
// by box_rows rows (and one of the third dimension); what lies outside reads as
// zeros.  strides in bytes.
inline cudaError_t encode_map(CUtensorMap *map, CUtensorMapDataType type, int elem, const void *base, int rank,
                              const int64_t (&dims)[3], const int64_t (&strides)[2], int box_rows) {
    static EncodeFn fn = [] {
        void *p = nullptr;
        cudaDriverEntryPointQueryResult q = cudaDriverEntryPointSymbolNotFound;
        const cudaError_t e = cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault, &q);
        return e == cudaSuccess && q == cudaDriverEntryPointSuccess ? reinterpret_cast<EncodeFn>(p) : nullptr;
    }();
    if (!fn) return cudaErrorNotSupported;
    const cuuint64_t d[3] = {(cuuint64_t)dims[0], (cuuint64_t)dims[1], (cuuint64_t)dims[2]};
    const cuuint64_t s[2] = {(cuuint64_t)strides[0], (cuuint64_t)strides[1]};
    const cuuint32_t box[3] = {(cuuint32_t)(128 / elem), (cuuint32_t)box_rows, 1u}, one[3] = {1, 1, 1};
    const CUresult r = fn(map, type, (cuuint32_t)rank, const_cast<void *>(base), d, s, box, one, CU_TENSOR_MAP_INTERLEAVE_NONE,
                          CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    return r == CUDA_SUCCESS ? cudaSuccess : cudaErrorInvalidValue;
}

}  // namespace tc
}  // namespace moe
