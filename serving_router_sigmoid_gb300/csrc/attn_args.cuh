// attn_args.cuh -- argument checks, launchers and element conversions shared
// by the paged-cache operators (plan, rotary append, attention, block norm).
// Internal.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_fp8.h>

#include "common.cuh"

namespace moe {

// Unsigned division by a host-known divisor as a multiplication: for n < 2^31
// and 1 <= d < 2^31, n / d = (n * mul) >> (32 + shift) with
// shift = ceil(log2 d) - 1 and mul = ceil(2^(32 + shift) / d) (Granlund and
// Montgomery 1994); d = 1 is flagged by mul = 0.
struct FastDiv {
    uint32_t mul, shift, d;
    __host__ __device__ FastDiv() : mul(0), shift(0), d(1) {}
    explicit FastDiv(uint32_t div) : mul(0), shift(0), d(div) {
        if (div <= 1) return;
        uint32_t l = 0;
        while ((1ull << l) < div) ++l;
        shift = l - 1;
        mul = (uint32_t)(((1ull << (32 + shift)) + div - 1) / div);
    }
    __device__ __forceinline__ uint32_t div(uint32_t n) const { return mul ? __umulhi(n, mul) >> shift : n; }
};

inline size_t dtype_bytes(int t) { return t == MOE_F32 ? 4 : t == MOE_E4M3 ? 1 : 2; }

// Element types as C++ types.
template <int DT> struct Elem;
template <> struct Elem<MOE_F32> { using type = float; };
template <> struct Elem<MOE_F16> { using type = __half; };
template <> struct Elem<MOE_BF16> { using type = __nv_bfloat16; };
template <> struct Elem<MOE_E4M3> { using type = uint8_t; };

__device__ __forceinline__ float to_f32(float v) { return v; }
__device__ __forceinline__ float to_f32(__half v) { return __half2float(v); }
__device__ __forceinline__ float to_f32(__nv_bfloat16 v) { return __bfloat162float(v); }
__device__ __forceinline__ void from_f32(float v, float &o) { o = v; }
__device__ __forceinline__ void from_f32(float v, __half &o) { o = __float2half_rn(v); }
__device__ __forceinline__ void from_f32(float v, __nv_bfloat16 &o) { o = __float2bfloat16_rn(v); }

// lo, hi -> two e4m3 codes (nearest, ties to even, saturating), lo in the low byte.
__device__ __forceinline__ uint32_t f32x2_to_e4m3x2(float lo, float hi) {
    uint32_t r;
    asm("{ .reg .b16 c; cvt.rn.satfinite.e4m3x2.f32 c, %2, %1; cvt.u32.u16 %0, c; }" : "=r"(r) : "f"(lo), "f"(hi));
    return r;
}

// 16 bytes read once: past L1 (not through the read-only path, so that an output
// may take the place of its input).
__device__ __forceinline__ uint4 ld_once16(const void *p) {
    uint4 v;
    asm volatile("ld.global.L1::no_allocate.v4.u32 {%0,%1,%2,%3}, [%4];"
                 : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
                 : "l"(p)
                 : "memory");
    return v;
}

// Loads of a kernel's inputs.  Coherent ones: the kernel before this one may
// have written them while this one was already resident (after_previous), and
// the read-only path (__ldg, ld.global.nc) holds only for what nobody writes in
// a kernel's lifetime.  Volatile, so that none moves above that wait.
__device__ __forceinline__ int32_t ld_in(const int32_t *p) {
    int32_t v;
    asm volatile("ld.global.s32 %0, [%1];" : "=r"(v) : "l"(p));
    return v;
}
__device__ __forceinline__ int64_t ld_in(const int64_t *p) {
    int64_t v;
    asm volatile("ld.global.s64 %0, [%1];" : "=l"(v) : "l"(p));
    return v;
}
__device__ __forceinline__ float ld_in(const float *p) {
    float v;
    asm volatile("ld.global.f32 %0, [%1];" : "=f"(v) : "l"(p));
    return v;
}
__device__ __forceinline__ float4 ld_in4(const float *p) {
    float4 v;
    asm volatile("ld.global.v4.f32 {%0,%1,%2,%3}, [%4];" : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w) : "l"(p));
    return v;
}

// N consecutive elements <-> fp32 registers, in vector accesses of up to 16
// bytes (the caller guarantees the alignment of N elements, at most 16 bytes).
template <int N>
__device__ __forceinline__ void load_vec(const float *p, float (&v)[N]) {
    static_assert(N % 4 == 0, "");
#pragma unroll
    for (int i = 0; i < N; i += 4) {
        const uint4 w = ld_once16(p + i);
        v[i] = __uint_as_float(w.x); v[i + 1] = __uint_as_float(w.y);
        v[i + 2] = __uint_as_float(w.z); v[i + 3] = __uint_as_float(w.w);
    }
}
__device__ __forceinline__ float2 half_pair(uint32_t w, __half) {
    return __half22float2(*reinterpret_cast<const __half2 *>(&w));
}
__device__ __forceinline__ float2 half_pair(uint32_t w, __nv_bfloat16) {
    return make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xFFFF0000u));
}
__device__ __forceinline__ uint32_t pack_pair(float lo, float hi, __half) {
    const __half2 h = __floats2half2_rn(lo, hi);
    return *reinterpret_cast<const uint32_t *>(&h);
}
__device__ __forceinline__ uint32_t pack_pair(float lo, float hi, __nv_bfloat16) {
    const __nv_bfloat162 h = __floats2bfloat162_rn(lo, hi);
    return *reinterpret_cast<const uint32_t *>(&h);
}
template <int N, typename H>
__device__ __forceinline__ void load_vec(const H *p, float (&v)[N]) {
    static_assert(N % 8 == 0, "");
#pragma unroll
    for (int i = 0; i < N; i += 8) {
        const uint4 w = ld_once16(p + i);
        const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const float2 f = half_pair(u[j], H());
            v[i + 2 * j] = f.x; v[i + 2 * j + 1] = f.y;
        }
    }
}
template <int N>
__device__ __forceinline__ void store_vec(float *p, const float (&v)[N]) {
#pragma unroll
    for (int i = 0; i < N; i += 4)
        *reinterpret_cast<float4 *>(p + i) = make_float4(v[i], v[i + 1], v[i + 2], v[i + 3]);
}
template <int N, typename H>
__device__ __forceinline__ void store_vec(H *p, const float (&v)[N]) {
#pragma unroll
    for (int i = 0; i < N; i += 8)
        *reinterpret_cast<uint4 *>(p + i) =
            make_uint4(pack_pair(v[i], v[i + 1], H()), pack_pair(v[i + 2], v[i + 3], H()),
                       pack_pair(v[i + 4], v[i + 5], H()), pack_pair(v[i + 6], v[i + 7], H()));
}
// e4m3 codes: 8 elements in one 8-byte store.
__device__ __forceinline__ void store_vec(uint8_t *p, const float (&v)[8]) {
    const uint32_t a = f32x2_to_e4m3x2(v[0], v[1]) | f32x2_to_e4m3x2(v[2], v[3]) << 16;
    const uint32_t b = f32x2_to_e4m3x2(v[4], v[5]) | f32x2_to_e4m3x2(v[6], v[7]) << 16;
    *reinterpret_cast<uint2 *>(p) = make_uint2(a, b);
}

// The operators of a decode step follow one another in a stream, each a few
// microseconds long: they are launched with programmatic stream serialisation,
// so that a kernel's launch overlaps the one before it, and touch no memory
// before that one is done (1 x 6144 block norm 3.35 -> 2.94 us a call in a row).
__device__ __forceinline__ void after_previous() {
    asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
}
inline cudaError_t launch_after(const void *fn, int grid, int block, size_t smem, cudaStream_t s, void **args) {
    cudaLaunchAttribute at[1];
    at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[0].val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t c = {};
    c.gridDim = dim3(grid);
    c.blockDim = dim3(block);
    c.dynamicSmemBytes = smem;
    c.stream = s;
    c.attrs = at;
    c.numAttrs = 1;
    return cudaLaunchKernelExC(&c, fn, args);
}

// Host launchers (defined in the .cu files).
struct KvPlanArgs {
    const int32_t *past, *fresh;
    int n_req;
    const int32_t *free_pages;
    int n_free;
    const int32_t *free_head;
    int page;
    int32_t *table;
    int64_t table_stride;
    int max_pages, max_new;
    int32_t *q_start, *seq_len, *positions;
    int64_t *slots;
    int32_t *info;
};
cudaError_t launch_kv_plan(const KvPlanArgs &a, cudaStream_t s);
cudaError_t launch_rope_append(const MoeRopeArgs &a, cudaStream_t s);
cudaError_t launch_block_norm(const MoeNormArgs &a, cudaStream_t s);

// What an attention handle holds; part: pieces of the segments that blocks
// share, arrived: how many of a segment's blocks have left theirs (a counter a
// request and head group, zero between calls).
struct AttnHandle {
    uint32_t magic;
    int device, num_sms;
    MoeAttnDesc d;
    float *part;
    int *arrived;
};
cudaError_t attn_prepare(const MoeAttnDesc &d, size_t *block_floats, int *groups);
bool attn_countable(const MoeAttnDesc &d, const MoeAttnArgs &a);
cudaError_t launch_attn_decode(const AttnHandle &h, const MoeAttnArgs &a, cudaStream_t s);

}  // namespace moe
