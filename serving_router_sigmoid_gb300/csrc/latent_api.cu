// latent_api.cu -- the C ABI of the FP8 products and the latent attention:
// argument checks, the handle, and the launches.
#include <cmath>
#include <cstring>
#include <new>

#include "latent_args.cuh"

using moe::cuda_fail;
using moe::fail;
using moe::LatentHandle;

namespace {

constexpr uint32_t kLatentMagic = 0x4d6f4c61u;  // handle tag
constexpr int kMaxInner = 65536;
constexpr int kMaxOuter = 1 << 20;
constexpr int kMaxPage = 65536;
constexpr int kMaxHeads = 1024;
constexpr float kMaxScale = 1.3292280e36f;  // 2^120: times log2(e) it stays finite

bool aligned(const void *p, size_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }
bool is_act(int t) { return t == MOE_F32 || t == MOE_F16 || t == MOE_BF16; }
bool is_half(int t) { return t == MOE_F16 || t == MOE_BF16; }

// The bytes from the first to behind the last element of a strided array.
struct Span {
    const void *p;
    int64_t n;
    bool meets(const Span &o) const {
        const uintptr_t a = reinterpret_cast<uintptr_t>(p), b = reinterpret_cast<uintptr_t>(o.p);
        return n > 0 && o.n > 0 && a < b + (uintptr_t)o.n && b < a + (uintptr_t)n;
    }
};
// n * stride, both from 0; what no address space holds stays at 2^60
int64_t reach(int64_t n, int64_t stride) { return stride > 0 && n > (1ll << 60) / stride ? 1ll << 60 : n * stride; }
// rows of `row` bytes, `stride` bytes apart
Span rows(const void *p, int64_t n, int64_t stride, int64_t row) { return {p, n > 0 ? reach(n - 1, stride) + row : 0}; }
// [n1][n2] rows of two-byte elements
Span rows2(const void *p, int64_t n1, int64_t s1, int64_t n2, int64_t s2, int64_t dim) {
    return rows(p, n1, 2 * s1, reach(n2 - 1, 2 * s2) + 2 * dim);
}
// Whether those rows are apart from each other.
bool apart(int64_t n1, int64_t s1, int64_t n2, int64_t s2, int64_t dim) {
    const auto nested = [&](int64_t no, int64_t so, int64_t ni, int64_t si) {
        return (ni <= 1 || si >= dim) && (no <= 1 || so >= reach(ni - 1, si) + dim);
    };
    return nested(n1, s1, n2, s2) || nested(n2, s2, n1, s1);
}

}  // namespace

extern "C" {

int moe_quant_act_fp8(const void *x, int act_type, int64_t x_stride, int n_tokens, int dim, uint8_t *x8,
                      int64_t x8_stride, float *scale, cudaStream_t stream) {
    if (n_tokens < 0 || dim < 16 || dim > kMaxInner || dim % 16)
        return fail(MOE_ERR_SHAPE, "n_tokens=%d dim=%d: need n_tokens >= 0 and a multiple of 16 in 16..%d", n_tokens,
                    dim, kMaxInner);
    if (!is_act(act_type)) return fail(MOE_ERR_INVALID_ARG, "act_type=%d", act_type);
    const int64_t ae = (int64_t)moe::dtype_bytes(act_type);
    if (n_tokens > 1 && (x_stride < 0 || x_stride > (1ll << 40) || x8_stride < dim || x8_stride > (1ll << 40)))
        return fail(MOE_ERR_SHAPE, "x_stride=%lld x8_stride=%lld: need 0 <= x_stride and dim <= x8_stride, below 2^40",
                    (long long)x_stride, (long long)x8_stride);
    if (n_tokens == 0) return MOE_OK;
    if (!x || !x8 || !scale) return fail(MOE_ERR_INVALID_ARG, "NULL pointer");
    if (!aligned(x, 16) || !aligned(x8, 16) || !aligned(scale, 4) ||
        (n_tokens > 1 && (x_stride * ae % 16 || x8_stride % 16)))
        return fail(MOE_ERR_INVALID_ARG, "rows of x and x8 must start on 16 bytes");
    const Span in = rows(x, n_tokens, x_stride * ae, dim * ae), codes = rows(x8, n_tokens, x8_stride, dim),
               sc = {scale, 4ll * n_tokens * ((dim + 127) / 128)};
    if (in.meets(codes) || in.meets(sc) || codes.meets(sc))
        return fail(MOE_ERR_INVALID_ARG, "an output overlaps x or the other output");
    const cudaError_t e = moe::launch_quant_act_fp8(x, act_type, x_stride, n_tokens, dim, x8, x8_stride, scale, stream);
    return e == cudaSuccess ? MOE_OK : cuda_fail(e, "quant_act_fp8 launch");
}

int moe_fp8_linear(const MoeFp8LinearArgs *p, cudaStream_t stream) {
    if (!p) return fail(MOE_ERR_INVALID_ARG, "args is NULL");
    const MoeFp8LinearArgs &a = *p;
    if (a.n_tokens < 0 || a.n_tokens > (1 << 24) || a.n_in < 16 || a.n_in > kMaxInner || a.n_in % 16 || a.n_out < 1 ||
        a.n_out > kMaxOuter)
        return fail(MOE_ERR_SHAPE, "n_tokens=%d n_in=%d n_out=%d: need 0..2^24, a multiple of 16 in 16..%d, 1..%d",
                    a.n_tokens, a.n_in, a.n_out, kMaxInner, kMaxOuter);
    if (!is_act(a.out_type)) return fail(MOE_ERR_INVALID_ARG, "out_type=%d", a.out_type);
    if ((int64_t)a.n_tokens * a.n_out > 1ll << 40) return fail(MOE_ERR_SHAPE, "n_tokens * n_out must stay within 2^40");
    if (a.n_tokens == 0) return MOE_OK;
    const int64_t most = 1ll << 38, oe = (int64_t)moe::dtype_bytes(a.out_type);
    if ((a.n_tokens > 1 && (a.x_stride < a.n_in || a.x_stride >= most || a.out_stride < a.n_out || a.out_stride >= most)) ||
        (a.n_out > 1 && (a.w_stride < a.n_in || a.w_stride >= most)))
        return fail(MOE_ERR_SHAPE, "rows may not overlap, strides must stay below 2^38");
    if (!a.x8 || !a.x_scale || !a.w8 || !a.w_scale || !a.out) return fail(MOE_ERR_INVALID_ARG, "NULL pointer");
    if (!aligned(a.x8, 16) || !aligned(a.w8, 16) || (a.n_tokens > 1 && a.x_stride % 16) ||
        (a.n_out > 1 && a.w_stride % 16))
        return fail(MOE_ERR_INVALID_ARG, "rows of x8 and w8 must start on 16 bytes");
    if (!aligned(a.x_scale, 4) || !aligned(a.w_scale, 4) || !aligned(a.out, (size_t)oe))
        return fail(MOE_ERR_INVALID_ARG, "misaligned pointer");
    const int64_t nb = (a.n_in + 127) / 128;
    const Span out = rows(a.out, a.n_tokens, a.out_stride * oe, a.n_out * oe);
    const Span in[] = {rows(a.x8, a.n_tokens, a.x_stride, a.n_in), rows(a.w8, a.n_out, a.w_stride, a.n_in),
                       {a.x_scale, 4 * nb * a.n_tokens}, {a.w_scale, 4 * nb * ((a.n_out + 127) / 128)}};
    for (const Span &i : in)
        if (out.meets(i)) return fail(MOE_ERR_INVALID_ARG, "out overlaps an input");
    const cudaError_t e = moe::launch_fp8_linear(a, stream);
    return e == cudaSuccess ? MOE_OK : cuda_fail(e, "fp8_linear launch");
}

int moe_latent_create(const MoeLatentDesc *d, void **handle_out) {
    if (!d || !handle_out) return fail(MOE_ERR_INVALID_ARG, "NULL pointer");
    *handle_out = nullptr;
    if (d->max_requests < 1 || d->max_requests > MOE_MAX_REQUESTS)
        return fail(MOE_ERR_SHAPE, "max_requests=%d: need 1..%d", d->max_requests, MOE_MAX_REQUESTS);
    if (d->n_heads < 1 || d->n_heads > kMaxHeads)
        return fail(MOE_ERR_SHAPE, "n_heads=%d: need 1..%d", d->n_heads, kMaxHeads);
    if (d->latent_dim < 64 || d->latent_dim > 512 || d->latent_dim % 64 || d->rope_dim < 0 || d->rope_dim > 64 ||
        d->rope_dim % 16)
        return fail(MOE_ERR_SHAPE, "latent_dim=%d rope_dim=%d: need a multiple of 64 in 64..512, of 16 in 0..64",
                    d->latent_dim, d->rope_dim);
    LatentHandle *h = new (std::nothrow) LatentHandle();
    if (!h) return fail(MOE_ERR_NOMEM, "host allocation failed");
    std::memset(h, 0, sizeof *h);
    h->d = *d;
    size_t bytes = 0;
    cudaError_t ce = cudaGetDevice(&h->device);
    if (ce == cudaSuccess) ce = cudaDeviceGetAttribute(&h->num_sms, cudaDevAttrMultiProcessorCount, h->device);
    if (ce == cudaSuccess) ce = moe::latent_prepare(*d, h->num_sms, &bytes);
    if (ce != cudaSuccess) {
        delete h;
        return cuda_fail(ce, "device query");
    }
    if ((ce = cudaMalloc(&h->part, bytes)) != cudaSuccess) {
        cudaGetLastError();
        delete h;
        return fail(MOE_ERR_NOMEM, "workspace of %zu bytes: %s", bytes, cudaGetErrorString(ce));
    }
    ce = cudaMemset(h->part, 0xff, bytes);  // no request is split before the first call says so
    if (ce == cudaSuccess) ce = cudaDeviceSynchronize();
    if (ce != cudaSuccess) {
        cudaFree(h->part);
        delete h;
        return cuda_fail(ce, "handle initialisation");
    }
    h->magic = kLatentMagic;
    *handle_out = h;
    return MOE_OK;
}

int moe_latent_destroy(void *handle) {
    if (!handle) return MOE_OK;
    LatentHandle *h = static_cast<LatentHandle *>(handle);
    if (h->magic != kLatentMagic) return fail(MOE_ERR_INVALID_ARG, "invalid handle");
    int dev = h->device;
    cudaGetDevice(&dev);
    if (dev != h->device) cudaSetDevice(h->device);  // its device is the one to wait for
    const cudaError_t ce = cudaDeviceSynchronize();
    cudaFree(h->part);
    if (dev != h->device) cudaSetDevice(dev);
    h->magic = 0;
    delete h;
    return ce == cudaSuccess ? MOE_OK : cuda_fail(ce, "destroy");
}

int moe_latent_decode(void *handle, const MoeLatentArgs *p, cudaStream_t stream) {
    LatentHandle *h = static_cast<LatentHandle *>(handle);
    if (!h || h->magic != kLatentMagic) return fail(MOE_ERR_INVALID_ARG, "invalid handle");
    if (!p) return fail(MOE_ERR_INVALID_ARG, "args is NULL");
    const MoeLatentArgs &a = *p;
    if (a.n_requests < 0 || a.n_requests > h->d.max_requests)
        return fail(MOE_ERR_SHAPE, "n_requests=%d outside [0, max_requests=%d]", a.n_requests, h->d.max_requests);
    if (a.page_size < 1 || a.page_size > kMaxPage)
        return fail(MOE_ERR_SHAPE, "page_size=%d: need 1 <= page_size <= %d", a.page_size, kMaxPage);
    if (a.max_pages < 0 || a.n_pages < 0 || a.n_pages > INT32_MAX)
        return fail(MOE_ERR_SHAPE, "max_pages=%d n_pages=%lld out of range", a.max_pages, (long long)a.n_pages);
    const int64_t row = (int64_t)a.max_pages * a.page_size;
    if (row > INT32_MAX - 64) return fail(MOE_ERR_SHAPE, "max_pages * page_size must stay below 2^31 - 64");
    if (row * a.n_requests >= 1ll << 36)
        return fail(MOE_ERR_SHAPE, "n_requests * max_pages * page_size must stay below 2^36");
    if (a.n_requests > 1 && a.table_stride < a.max_pages)
        return fail(MOE_ERR_SHAPE, "table_stride=%lld is below max_pages=%d", (long long)a.table_stride, a.max_pages);
    if (!is_half(a.act_type) || (a.cache_type != a.act_type && a.cache_type != MOE_E4M3))
        return fail(MOE_ERR_INVALID_ARG, "act_type=%d cache_type=%d: need F16 or BF16, and the same or E4M3",
                    a.act_type, a.cache_type);
    if (!(a.k_scale > 0) || !std::isfinite(a.k_scale) || !(std::fabs(a.scale * a.k_scale) <= kMaxScale))
        return fail(MOE_ERR_INVALID_ARG, "k_scale must be positive, |scale * k_scale| at most 2^120");
    if (a.cache_type != MOE_E4M3 && a.k_scale != 1.f)
        return fail(MOE_ERR_INVALID_ARG, "k_scale belongs to E4M3 caches");
    if (a.n_requests == 0) return MOE_OK;
    if (!a.seq_len || !a.q || !a.out || (a.max_pages > 0 && !a.block_table) || (a.n_pages > 0 && !a.cache))
        return fail(MOE_ERR_INVALID_ARG, "NULL pointer");
    if (!aligned(a.out, 2) || !aligned(a.seq_len, 4) || !aligned(a.block_table, 4) || !aligned(a.lse, 4))
        return fail(MOE_ERR_INVALID_ARG, "misaligned pointer");
    const int64_t ce = (int64_t)moe::dtype_bytes(a.cache_type);
    if (!aligned(a.q, 16) || a.q_stride_b % 8 || a.q_stride_h % 8)
        return fail(MOE_ERR_INVALID_ARG, "rows of q must start on 16 bytes");
    if (!aligned(a.cache, 16) || a.c_stride_page * ce % 16 || a.c_stride_tok * ce % 16)
        return fail(MOE_ERR_INVALID_ARG, "cache rows must start on 16 bytes");
    for (int64_t st : {a.c_stride_page, a.c_stride_tok})
        if (st < 0 || st > INT32_MAX / ce) return fail(MOE_ERR_SHAPE, "cache strides must lie in [0, 2^31) bytes");
    for (int64_t st : {a.q_stride_b, a.q_stride_h, a.out_stride_b, a.out_stride_h})
        if (st < 0 || st >= 1ll << 37) return fail(MOE_ERR_SHAPE, "strides of q and out must lie in [0, 2^38) bytes");
    const int64_t n = a.n_requests, dim = h->d.latent_dim + h->d.rope_dim;
    if (!apart(n, a.out_stride_b, h->d.n_heads, a.out_stride_h, h->d.latent_dim))
        return fail(MOE_ERR_INVALID_ARG, "rows of out overlap");
    const Span out = rows2(a.out, n, a.out_stride_b, h->d.n_heads, a.out_stride_h, h->d.latent_dim),
               lse = {a.lse, a.lse ? 4 * n * h->d.n_heads : 0};
    const Span in[] = {rows2(a.q, n, a.q_stride_b, h->d.n_heads, a.q_stride_h, dim),
                       rows(a.cache, a.n_pages, a.c_stride_page * ce, (a.page_size - 1) * a.c_stride_tok * ce + dim * ce),
                       rows(a.block_table, a.max_pages ? n : 0, 4 * a.table_stride, 4ll * a.max_pages), {a.seq_len, 4 * n}};
    for (const Span &i : in)
        if (out.meets(i) || lse.meets(i)) return fail(MOE_ERR_INVALID_ARG, "an output overlaps an input");
    if (out.meets(lse)) return fail(MOE_ERR_INVALID_ARG, "out and lse overlap");
    int dev = -1;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return cuda_fail(e, "cudaGetDevice");
    if (dev != h->device)
        return fail(MOE_ERR_INVALID_ARG, "current device %d is not the handle's device %d", dev, h->device);
    e = moe::launch_latent_decode(*h, a, stream);
    return e == cudaSuccess ? MOE_OK : cuda_fail(e, "latent_decode launch");
}

int moe_latent_prompt(const MoePromptArgs *p, cudaStream_t stream) {
    if (!p) return fail(MOE_ERR_INVALID_ARG, "args is NULL");
    const MoePromptArgs &a = *p;
    if (a.n_requests < 0 || a.n_requests > MOE_MAX_REQUESTS || a.n_heads < 1 || a.n_heads > kMaxHeads)
        return fail(MOE_ERR_SHAPE, "n_requests=%d n_heads=%d: need 0..%d and 1..%d", a.n_requests, a.n_heads,
                    MOE_MAX_REQUESTS, kMaxHeads);
    if (a.n_queries < 0 || a.n_keys < 0 || a.n_queries > INT32_MAX - 256 || a.n_keys > INT32_MAX - 256)
        return fail(MOE_ERR_SHAPE, "n_queries=%d n_keys=%d: need 0 <= n < 2^31 - 256", a.n_queries, a.n_keys);
    if (a.nope_dim < 16 || a.nope_dim % 16 || a.rope_dim < 0 || a.rope_dim > 64 || a.rope_dim % 16 ||
        a.nope_dim + a.rope_dim > 256 || a.v_dim < 16 || a.v_dim > 256 || a.v_dim % 16)
        return fail(MOE_ERR_SHAPE, "nope_dim=%d rope_dim=%d v_dim=%d: need multiples of 16, rope_dim <= 64, "
                    "nope_dim + rope_dim and v_dim <= 256", a.nope_dim, a.rope_dim, a.v_dim);
    if (!is_half(a.act_type)) return fail(MOE_ERR_INVALID_ARG, "act_type=%d: need F16 or BF16", a.act_type);
    if (!(std::fabs(a.scale) <= kMaxScale)) return fail(MOE_ERR_INVALID_ARG, "|scale| must be at most 2^120");
    if (a.n_requests == 0 || a.n_queries == 0) return MOE_OK;
    if (!a.q_start || !a.kv_start || !a.q || !a.out ||
        (a.n_keys > 0 && (!a.k || !a.v || (a.rope_dim > 0 && !a.k_rope))))
        return fail(MOE_ERR_INVALID_ARG, "NULL pointer");
    if (!aligned(a.q_start, 4) || !aligned(a.kv_start, 4) || !aligned(a.lse, 4) || !aligned(a.out, 2))
        return fail(MOE_ERR_INVALID_ARG, "misaligned pointer");
    for (int64_t st : {a.q_stride_t, a.q_stride_h, a.k_stride_t, a.k_stride_h, a.kr_stride_t, a.v_stride_t, a.v_stride_h})
        if (st < 0 || st >= 1ll << 37 || st % 8)
            return fail(MOE_ERR_INVALID_ARG, "rows of q, k, k_rope and v must start on 16 bytes, strides below 2^38 bytes");
    if ((a.n_queries > 1 && a.q_stride_t == 0) ||
        (a.n_keys > 1 && (a.k_stride_t == 0 || a.v_stride_t == 0 || (a.rope_dim > 0 && a.kr_stride_t == 0))))
        return fail(MOE_ERR_INVALID_ARG, "tokens of q, k, k_rope and v have rows of their own");
    for (int64_t st : {a.out_stride_t, a.out_stride_h})
        if (st < 0 || st >= 1ll << 37) return fail(MOE_ERR_INVALID_ARG, "out strides must lie in [0, 2^38) bytes");
    if (!aligned(a.q, 16) || !aligned(a.k, 16) || !aligned(a.v, 16) || (a.rope_dim > 0 && !aligned(a.k_rope, 16)))
        return fail(MOE_ERR_INVALID_ARG, "rows of q, k, k_rope and v must start on 16 bytes");
    if (!apart(a.n_queries, a.out_stride_t, a.n_heads, a.out_stride_h, a.v_dim))
        return fail(MOE_ERR_INVALID_ARG, "rows of out overlap");
    const auto span = [&](const void *q, int64_t n, int64_t st, int64_t sh, int64_t dim) {
        return rows2(q, n, st, a.n_heads, sh, dim);
    };
    const Span out = span(a.out, a.n_queries, a.out_stride_t, a.out_stride_h, a.v_dim);
    const Span lse = {a.lse, a.lse ? 4ll * a.n_queries * a.n_heads : 0};
    const Span in[] = {span(a.q, a.n_queries, a.q_stride_t, a.q_stride_h, a.nope_dim + a.rope_dim),
                       span(a.k, a.n_keys, a.k_stride_t, a.k_stride_h, a.nope_dim),
                       span(a.v, a.n_keys, a.v_stride_t, a.v_stride_h, a.v_dim),
                       rows(a.k_rope, a.rope_dim ? a.n_keys : 0, 2 * a.kr_stride_t, 2 * a.rope_dim),
                       {a.q_start, 4ll * (a.n_requests + 1)}, {a.kv_start, 4ll * (a.n_requests + 1)}};
    for (const Span &i : in)
        if (out.meets(i) || lse.meets(i)) return fail(MOE_ERR_INVALID_ARG, "an output overlaps an input");
    if (out.meets(lse)) return fail(MOE_ERR_INVALID_ARG, "out and lse overlap");
    const cudaError_t e = moe::launch_latent_prompt(a, stream);
    return e == cudaSuccess ? MOE_OK : cuda_fail(e, "latent_prompt launch");
}

int moe_dense_status(cudaStream_t stream, int *status_out) {
    if (!status_out) return fail(MOE_ERR_INVALID_ARG, "status_out is NULL");
    *status_out = 0;
    cudaError_t e = cudaStreamSynchronize(stream);
    for (const auto flags : {moe::fp8_linear_flags, moe::latent_decode_flags, moe::latent_prompt_flags}) {
        int32_t v = 0;
        if (e == cudaSuccess) e = flags(&v);
        *status_out |= v;
    }
    if (e != cudaSuccess) return cuda_fail(e, "dense_status");
    return *status_out ? fail(MOE_ERR_DEVICE, "device flags %d", *status_out) : MOE_OK;
}

}  // extern "C"
