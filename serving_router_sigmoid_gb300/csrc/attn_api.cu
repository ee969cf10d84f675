// attn_api.cu -- the C ABI of the paged-cache operators: argument checks, the
// attention handle, and the launches.
#include <cmath>
#include <cstring>
#include <new>

#include "attn_args.cuh"

using moe::AttnHandle;
using moe::cuda_fail;
using moe::fail;

namespace {

constexpr uint32_t kAttnMagic = 0x4d6f4174u;  // handle tag
constexpr int kMaxPage = 65536;
constexpr int kMaxRopeDim = 512;

bool aligned(const void *p, size_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }
bool is_act(int t) { return t == MOE_F32 || t == MOE_F16 || t == MOE_BF16; }
bool is_cache(int t) { return t == MOE_F16 || t == MOE_BF16 || t == MOE_E4M3; }
bool finite_pos(double v) { return v > 0 && std::isfinite(v); }

// Bytes of an array.
struct Span {
    const void *p;
    size_t n;
    bool meets(const Span &o) const {
        const uintptr_t a = reinterpret_cast<uintptr_t>(p), b = reinterpret_cast<uintptr_t>(o.p);
        return n && o.n && a < b + o.n && b < a + n;
    }
};

// Frequencies theta_i of a rotary description, in 64 bits.
double rope_theta(const MoeRopeDesc &d, int i) {
    double base = d.base;
    if (d.scaling == MOE_ROPE_NTK && d.rot_dim > 2) base *= std::pow(d.factor, d.rot_dim / (d.rot_dim - 2.0));
    double theta = std::pow(base, -2.0 * i / d.rot_dim);
    if (d.scaling == MOE_ROPE_LINEAR) theta /= d.factor;
    if (d.scaling == MOE_ROPE_PARTS) {
        const double turns = d.original_len * theta / (2 * M_PI);
        double keep = (turns - d.beta_slow) / (d.beta_fast - d.beta_slow);
        keep = keep < 0 ? 0 : keep > 1 ? 1 : keep;
        theta *= keep + (1 - keep) / d.factor;
    }
    if (d.scaling == MOE_ROPE_PARTS_INDEX) {
        // the index, a real number, whose pair turns n times in original_len
        const auto index = [&](double n) {
            return d.rot_dim * std::log(d.original_len / (2 * M_PI * n)) / (2 * std::log(d.base));
        };
        const double last = d.rot_dim - 1;
        const double from = std::fmin(std::fmax(std::floor(index(d.beta_fast)), 0), last);
        const double to = std::fmin(std::fmax(std::ceil(index(d.beta_slow)), 0), last);
        double part = to > from ? (i - from) / (to - from) : i > from;
        part = part < 0 ? 0 : part > 1 ? 1 : part;
        theta *= 1 - part + part / d.factor;
    }
    return theta;
}

}  // namespace

extern "C" {

int moe_kv_plan(const int32_t *past_len, const int32_t *new_len, int n_requests, const int32_t *free_pages,
                int n_free, const int32_t *free_head, int page_size, int32_t *block_table, int64_t table_stride,
                int max_pages, int max_new_tokens, int32_t *q_start, int32_t *seq_len, int32_t *positions,
                int64_t *slots, int32_t *info, cudaStream_t stream) {
    if (n_requests < 0 || n_requests > MOE_MAX_REQUESTS)
        return fail(MOE_ERR_SHAPE, "n_requests=%d: need 0 <= n_requests <= %d", n_requests, MOE_MAX_REQUESTS);
    if (page_size < 1 || page_size > kMaxPage)
        return fail(MOE_ERR_SHAPE, "page_size=%d: need 1 <= page_size <= %d", page_size, kMaxPage);
    if (n_free < 0 || max_pages < 0 || max_new_tokens < 0)
        return fail(MOE_ERR_SHAPE, "n_free=%d max_pages=%d max_new_tokens=%d must be >= 0", n_free, max_pages,
                    max_new_tokens);
    if (n_requests > 1 && table_stride < max_pages)
        return fail(MOE_ERR_SHAPE, "table_stride=%lld is below max_pages=%d", (long long)table_stride, max_pages);
    if (!free_head || !q_start || !info) return fail(MOE_ERR_INVALID_ARG, "NULL pointer");
    if (n_requests > 0 && (!past_len || !new_len || !seq_len || (max_pages > 0 && !block_table)))
        return fail(MOE_ERR_INVALID_ARG, "NULL pointer");
    if ((n_free > 0 && !free_pages) || (max_new_tokens > 0 && (!positions || !slots)))
        return fail(MOE_ERR_INVALID_ARG, "NULL pointer");
    // every block reads the inputs while others write the outputs
    const size_t n = (size_t)n_requests;
    const size_t row = max_pages > 0 && n ? (n - 1) * (size_t)table_stride + max_pages : 0;
    const Span in[] = {{past_len, 4 * n}, {new_len, 4 * n}, {free_pages, 4 * (size_t)n_free}, {free_head, 4}};
    const Span out[] = {{q_start, 4 * (n + 1)}, {seq_len, 4 * n}, {positions, 4 * (size_t)max_new_tokens},
                        {slots, 8 * (size_t)max_new_tokens}, {info, 16}, {block_table, 4 * row}};
    for (const Span &o : out) {
        for (const Span &i : in)
            if (o.meets(i)) return fail(MOE_ERR_INVALID_ARG, "an output overlaps an input");
        for (const Span &p : out)
            if (&o != &p && o.meets(p)) return fail(MOE_ERR_INVALID_ARG, "two outputs overlap");
    }
    moe::KvPlanArgs a{past_len, new_len, n_requests, free_pages, n_free, free_head, page_size, block_table,
                      table_stride, max_pages, max_new_tokens, q_start, seq_len, positions, slots, info};
    const cudaError_t ce = moe::launch_kv_plan(a, stream);
    return ce == cudaSuccess ? MOE_OK : cuda_fail(ce, "kv_plan launch");
}

int moe_rope_turns(const MoeRopeDesc *d, uint64_t *turns_host, float *amplitude_host) {
    if (!d || !turns_host || !amplitude_host) return fail(MOE_ERR_INVALID_ARG, "NULL pointer");
    if (d->rot_dim < 2 || d->rot_dim > kMaxRopeDim || d->rot_dim % 2)
        return fail(MOE_ERR_SHAPE, "rot_dim=%d: need an even number in 2..%d", d->rot_dim, kMaxRopeDim);
    if (!finite_pos(d->base)) return fail(MOE_ERR_INVALID_ARG, "base must be positive");
    if (d->scaling < MOE_ROPE_NONE || d->scaling > MOE_ROPE_PARTS_INDEX)
        return fail(MOE_ERR_INVALID_ARG, "unknown scaling %d", d->scaling);
    if (d->scaling != MOE_ROPE_NONE && !(d->factor >= 1 && std::isfinite(d->factor)))
        return fail(MOE_ERR_INVALID_ARG, "factor must be at least 1");
    const bool parts = d->scaling == MOE_ROPE_PARTS || d->scaling == MOE_ROPE_PARTS_INDEX;
    if (parts &&
        (d->original_len < 1 || !(d->beta_fast > d->beta_slow) || !std::isfinite(d->beta_fast - d->beta_slow)))
        return fail(MOE_ERR_INVALID_ARG, "parts scaling needs original_len >= 1 and beta_fast > beta_slow");
    if (d->scaling == MOE_ROPE_PARTS_INDEX && !(d->beta_slow > 0 && d->base > 1))
        return fail(MOE_ERR_INVALID_ARG, "parts scaling by index needs beta_slow > 0 and base > 1");
    for (int i = 0; i < d->rot_dim / 2; ++i) {
        double turns = rope_theta(*d, i) / (2 * M_PI);
        turns -= std::floor(turns);
        const double fixed = std::rint(std::ldexp(turns, 64));
        turns_host[i] = fixed >= 0x1p64 ? 0 : (uint64_t)fixed;
    }
    *amplitude_host = parts ? (float)(0.1 * std::log(d->factor) + 1.0) : 1.f;
    return MOE_OK;
}

int moe_rope_append(const MoeRopeArgs *p, cudaStream_t stream) {
    if (!p) return fail(MOE_ERR_INVALID_ARG, "args is NULL");
    const MoeRopeArgs &a = *p;
    if (a.n_tokens < 0 || a.n_heads < 0 || a.n_kv_heads < 0 || a.n_heads > 4096 || a.n_kv_heads > 4096)
        return fail(MOE_ERR_SHAPE, "n_tokens=%d n_heads=%d n_kv_heads=%d: need 0 <= heads <= 4096", a.n_tokens,
                    a.n_heads, a.n_kv_heads);
    if (a.head_dim < 2 || a.head_dim > kMaxRopeDim || a.v_dim < 0 || a.v_dim > kMaxRopeDim)
        return fail(MOE_ERR_SHAPE, "head_dim=%d v_dim=%d: need 2..%d and 0..%d", a.head_dim, a.v_dim, kMaxRopeDim,
                    kMaxRopeDim);
    if (a.rot_dim < 2 || a.rot_dim % 2 || a.rot_offset < 0 || a.rot_offset > a.head_dim - a.rot_dim)
        return fail(MOE_ERR_SHAPE, "rot_dim=%d rot_offset=%d: need an even part of head_dim=%d", a.rot_dim,
                    a.rot_offset, a.head_dim);
    if (a.page_size < 1 || a.page_size > kMaxPage)
        return fail(MOE_ERR_SHAPE, "page_size=%d: need 1 <= page_size <= %d", a.page_size, kMaxPage);
    if (a.n_pages < 0 || a.n_pages > INT32_MAX) return fail(MOE_ERR_SHAPE, "n_pages out of range");
    if (!is_act(a.act_type) || !is_cache(a.cache_type))
        return fail(MOE_ERR_INVALID_ARG, "act_type=%d cache_type=%d", a.act_type, a.cache_type);
    if (!finite_pos(a.k_scale) || !finite_pos(a.v_scale) || !std::isfinite(a.amplitude))
        return fail(MOE_ERR_INVALID_ARG, "k_scale and v_scale must be positive, amplitude finite");
    if (a.cache_type != MOE_E4M3 && (a.k_scale != 1.f || a.v_scale != 1.f))
        return fail(MOE_ERR_INVALID_ARG, "k_scale and v_scale belong to E4M3 caches");
    if (a.n_tokens == 0 || (a.n_heads == 0 && a.n_kv_heads == 0)) return MOE_OK;
    if (!a.turns || !a.positions || !a.slots) return fail(MOE_ERR_INVALID_ARG, "NULL pointer");
    if (a.n_heads > 0 && (!a.q || !a.q_out)) return fail(MOE_ERR_INVALID_ARG, "q or q_out is NULL");
    if (a.n_kv_heads > 0 && (!a.k || (a.v_dim > 0 && !a.v))) return fail(MOE_ERR_INVALID_ARG, "k or v is NULL");
    if (a.n_kv_heads > 0 && a.n_pages > 0 && (!a.k_cache || (a.v_dim > 0 && !a.v_cache)))
        return fail(MOE_ERR_INVALID_ARG, "k_cache or v_cache is NULL");
    const size_t ae = moe::dtype_bytes(a.act_type), ce = moe::dtype_bytes(a.cache_type);
    if (!aligned(a.q, ae) || !aligned(a.q_out, ae) || !aligned(a.k, ae) || !aligned(a.v, ae) ||
        !aligned(a.k_cache, ce) || !aligned(a.v_cache, ce) || !aligned(a.turns, 8) || !aligned(a.positions, 4) ||
        !aligned(a.slots, 8))
        return fail(MOE_ERR_INVALID_ARG, "misaligned pointer");
    const cudaError_t e = moe::launch_rope_append(a, stream);
    return e == cudaSuccess ? MOE_OK : cuda_fail(e, "rope_append launch");
}

int moe_attn_create(const MoeAttnDesc *d, void **handle_out) {
    if (!d || !handle_out) return fail(MOE_ERR_INVALID_ARG, "NULL pointer");
    *handle_out = nullptr;
    if (d->max_requests < 1 || d->max_requests > MOE_MAX_REQUESTS)
        return fail(MOE_ERR_SHAPE, "max_requests=%d: need 1..%d", d->max_requests, MOE_MAX_REQUESTS);
    if (d->n_kv_heads < 1 || d->n_heads < 1 || d->n_heads > 1024 || d->n_heads % d->n_kv_heads)
        return fail(MOE_ERR_SHAPE, "n_heads=%d n_kv_heads=%d: need a multiple, at most 1024", d->n_heads,
                    d->n_kv_heads);
    for (int v : {d->k_dim, d->v_dim})
        if (v < 8 || v > 256 || v % 8)
            return fail(MOE_ERR_SHAPE, "k_dim=%d v_dim=%d: need multiples of 8 in 8..256", d->k_dim, d->v_dim);
    AttnHandle *h = new (std::nothrow) AttnHandle();
    if (!h) return fail(MOE_ERR_NOMEM, "host allocation failed");
    std::memset(h, 0, sizeof *h);
    h->d = *d;
    cudaError_t ce = cudaGetDevice(&h->device);
    if (ce == cudaSuccess) ce = cudaDeviceGetAttribute(&h->num_sms, cudaDevAttrMultiProcessorCount, h->device);
    if (ce != cudaSuccess) {
        delete h;
        return cuda_fail(ce, "device query");
    }
    size_t piece = 0;
    int groups = 0;
    if ((ce = moe::attn_prepare(*d, &piece, &groups)) != cudaSuccess) {
        delete h;
        return cuda_fail(ce, "kernel attributes");
    }
    // a block's pieces; one arrival counter a request and head group, zero between calls
    const size_t part = sizeof(float) * h->num_sms * piece, cnt = sizeof(int) * (size_t)d->max_requests * groups;
    if ((ce = cudaMalloc(&h->part, part)) != cudaSuccess || (ce = cudaMalloc(&h->arrived, cnt)) != cudaSuccess) {
        cudaGetLastError();
        cudaFree(h->part);
        delete h;
        return fail(MOE_ERR_NOMEM, "workspace of %zu bytes: %s", part + cnt, cudaGetErrorString(ce));
    }
    ce = cudaMemset(h->arrived, 0, cnt);
    if (ce == cudaSuccess) ce = cudaDeviceSynchronize();
    if (ce != cudaSuccess) {
        cudaFree(h->part);
        cudaFree(h->arrived);
        delete h;
        return cuda_fail(ce, "handle initialisation");
    }
    h->magic = kAttnMagic;
    *handle_out = h;
    return MOE_OK;
}

int moe_attn_destroy(void *handle) {
    if (!handle) return MOE_OK;
    AttnHandle *h = static_cast<AttnHandle *>(handle);
    if (h->magic != kAttnMagic) return fail(MOE_ERR_INVALID_ARG, "invalid handle");
    int dev = h->device;
    cudaGetDevice(&dev);
    if (dev != h->device) cudaSetDevice(h->device);  // its device is the one to wait for
    const cudaError_t ce = cudaDeviceSynchronize();
    cudaFree(h->part);
    cudaFree(h->arrived);
    if (dev != h->device) cudaSetDevice(dev);
    h->magic = 0;
    delete h;
    return ce == cudaSuccess ? MOE_OK : cuda_fail(ce, "destroy");
}

int moe_attn_decode(void *handle, const MoeAttnArgs *p, cudaStream_t stream) {
    AttnHandle *h = static_cast<AttnHandle *>(handle);
    if (!h || h->magic != kAttnMagic) return fail(MOE_ERR_INVALID_ARG, "invalid handle");
    if (!p) return fail(MOE_ERR_INVALID_ARG, "args is NULL");
    const MoeAttnArgs &a = *p;
    if (a.n_requests < 0 || a.n_requests > h->d.max_requests)
        return fail(MOE_ERR_SHAPE, "n_requests=%d outside [0, max_requests=%d]", a.n_requests, h->d.max_requests);
    if (a.page_size < 1 || a.page_size > kMaxPage)
        return fail(MOE_ERR_SHAPE, "page_size=%d: need 1 <= page_size <= %d", a.page_size, kMaxPage);
    if (a.max_pages < 0 || a.n_pages < 0 || a.n_pages > INT32_MAX || a.window < 0)
        return fail(MOE_ERR_SHAPE, "max_pages=%d n_pages=%lld window=%d must be >= 0", a.max_pages,
                    (long long)a.n_pages, a.window);
    if ((int64_t)a.max_pages * a.page_size > INT32_MAX - 64)  // a step's end is counted in 32 bits
        return fail(MOE_ERR_SHAPE, "max_pages * page_size must stay below 2^31 - 64");
    if (!moe::attn_countable(h->d, a))
        return fail(MOE_ERR_SHAPE, "n_requests * max_pages * page_size * key heads is beyond 2^34 token heads");
    if (a.n_requests > 1 && a.table_stride < a.max_pages)
        return fail(MOE_ERR_SHAPE, "table_stride=%lld is below max_pages=%d", (long long)a.table_stride, a.max_pages);
    if (!is_act(a.act_type) || !is_cache(a.cache_type))
        return fail(MOE_ERR_INVALID_ARG, "act_type=%d cache_type=%d", a.act_type, a.cache_type);
    if (!std::isfinite(a.scale) || !finite_pos(a.k_scale) || !finite_pos(a.v_scale))
        return fail(MOE_ERR_INVALID_ARG, "scale must be finite, k_scale and v_scale positive");
    if (a.cache_type != MOE_E4M3 && (a.k_scale != 1.f || a.v_scale != 1.f))
        return fail(MOE_ERR_INVALID_ARG, "k_scale and v_scale belong to E4M3 caches");
    const size_t ae = moe::dtype_bytes(a.act_type), ce = moe::dtype_bytes(a.cache_type);
    if (ce == 1 && (h->d.k_dim % 16 || h->d.v_dim % 16))
        return fail(MOE_ERR_SHAPE, "k_dim=%d v_dim=%d: E4M3 caches need multiples of 16", h->d.k_dim, h->d.v_dim);
    if (a.n_requests == 0) return MOE_OK;
    if (!a.seq_len || !a.q || !a.out || (a.max_pages > 0 && !a.block_table) ||
        (a.n_pages > 0 && (!a.k_cache || !a.v_cache)))
        return fail(MOE_ERR_INVALID_ARG, "NULL pointer");
    if (!aligned(a.q, ae) || !aligned(a.out, ae) || !aligned(a.seq_len, 4) || !aligned(a.block_table, 4) ||
        !aligned(a.lse, 4))
        return fail(MOE_ERR_INVALID_ARG, "misaligned pointer");
    const int64_t per16 = 16 / (int64_t)ce;
    if (!aligned(a.k_cache, 16) || !aligned(a.v_cache, 16) || a.kc_stride_page % per16 || a.kc_stride_tok % per16 ||
        a.kc_stride_head % per16 || a.vc_stride_page % per16 || a.vc_stride_tok % per16 || a.vc_stride_head % per16)
        return fail(MOE_ERR_INVALID_ARG, "cache rows must start on 16 bytes");
    for (int64_t st : {a.kc_stride_page, a.kc_stride_tok, a.kc_stride_head, a.vc_stride_page, a.vc_stride_tok,
                       a.vc_stride_head})
        if (st < 0 || st > INT32_MAX / (int64_t)ce)
            return fail(MOE_ERR_SHAPE, "cache strides must lie in [0, 2^31) bytes");
    int dev = -1;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return cuda_fail(e, "cudaGetDevice");
    if (dev != h->device)
        return fail(MOE_ERR_INVALID_ARG, "current device %d is not the handle's device %d", dev, h->device);
    e = moe::launch_attn_decode(*h, a, stream);
    return e == cudaSuccess ? MOE_OK : cuda_fail(e, "attn_decode launch");
}

int moe_block_norm(const MoeNormArgs *p, cudaStream_t stream) {
    if (!p) return fail(MOE_ERR_INVALID_ARG, "args is NULL");
    const MoeNormArgs &a = *p;
    if (a.n_tokens < 0 || a.dim < 1 || a.dim > 16384)
        return fail(MOE_ERR_SHAPE, "n_tokens=%d dim=%d: need n_tokens >= 0 and dim in 1..16384", a.n_tokens, a.dim);
    if (!is_act(a.act_type)) return fail(MOE_ERR_INVALID_ARG, "act_type=%d", a.act_type);
    if (a.gate_stride_d != 0 && a.gate_stride_d != 1)
        return fail(MOE_ERR_SHAPE, "gate_stride_d=%lld: need 0 or 1", (long long)a.gate_stride_d);
    if (!(a.eps >= 0.f) || !std::isfinite(a.eps) || !std::isfinite(a.alpha) || !std::isfinite(a.beta))
        return fail(MOE_ERR_INVALID_ARG, "eps must be >= 0, alpha and beta finite");
    if (a.n_tokens == 0) return MOE_OK;
    if (!a.x || !a.out) return fail(MOE_ERR_INVALID_ARG, "x or out is NULL");
    if (!a.y && (a.w_post || a.gate)) return fail(MOE_ERR_INVALID_ARG, "w_post and gate need y");
    const size_t ae = moe::dtype_bytes(a.act_type);
    if (!aligned(a.x, ae) || !aligned(a.y, ae) || !aligned(a.gate, ae) || !aligned(a.out, ae) ||
        !aligned(a.normed, ae) || !aligned(a.w_post, 4) || !aligned(a.w_pre, 4))
        return fail(MOE_ERR_INVALID_ARG, "misaligned pointer");
    const cudaError_t e = moe::launch_block_norm(a, stream);
    return e == cudaSuccess ? MOE_OK : cuda_fail(e, "block_norm launch");
}

}  // extern "C"
