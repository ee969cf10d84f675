// k_attn.cu -- launch of the paged-cache attention (moe_attn_decode): the
// kernel's form by sizes and types, its attributes and its parameters.
#include "attn_dev.cuh"

namespace moe {
namespace {

attn::Form form_of(const MoeAttnDesc &d, int cache_type, bool wide) {
    const int dim = d.k_dim > d.v_dim ? d.k_dim : d.v_dim, group = d.n_heads / d.n_kv_heads;
    switch (cache_type) {
        case MOE_F16: return attn::pick_f16(dim, group, wide);
        case MOE_BF16: return attn::pick_bf16(dim, group, wide);
        default: return attn::pick_e4m3(dim, group, wide);
    }
}

}  // namespace

// Floats of the pieces of a block, over all forms of a handle, and head groups.
cudaError_t attn_prepare(const MoeAttnDesc &d, size_t *block_floats, int *groups) {
    *block_floats = 0;
    *groups = 0;
    for (int ct : {MOE_F16, MOE_BF16, MOE_E4M3})
        for (bool wide : {false, true}) {
            const attn::Form f = form_of(d, ct, wide);
            const cudaError_t ce = cudaFuncSetAttribute(reinterpret_cast<const void *>(f.fn),
                                                        cudaFuncAttributeMaxDynamicSharedMemorySize,
                                                        (int)f.smem);
            if (ce != cudaSuccess) return ce;
            const int per = (d.n_heads / d.n_kv_heads + f.rows - 1) / f.rows;
            const size_t n = 2 * (size_t)f.piece;
            if (n > *block_floats) *block_floats = n;
            if (d.n_kv_heads * per > *groups) *groups = d.n_kv_heads * per;
        }
    return cudaSuccess;
}

// The line of all segments' steps is counted in 32 bits.
bool attn_countable(const MoeAttnDesc &d, const MoeAttnArgs &a) {
    const int64_t steps = (int64_t)a.max_pages * a.page_size / 16 + 2 + attn::kSegCost;
    const int64_t groups = d.n_kv_heads * ((d.n_heads / d.n_kv_heads + 7) / 8);
    return steps * a.n_requests <= INT32_MAX / 2 / groups;
}

cudaError_t launch_attn_decode(const AttnHandle &h, const MoeAttnArgs &a, cudaStream_t s) {
    // fp32 queries, and f16 queries on bf16 keys, enter the products in several terms
    const bool wide = a.act_type == MOE_F32 || (a.act_type == MOE_F16 && a.cache_type == MOE_BF16);
    const attn::Form f = form_of(h.d, a.cache_type, wide);
    const int64_t ae = (int64_t)dtype_bytes(a.act_type), ce = (int64_t)dtype_bytes(a.cache_type);
    const auto on16 = [&](const void *p, int64_t s0, int64_t s1) {
        return reinterpret_cast<uintptr_t>(p) % 16 == 0 && s0 * ae % 16 == 0 && s1 * ae % 16 == 0;
    };
    attn::Params p;
    p.a = a;
    p.n_heads = h.d.n_heads;
    p.n_kv = h.d.n_kv_heads;
    p.group = h.d.n_heads / h.d.n_kv_heads;
    p.n_groups = (p.group + f.rows - 1) / f.rows;
    p.k_dim = h.d.k_dim;
    p.v_dim = h.d.v_dim;
    p.q16 = on16(a.q, a.q_stride_b, a.q_stride_h);
    p.out16 = on16(a.out, a.out_stride_b, a.out_stride_h);
    p.by16 = a.page_size % 16 == 0;
    p.n_pages = (uint32_t)a.n_pages;
    p.k_page = (int)(a.kc_stride_page * ce);
    p.k_tok = (int)(a.kc_stride_tok * ce);
    p.k_head = (int)(a.kc_stride_head * ce);
    p.v_page = (int)(a.vc_stride_page * ce);
    p.v_tok = (int)(a.vc_stride_tok * ce);
    p.v_head = (int)(a.vc_stride_head * ce);
    p.by_page = FastDiv((uint32_t)a.page_size);
    p.part = h.part;
    p.arrived = h.arrived;
    p.by_hg = FastDiv((uint32_t)(p.n_kv * p.n_groups));
    void *args[] = {&p};
    return launch_after(reinterpret_cast<const void *>(f.fn), h.num_sms, f.threads, f.smem, s, args);
}

}  // namespace moe
