// k_attn_bf16.cu -- the attention kernel's forms for BF16 caches.
#include "attn_dev.cuh"

namespace moe {
namespace attn {

Form pick_bf16(int dim, int group, bool wide) { return pick<MOE_BF16>(dim, group, wide); }

}  // namespace attn
}  // namespace moe
