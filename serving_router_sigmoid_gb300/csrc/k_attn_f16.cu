// k_attn_f16.cu -- the attention kernel's forms for F16 caches.
#include "attn_dev.cuh"

namespace moe {
namespace attn {

Form pick_f16(int dim, int group, bool wide) { return pick<MOE_F16>(dim, group, wide); }

}  // namespace attn
}  // namespace moe
