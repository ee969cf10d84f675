// k_attn_e4m3.cu -- the attention kernel's forms for E4M3 caches.
#include "attn_dev.cuh"

namespace moe {
namespace attn {

Form pick_e4m3(int dim, int group, bool wide) { return pick<MOE_E4M3>(dim, group, wide); }

}  // namespace attn
}  // namespace moe
