// The kernels for many query rows per key head, over a cache of 8 bits.
#include "attn_wide.hpp"

namespace qg {

hipError_t launch_attn_wide8(const AttnArgs& a, hipStream_t s) {
  if (a.head_dim == 128) return a.bf16 ? tree_d<BF16, 128, true>(a, s) : tree_d<F16, 128, true>(a, s);
  return a.bf16 ? tree_d<BF16, 64, true>(a, s) : tree_d<F16, 64, true>(a, s);
}

}  // namespace qg
