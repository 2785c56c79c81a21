// The kernels for many query rows per key head, over keys and values of 16 bits.
#include "attn_wide.hpp"

namespace qg {
namespace {

template <typename E, int D>
hipError_t launch(const AttnArgs& a, hipStream_t s) {
  return a.tables ? tree_d<E, D, false>(a, s) : prompt<E, D, PROMPT_WAVES>(a, s);
}

}  // namespace

hipError_t launch_attn_wide(const AttnArgs& a, hipStream_t s) {
  if (a.k_exps) return launch_attn_wide8(a, s);
  if (a.head_dim == 128) return a.bf16 ? launch<BF16, 128>(a, s) : launch<F16, 128>(a, s);
  return a.bf16 ? launch<BF16, 64>(a, s) : launch<F16, 64>(a, s);
}

}  // namespace qg
