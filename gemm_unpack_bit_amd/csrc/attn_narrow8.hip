// The kernel for few query rows per key head, over a cache of 8 bits.
#include "attn_narrow.hpp"

namespace qg {

hipError_t launch_attn_narrow8(const AttnArgs& a, int rt, hipStream_t s) {
  return rt == 1 ? launch_d<1, true, true>(a, s) : launch_d<2, true, true>(a, s);
}

}  // namespace qg
