// The kernel for few query rows per key head, over keys and values of 16 bits.
#include "attn_narrow.hpp"

namespace qg {

// Joining a part with R queries takes about R / 64 of the time of a unit of keys:
// 16 rows of them at once and 4 parts in flight.  Over an average item's n units
// the least time is at sqrt(n * R / 64) units a part.  Measured against parts as
// small as the workgroups allow: 8 tokens on 16000 keys 63 -> 35 us, 8-token
// trees on 4000 keys 31 -> 22 us, one key head with 8 heads on 131072 keys
// 43 -> 35 us; single tokens of 4 heads a key head stay as they were.
hipError_t launch_attn_narrow(const AttnArgs& args, int rt, hipStream_t s) {
  AttnArgs a = args;
  const float items = (float)a.rows * (float)a.heads_kv;
  const float queries = (float)a.tokens * (float)a.group / (float)a.rows;
  a.join_cost = (queries < 16.f * rt ? queries : 16.f * rt) / (64.f * items);
  if (a.k_exps) return launch_attn_narrow8(a, rt, s);
  if (a.tables) return rt == 1 ? launch_d<1, true, false>(a, s) : launch_d<2, true, false>(a, s);
  return rt == 1 ? launch_d<1, false, false>(a, s) : launch_d<2, false, false>(a, s);
}

}  // namespace qg
