// Internal interface of the attention and cache kernels (api_attn.cpp calls
// the launchers; attn_*.hip and kv_pages.hip hold the kernels).
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace qg {

// the paged cache as the kernels take it (page_size = 1 << page_shift)
struct KvArgs {
  int layers, pages, page_shift, heads_kv, head_dim, rows, max_pages;
  uint16_t *k, *v;
  int32_t *tables, *lens, *refs, *status;
};

struct KvScratch {
  int32_t* free_list;  // [pages]: free pages found, lowest first
  int32_t* src;        // [rows] fork: the page to copy from, or -1; compact: 1 if the row is compacted
  int32_t* dst;        // [rows] fork: the page to copy to
};

// status bits (QGEMV_KV_*)
enum { KV_NO_PAGES = 1, KV_TABLE_FULL = 2, KV_BAD_INDEX = 4, KV_SHARED = 8 };

hipError_t launch_kv_reserve(const KvArgs& c, const int32_t* cu, int32_t* pos, const KvScratch& w, hipStream_t s);

struct KvWriteArgs {
  KvArgs c;
  int layer, tokens;
  const uint16_t *k, *v;
  int64_t k_token, k_head, v_token, v_head;
  const int32_t *cu, *pos;
};
hipError_t launch_kv_write(const KvWriteArgs& a, hipStream_t s);

hipError_t launch_kv_fork(const KvArgs& c, const int32_t* parents, const KvArgs& out, const KvScratch& w,
                          hipStream_t s);
hipError_t launch_kv_compact(const KvArgs& c, const int32_t* pos, const int32_t* keep, int max_keep,
                             const int32_t* count, const KvScratch& w, hipStream_t s);

// Attention.  One form for both sources of keys: packed rows (tables NULL;
// cu_k, k_token .. v_head) or one layer of a paged cache (tables set; k and v
// point at the layer, a page holds [page_size][heads_kv][head_dim]).
struct AttnArgs {
  int bf16, head_dim, heads, heads_kv, group;  // group = heads / heads_kv
  int tokens, rows;
  int causal;     // packed keys only
  float scale;    // score scale times log2(e): the kernels work in powers of two
  const uint16_t *q, *k, *v;
  uint16_t* o;
  int64_t q_token, q_head, k_token, k_head, v_token, v_head, o_token, o_head;
  const int32_t* cu;
  // packed keys
  int tokens_k;
  const int32_t* cu_k;
  // paged keys
  const int32_t *tables, *pos;
  int pages, page_shift, max_pages;
  const uint64_t* mask;
  int mask_words;
  float* ws;
  float join_cost;  // of one part in units of keys, over the call's items (narrow kernel, Walk::init)
  uint64_t nonce;  // of the call (attn_narrow.hip, last_part): 48 bits, not 0
};

// The choice of kernel, its split of the keys, and so the workspace, depend on
// the sizes that the host knows (not on lengths on the device).
// Waves per SIMD that the kernels' registers allow, and the workgroups (of one
// wave per SIMD) that then fill the 256 compute units: the split of a tree's
// keys is over that many.
// (The narrow kernel's parts of an item are joined by one workgroup.  Where all
// are parts of one item, half the workgroups leave half of them: one query head
// on 131072 keys 21 us with 256, 26 with 512, eight heads 33.5 with either.  Of
// two items one may still have nearly all parts: a row of 300000 keys beside one
// of a single key 38 us, alone 34.)
inline int narrow_workgroups(int rows, int heads_kv) { return (int64_t)rows * heads_kv < 2 ? 256 : 512; }
// (waves: per workgroup, 4 or 8; of 8, one workgroup fits a compute unit)
constexpr int wide_waves(int head_dim, int waves) { return head_dim == 64 && waves == 4 ? 3 : 2; }
constexpr int wide_workgroups(int head_dim, int waves) { return 256 * wide_waves(head_dim, waves) * 4 / waves; }
constexpr int PROMPT_WAVES = 4;
constexpr size_t partial_bytes(size_t slots, int bm, int d) { return slots * bm * (size_t)(d + 2) * 4; }

// 16-row tiles a wave of the narrow kernel holds (1 or 2) for the average
// row's queries, or 0: the wide kernel.  Both sides at 16 query rows a key head
// (one tile, two tiles): 16 rows of 4000 keys and 8 key heads 48 and 55 us, one
// row of them 13.5 and 17; at 32 (two tiles, wide kernel): 58 and 58, one row 22
// and 40, 16 rows of 1000 to 8200 keys 59 and 55.
inline int narrow_tiles(int tokens, int rows, int group) {
  const int64_t avg = ((int64_t)tokens + rows - 1) / rows * group;
  return avg <= 16 ? 1 : avg <= 32 ? 2 : 0;
}
// Waves of a workgroup of the wide kernel over a paged cache (32 query rows
// each).  With 8, more than 128 rows of a row and key head share one read of
// its keys.
inline int tree_waves(int tokens, int rows, int group) {
  return ((int64_t)tokens + rows - 1) / rows * group > 128 ? 8 : 4;
}
inline int wide_tiles(int tokens, int rows, int group, int waves) {
  return (int)((int64_t)tokens * group / (32 * waves)) + rows;
}
// parts of the keys of each tile, where whole tiles would leave compute units
// idle: as many workgroups as fit, of at least 1024 keys on average.  (With 256
// keys instead, 32 heads over 8: fresh prompts of 512 and 1000 tokens 17 -> 22
// and 27 -> 36 us, 100 tokens behind 700 and 1900 23 -> 20 and 43 -> 26.)
inline int prompt_splits(int tokens, int tokens_k, int rows, int heads_kv, int group, int head_dim, int waves) {
  const int64_t items = (int64_t)wide_tiles(tokens, rows, group, waves) * heads_kv;
  const int64_t most = tokens_k / rows / 1024, fit = wide_workgroups(head_dim, waves) / items;
  const int64_t s = fit < most ? fit : most;
  return s < 1 ? 1 : (int)s;
}

hipError_t launch_attn_narrow(const AttnArgs& a, int rt, hipStream_t s);
hipError_t launch_attn_wide(const AttnArgs& a, hipStream_t s);

}  // namespace qg
