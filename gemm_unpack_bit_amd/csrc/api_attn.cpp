// C ABI of the attention and cache calls (qgemv_attn.h): argument checks and
// dispatch.  Host-only code; kernels live in attn_*.hip and kv_pages.hip.
#include "qgemv_attn.h"

#include <hip/hip_runtime.h>
#include <unistd.h>

#include <atomic>
#include <chrono>
#include <cmath>
#include <cstdint>
#include <initializer_list>

#include "attn.hpp"
#include "kernels.hpp"
#include "spans.hpp"

namespace {

using qg::aligned;
using qg::overlap;
using qg::Span;
using qg::span;

Span span(const qgemv_heads& x, int tokens, int heads, int dim) {
  if (tokens < 1 || heads < 1) return span(x.data, 0);
  return span(x.data, 2 * ((tokens - 1) * x.token + (heads - 1) * x.head + dim));
}

constexpr int64_t STRIDE_MAX = (int64_t)1 << 40;  // (products with 32-bit counts stay in 64 bits once checked)
constexpr int64_t KEYS_MAX = ((int64_t)1 << 31) - 1024;  // (the kernels look a few steps past a row's last key, in 32 bits)
constexpr int WRITE_MAX = (1 << 26) - 4;  // tokens of one kv_write: a wave each, launches stay under 2^32 threads
constexpr int64_t KEY_STRIDE_MAX = (int64_t)1 << 26;  // 16 keys of a tile lie within 32-bit offsets of one another

// the array with the strides that lead anywhere (that of a single token or head
// may be anything: a view's of a padded row, say)
qgemv_heads used(const qgemv_heads& x, int tokens, int heads) {
  return {x.data, tokens > 1 ? x.token : 0, heads > 1 ? x.head : 0};
}

// strides in range and, for an output, no element shared
int check_heads(const qgemv_heads& x, int tokens, int heads, int dim, bool output) {
  if (x.token < 0 || x.head < 0 || x.token > STRIDE_MAX || x.head > STRIDE_MAX) return QGEMV_ERR_SHAPE;
  if (tokens > 0 && heads > 0) {
    const double reach = (double)(tokens - 1) * x.token + (double)(heads - 1) * x.head + dim;
    if (reach >= 4.6e18 / 2) return QGEMV_ERR_SHAPE;
    if (output) {
      const bool t1 = tokens == 1, h1 = heads == 1;
      const bool heads_in_token = (h1 || x.head >= dim) && (t1 || x.token >= (heads - 1) * x.head + dim);
      const bool tokens_in_head = (t1 || x.token >= dim) && (h1 || x.head >= (tokens - 1) * x.token + dim);
      if (!heads_in_token && !tokens_in_head) return QGEMV_ERR_SHAPE;
    }
  }
  return QGEMV_OK;
}
bool aligned_heads(const qgemv_heads& x) { return aligned(x.data, 16) && x.token % 8 == 0 && x.head % 8 == 0; }

int check_kind(int dtype, int head_dim) {
  if (dtype != QGEMV_F16 && dtype != QGEMV_BF16) return QGEMV_ERR_UNSUPPORTED;
  return head_dim == 64 || head_dim == 128 ? QGEMV_OK : QGEMV_ERR_UNSUPPORTED;
}

int check_counts(int tokens, int rows, int heads, int heads_kv) {
  if (tokens < 0 || rows < 0 || heads < 1 || heads_kv < 1 || heads % heads_kv) return QGEMV_ERR_SHAPE;
  if ((int64_t)tokens * heads >= (int64_t)1 << 31 || rows >= 1 << 24) return QGEMV_ERR_SHAPE;
  return QGEMV_OK;
}

// Whether the wide kernels' launches stay under 2^32 threads: up to 8 workgroups
// of 256 threads per 128 query rows and key head.
bool launchable(int tokens, int rows, int heads, int heads_kv) {
  const int group = heads / heads_kv;
  if (!tokens || !rows || qg::narrow_tiles(tokens, rows, group)) return true;
  return (int64_t)qg::wide_tiles(tokens, rows, group, 4) * heads_kv < 1 << 21 && heads_kv < 65536;
}

// Whether the units of work that the device shares out (Walk) stay within its
// sums, whatever the offsets say (each row may seem to have all tokens and all
// keys): those of 64 rows in two sums of 32 bits (over units / 2^24), those of
// all rows in 63.  Packed prompts in the wide kernel are not shared out so.
bool countable(int tokens, int rows, int heads, int heads_kv, int64_t keys, bool paged) {
  if (!tokens || !rows) return true;
  const int rt = qg::narrow_tiles(tokens, rows, heads / heads_kv);
  if (!rt && !paged) return true;
  const double tiles = (double)tokens * heads / (rt ? 16 * rt : 128) + heads_kv;
  const double units = tiles * ((double)keys / (rt ? 128 : 64) + 1);
  return units < 0x1p50 && units * rows < 0x1p62;
}

size_t narrow_bytes(int rows, int heads_kv, int rt, int head_dim) {
  const size_t n = (size_t)qg::narrow_workgroups(rows, heads_kv);
  return qg::partial_bytes(2 * n, 16 * rt, head_dim) + 16 * n;  // (and two words per share for the tickets)
}

// A number of 48 bits for the tickets of one call's parts: counted up from a
// random start, so that what an uninitialized workspace holds is not taken for
// one; never 0.  (getentropy reports an error where std::random_device throws;
// then the clock and a stack address have to do.)
uint64_t next_nonce() {
  static std::atomic<uint64_t> count{[] {
    uint64_t r = 0;
    if (getentropy(&r, sizeof r))
      r = (uint64_t)std::chrono::steady_clock::now().time_since_epoch().count() * 0x9E3779B97F4A7C15u ^
          reinterpret_cast<uintptr_t>(&r);
    return r;
  }()};
  for (;;)
    if (const uint64_t n = count.fetch_add(1) & 0xFFFFFFFFFFFFu) return n;
}

int check_scale(float scale) { return std::isfinite(scale) && scale >= 0.f ? QGEMV_OK : QGEMV_ERR_VALUE; }

// A cache of either kind: 16 bits, or 8 bits with exponents
struct Cache {
  int layers, pages, page_size, heads_kv, head_dim, rows, max_pages;
  void *k, *v;
  uint8_t *k_exps, *v_exps;
  int32_t *tables, *lens, *refs, *status;
  bool given, bits8;
};
Cache view(const qgemv_kv_cache* c) {
  if (!c) return Cache{};
  return {c->layers, c->pages, c->page_size, c->heads_kv, c->head_dim, c->rows, c->max_pages, c->k, c->v, nullptr, nullptr,
          c->tables, c->lens, c->refs, c->status, true, false};
}
Cache view(const qgemv_kv8_cache* c) {
  if (!c) return Cache{};
  return {c->layers, c->pages, c->page_size, c->heads_kv, c->head_dim, c->rows, c->max_pages, c->k, c->v, c->k_exps, c->v_exps,
          c->tables, c->lens, c->refs, c->status, true, true};
}

// The pools of a cache and its bookkeeping: null, format, shape, alignment.
// Every call but those that write or read tokens changes refs and tables.
bool missing(const Cache& c) {
  return !c.given || !c.k || !c.v || !c.tables || (c.bits8 && (!c.k_exps || !c.v_exps));
}
int check_cache(const Cache& c, bool state) {
  if (missing(c)) return QGEMV_ERR_NULL;
  if (state && (!c.lens || !c.refs || !c.status)) return QGEMV_ERR_NULL;
  if (c.head_dim != 64 && c.head_dim != 128) return QGEMV_ERR_UNSUPPORTED;
  if (c.page_size < 16 || c.page_size > 256 || (c.page_size & (c.page_size - 1))) return QGEMV_ERR_UNSUPPORTED;
  if (c.layers < 1 || c.pages < 1 || c.heads_kv < 1 || c.rows < 0 || c.rows > 65535 || c.max_pages < 1)
    return QGEMV_ERR_SHAPE;
  if ((int64_t)c.max_pages * c.page_size > KEYS_MAX || (int64_t)c.heads_kv * c.head_dim >= KEY_STRIDE_MAX || c.layers > 65536 ||
      (double)c.layers * c.pages * c.page_size * c.heads_kv * c.head_dim >= 1e15 ||
      (int64_t)c.layers * c.heads_kv * c.head_dim >= (int64_t)1 << 32)  // (a launch's threads: a thread per 16 bytes)
    return QGEMV_ERR_SHAPE;
  if (!aligned(c.k, 16) || !aligned(c.v, 16) || !aligned(c.tables, 4)) return QGEMV_ERR_ALIGN;
  if (state && (!aligned(c.lens, 4) || !aligned(c.refs, 4) || !aligned(c.status, 4))) return QGEMV_ERR_ALIGN;
  return QGEMV_OK;
}

int64_t elements(const Cache& c) { return (int64_t)c.layers * c.pages * c.page_size * c.heads_kv * c.head_dim; }
int64_t pool_bytes(const Cache& c) { return (c.bits8 ? 1 : 2) * elements(c); }
int64_t exps_bytes(const Cache& c) { return c.bits8 ? elements(c) / (qg::KV_BLOCK * c.head_dim) : 0; }

qg::KvArgs cache_args(const Cache& c) {
  qg::KvArgs a;
  a.layers = c.layers;
  a.pages = c.pages;
  a.page_shift = __builtin_ctz((unsigned)c.page_size);
  a.heads_kv = c.heads_kv;
  a.head_dim = c.head_dim;
  a.rows = c.rows;
  a.max_pages = c.max_pages;
  a.k = reinterpret_cast<uint16_t*>(c.k);
  a.v = reinterpret_cast<uint16_t*>(c.v);
  a.k_exps = c.k_exps;
  a.v_exps = c.v_exps;
  a.tables = c.tables;
  a.lens = c.lens;
  a.refs = c.refs;
  a.status = c.status;
  return a;
}

// (the pools of one cache and their exponents)
struct Pools {
  Span of[4];
};
Pools pools(const Cache& c) {
  return {{span(c.k, pool_bytes(c)), span(c.v, pool_bytes(c)), span(c.k_exps, exps_bytes(c)), span(c.v_exps, exps_bytes(c))}};
}
bool overlap(const Pools& p, const Span& x) {
  for (const Span& s : p.of)
    if (qg::overlap(s, x)) return true;
  return false;
}
bool apart(const Pools& p, std::initializer_list<Span> others) {
  for (const Span& x : others)
    if (overlap(p, x)) return false;
  return true;
}
// whether no pool (or its exponents) lies over another one
bool distinct(const Pools& p) {
  for (int i = 0; i < 4; ++i)
    for (int j = 0; j < i; ++j)
      if (qg::overlap(p.of[i], p.of[j])) return false;
  return true;
}
Span tables_of(const Cache& c) { return span(c.tables, (int64_t)4 * c.rows * c.max_pages); }
Span lens_of(const Cache& c) { return span(c.lens, c.lens ? (int64_t)4 * c.rows : 0); }
Span refs_of(const Cache& c) { return span(c.refs, c.refs ? (int64_t)4 * c.pages : 0); }
Span status_of(const Cache& c) { return span(c.status, c.status ? 4 : 0); }
Span kv_scratch(int rows, int pages, const void* ws) {
  return span(ws, ws ? (int64_t)qgemv_kv_workspace_bytes(rows, pages) : 0);
}

// cache calls: what one writes lies apart from all else that it writes, and
// from what it reads
bool apart(std::initializer_list<Span> writes, std::initializer_list<Span> reads) {
  for (auto w = writes.begin(); w != writes.end(); ++w) {
    for (auto x = writes.begin(); x != w; ++x)
      if (overlap(*w, *x)) return false;
    for (const Span& r : reads)
      if (overlap(*w, r)) return false;
  }
  return true;
}

size_t up16(size_t n) { return (n + 15) / 16 * 16; }

int scratch(int rows, int pages, void* ws, size_t ws_bytes, qg::KvScratch* w) {
  if (!ws || ws_bytes < qgemv_kv_workspace_bytes(rows, pages)) return QGEMV_ERR_WORKSPACE;
  if (!aligned(ws, 16)) return QGEMV_ERR_ALIGN;
  char* p = reinterpret_cast<char*>(ws);
  w->free_list = reinterpret_cast<int32_t*>(p);
  w->src = reinterpret_cast<int32_t*>(p + up16((size_t)pages * 4));
  w->dst = reinterpret_cast<int32_t*>(p + up16((size_t)pages * 4) + up16((size_t)rows * 4));
  return QGEMV_OK;
}

// attention: o against what the call reads (or the cache keeps) and its workspace
bool writes_input(const Span& o, const Span& ws, const Span* in, int n) {
  for (int i = 0; i < n; ++i)
    if (overlap(o, in[i]) || overlap(ws, in[i])) return true;
  return overlap(o, ws);
}

hipStream_t stream_of(qgemv_stream_t s) { return reinterpret_cast<hipStream_t>(s); }

}  // namespace

extern "C" {

size_t qgemv_attn_prompt_workspace_bytes(int tokens, int tokens_k, int batch, int heads, int heads_kv, int head_dim) {
  if (check_counts(tokens, batch, heads, heads_kv) || tokens_k < 0 || tokens_k > KEYS_MAX || !tokens || !batch) return 0;
  if (head_dim != 64 && head_dim != 128) return 0;
  const int group = heads / heads_kv, rt = qg::narrow_tiles(tokens, batch, group);
  if (rt) return narrow_bytes(batch, heads_kv, rt, head_dim);
  const int waves = qg::PROMPT_WAVES, splits = qg::prompt_splits(tokens, tokens_k, batch, heads_kv, group, head_dim, waves);
  if (splits == 1) return 0;
  return qg::partial_bytes((size_t)qg::wide_tiles(tokens, batch, group, waves) * heads_kv * splits, 32 * waves, head_dim);
}

int qgemv_attn_prompt(int dtype, int causal, int tokens, int tokens_k, int batch, int heads, int heads_kv,
                      int head_dim, float scale, const qgemv_heads* q_, const qgemv_heads* k_, const qgemv_heads* v_,
                      const int32_t* cu_q, const int32_t* cu_k, const qgemv_heads* o_, void* ws, size_t ws_bytes,
                      qgemv_stream_t stream) {
  if (!q_ || !k_ || !v_ || !o_ || !cu_q || !cu_k || !q_->data || !k_->data || !v_->data || !o_->data) return QGEMV_ERR_NULL;
  int rc = check_kind(dtype, head_dim);
  if (rc) return rc;
  if ((rc = check_counts(tokens, batch, heads, heads_kv))) return rc;
  if (tokens_k < 0 || tokens_k > KEYS_MAX || !launchable(tokens, batch, heads, heads_kv) ||
      !countable(tokens, batch, heads, heads_kv, tokens_k, false))
    return QGEMV_ERR_SHAPE;
  const qgemv_heads q = used(*q_, tokens, heads), k = used(*k_, tokens_k, heads_kv), v = used(*v_, tokens_k, heads_kv),
                    o = used(*o_, tokens, heads);
  if ((rc = check_heads(q, tokens, heads, head_dim, false)) || (rc = check_heads(k, tokens_k, heads_kv, head_dim, false)) ||
      (rc = check_heads(v, tokens_k, heads_kv, head_dim, false)) || (rc = check_heads(o, tokens, heads, head_dim, true)))
    return rc;
  if (k.token >= KEY_STRIDE_MAX || v.token >= KEY_STRIDE_MAX) return QGEMV_ERR_SHAPE;
  if ((rc = check_scale(scale))) return rc;
  if (!aligned_heads(q) || !aligned_heads(k) || !aligned_heads(v) || !aligned_heads(o) || !aligned(cu_q, 4) ||
      !aligned(cu_k, 4))
    return QGEMV_ERR_ALIGN;
  const size_t need = qgemv_attn_prompt_workspace_bytes(tokens, tokens_k, batch, heads, heads_kv, head_dim);
  const Span so = span(o, tokens, heads, head_dim), sw = span(ws, need && ws ? (int64_t)need : 0);
  const Span in[] = {span(q, tokens, heads, head_dim), span(k, tokens_k, heads_kv, head_dim),
                     span(v, tokens_k, heads_kv, head_dim), span(cu_q, 4 * ((int64_t)batch + 1)),
                     span(cu_k, 4 * ((int64_t)batch + 1))};
  if (writes_input(so, sw, in, 5)) return QGEMV_ERR_VALUE;
  if (need && (!ws || ws_bytes < need)) return QGEMV_ERR_WORKSPACE;
  if (need && !aligned(ws, 16)) return QGEMV_ERR_ALIGN;
  if (!tokens || !batch) return QGEMV_OK;
  qg::AttnArgs a{};
  a.bf16 = dtype == QGEMV_BF16;
  a.head_dim = head_dim;
  a.heads = heads;
  a.heads_kv = heads_kv;
  a.group = heads / heads_kv;
  a.tokens = tokens;
  a.rows = batch;
  a.causal = causal != 0;
  a.scale = scale * 1.4426950408889634f;
  a.q = q.data, a.q_token = q.token, a.q_head = q.head;
  a.k = k.data, a.k_token = k.token, a.k_head = k.head;
  a.v = v.data, a.v_token = v.token, a.v_head = v.head;
  a.o = o.data, a.o_token = o.token, a.o_head = o.head;
  a.cu = cu_q;
  a.cu_k = cu_k;
  a.tokens_k = tokens_k;
  a.ws = reinterpret_cast<float*>(ws);
  a.nonce = next_nonce();
  const int rt = qg::narrow_tiles(tokens, batch, a.group);
  return qg::hip_status(rt ? qg::launch_attn_narrow(a, rt, stream_of(stream)) : qg::launch_attn_wide(a, stream_of(stream)));
}

size_t qgemv_attn_tree_workspace_bytes(int tokens, int rows, int heads, int heads_kv, int head_dim) {
  if (check_counts(tokens, rows, heads, heads_kv) || !tokens || !rows) return 0;
  if (head_dim != 64 && head_dim != 128) return 0;
  const int rt = qg::narrow_tiles(tokens, rows, heads / heads_kv);
  if (rt) return narrow_bytes(rows, heads_kv, rt, head_dim);
  const int waves = qg::tree_waves(tokens, rows, heads / heads_kv);
  return qg::partial_bytes(2 * (size_t)qg::wide_workgroups(head_dim, waves), 32 * waves, head_dim);
}

namespace {
int attn_tree(int dtype, const Cache& c, int layer, int tokens, int heads, float scale, const qgemv_heads* q_,
              const int32_t* cu, const int32_t* pos, const uint64_t* mask, int mask_words, const qgemv_heads* o_, void* ws,
              size_t ws_bytes, qgemv_stream_t stream) {
  if (missing(c) || !q_ || !q_->data || !o_ || !o_->data || !cu || !pos) return QGEMV_ERR_NULL;
  int rc = check_kind(dtype, c.head_dim);
  if (rc) return rc;
  if ((rc = check_cache(c, false))) return rc;
  if ((rc = check_counts(tokens, c.rows, heads, c.heads_kv))) return rc;
  if (!launchable(tokens, c.rows, heads, c.heads_kv) ||
      !countable(tokens, c.rows, heads, c.heads_kv, (int64_t)c.max_pages * c.page_size, true))
    return QGEMV_ERR_SHAPE;
  if (layer < 0 || layer >= c.layers || mask_words < 0 || mask_words > 1 << 20 || (mask != nullptr) != (mask_words > 0))
    return QGEMV_ERR_SHAPE;
  const qgemv_heads q = used(*q_, tokens, heads), o = used(*o_, tokens, heads);
  if ((rc = check_heads(q, tokens, heads, c.head_dim, false)) || (rc = check_heads(o, tokens, heads, c.head_dim, true)))
    return rc;
  if ((rc = check_scale(scale))) return rc;
  if (!aligned_heads(q) || !aligned_heads(o) || !aligned(cu, 4) || !aligned(pos, 4) || !aligned(mask, 8))
    return QGEMV_ERR_ALIGN;
  const size_t need = qgemv_attn_tree_workspace_bytes(tokens, c.rows, heads, c.heads_kv, c.head_dim);
  const Span so = span(o, tokens, heads, c.head_dim), sw = span(ws, need && ws ? (int64_t)need : 0);
  const Pools p = pools(c);
  const Span in[] = {span(q, tokens, heads, c.head_dim), p.of[0], p.of[1], p.of[2], p.of[3], tables_of(c), lens_of(c),
                     refs_of(c), status_of(c), span(cu, 4 * ((int64_t)c.rows + 1)), span(pos, (int64_t)4 * c.rows),
                     span(mask, (int64_t)8 * tokens * mask_words)};
  if (writes_input(so, sw, in, 12)) return QGEMV_ERR_VALUE;
  if (need && (!ws || ws_bytes < need)) return QGEMV_ERR_WORKSPACE;
  if (need && !aligned(ws, 16)) return QGEMV_ERR_ALIGN;
  if (!tokens || !c.rows) return QGEMV_OK;
  qg::AttnArgs a{};
  a.bf16 = dtype == QGEMV_BF16;
  a.head_dim = c.head_dim;
  a.heads = heads;
  a.heads_kv = c.heads_kv;
  a.group = heads / c.heads_kv;
  a.tokens = tokens;
  a.rows = c.rows;
  a.causal = 1;
  a.scale = scale * 1.4426950408889634f;
  const int64_t row = (int64_t)c.heads_kv * c.head_dim, in_layer = (int64_t)c.pages * c.page_size * row;
  a.q = q.data, a.q_token = q.token, a.q_head = q.head;
  const int64_t at = layer * in_layer / (c.bits8 ? 2 : 1);  // (codes are a byte each; a layer has a multiple of 16)
  a.k = reinterpret_cast<const uint16_t*>(c.k) + at, a.k_token = row, a.k_head = c.head_dim;
  a.v = reinterpret_cast<const uint16_t*>(c.v) + at, a.v_token = row, a.v_head = c.head_dim;
  if (c.bits8) {
    const int64_t block = layer * (in_layer / (qg::KV_BLOCK * c.head_dim));
    a.k_exps = c.k_exps + block;
    a.v_exps = c.v_exps + block;
  }
  a.o = o.data, a.o_token = o.token, a.o_head = o.head;
  a.cu = cu;
  a.tables = c.tables;
  a.pos = pos;
  a.pages = c.pages;
  a.page_shift = __builtin_ctz((unsigned)c.page_size);
  a.max_pages = c.max_pages;
  a.mask = mask;
  a.mask_words = mask_words;
  a.ws = reinterpret_cast<float*>(ws);
  a.nonce = next_nonce();
  const int rt = qg::narrow_tiles(tokens, a.rows, a.group);
  return qg::hip_status(rt ? qg::launch_attn_narrow(a, rt, stream_of(stream)) : qg::launch_attn_wide(a, stream_of(stream)));
}
}  // namespace

int qgemv_attn_tree(int dtype, const qgemv_kv_cache* c, int layer, int tokens, int heads, float scale,
                    const qgemv_heads* q, const int32_t* cu, const int32_t* pos, const uint64_t* mask,
                    int mask_words, const qgemv_heads* o, void* ws, size_t ws_bytes, qgemv_stream_t stream) {
  return attn_tree(dtype, view(c), layer, tokens, heads, scale, q, cu, pos, mask, mask_words, o, ws, ws_bytes, stream);
}
int qgemv_attn_tree8(int dtype, const qgemv_kv8_cache* c, int layer, int tokens, int heads, float scale,
                     const qgemv_heads* q, const int32_t* cu, const int32_t* pos, const uint64_t* mask,
                     int mask_words, const qgemv_heads* o, void* ws, size_t ws_bytes, qgemv_stream_t stream) {
  return attn_tree(dtype, view(c), layer, tokens, heads, scale, q, cu, pos, mask, mask_words, o, ws, ws_bytes, stream);
}

size_t qgemv_kv_workspace_bytes(int rows, int pages) {
  if (rows < 0 || pages < 1) return 0;
  return up16((size_t)pages * 4) + 2 * up16((size_t)rows * 4);
}

namespace {

int kv_reserve(const Cache& c, const int32_t* cu, int32_t* pos, void* ws, size_t ws_bytes,
                     qgemv_stream_t stream) {
  int rc = check_cache(c, true);
  if (rc) return rc;
  if (!cu || !pos) return QGEMV_ERR_NULL;
  if (!aligned(cu, 4) || !aligned(pos, 4)) return QGEMV_ERR_ALIGN;
  const Span sp = span(pos, (int64_t)4 * c.rows), sw = kv_scratch(c.rows, c.pages, ws);
  if (!apart({sp, sw, tables_of(c), lens_of(c), refs_of(c), status_of(c)}, {span(cu, (int64_t)4 * (c.rows + 1))}) ||
      !apart(pools(c), {sp, sw, tables_of(c), lens_of(c), refs_of(c), status_of(c)}))
    return QGEMV_ERR_VALUE;
  qg::KvScratch w;
  if ((rc = scratch(c.rows, c.pages, ws, ws_bytes, &w))) return rc;
  if (!c.rows) return QGEMV_OK;
  return qg::hip_status(qg::launch_kv_reserve(cache_args(c), cu, pos, w, stream_of(stream)));
}

int kv_fork(const Cache& c, const int32_t* parents, const Cache& out, void* ws,
                  size_t ws_bytes, qgemv_stream_t stream) {
  int rc = check_cache(c, true);
  if (rc) return rc;
  if ((rc = check_cache(out, true))) return rc;
  if (!parents) return QGEMV_ERR_NULL;
  if (out.layers != c.layers || out.pages != c.pages || out.page_size != c.page_size ||
      out.heads_kv != c.heads_kv || out.head_dim != c.head_dim || out.max_pages != c.max_pages)
    return QGEMV_ERR_SHAPE;
  if (!aligned(parents, 4)) return QGEMV_ERR_ALIGN;
  const int rows = c.rows > out.rows ? c.rows : out.rows;
  const Span sp = span(parents, (int64_t)4 * out.rows);
  if (out.k != c.k || out.v != c.v || out.k_exps != c.k_exps || out.v_exps != c.v_exps || out.refs != c.refs || out.status != c.status ||
      !apart({tables_of(out), lens_of(out), kv_scratch(rows, c.pages, ws), refs_of(c), status_of(c)},
             {sp, tables_of(c), lens_of(c)}) ||
      !apart(pools(c), {sp, tables_of(c), lens_of(c), tables_of(out), lens_of(out), kv_scratch(rows, c.pages, ws), refs_of(c),
                        status_of(c)}) ||
      (c.bits8 && !distinct(pools(c))))
    return QGEMV_ERR_VALUE;
  qg::KvScratch w;
  if ((rc = scratch(rows, c.pages, ws, ws_bytes, &w))) return rc;
  if (!rows) return QGEMV_OK;
  return qg::hip_status(qg::launch_kv_fork(cache_args(c), parents, cache_args(out), w, stream_of(stream)));
}

int kv_compact(const Cache& c, const int32_t* pos, const int32_t* keep, int max_keep,
                     const int32_t* count, void* ws, size_t ws_bytes, qgemv_stream_t stream) {
  int rc = check_cache(c, true);
  if (rc) return rc;
  if (!pos || !count || (max_keep > 0 && !keep)) return QGEMV_ERR_NULL;
  if (max_keep < 0) return QGEMV_ERR_SHAPE;
  if (!aligned(pos, 4) || !aligned(keep, 4) || !aligned(count, 4)) return QGEMV_ERR_ALIGN;
  const Span sp = span(pos, (int64_t)4 * c.rows), sk = span(keep, (int64_t)4 * c.rows * max_keep),
             sc = span(count, (int64_t)4 * c.rows), sw = kv_scratch(c.rows, c.pages, ws);
  // (a row's length is written after its position and count are read: pos may be lens)
  if (!apart({sw, tables_of(c), refs_of(c), status_of(c)}, {sp, sk, sc, lens_of(c)}) ||
      !apart(pools(c), {sp, sk, sc, lens_of(c), sw, tables_of(c), refs_of(c), status_of(c)}) ||
      (c.bits8 && !distinct(pools(c))))
    return QGEMV_ERR_VALUE;
  qg::KvScratch w;
  if ((rc = scratch(c.rows, c.pages, ws, ws_bytes, &w))) return rc;
  if (!c.rows) return QGEMV_OK;
  return qg::hip_status(qg::launch_kv_compact(cache_args(c), pos, keep, max_keep, count, w, stream_of(stream)));
}

// whether two arrays share elements; parts of one array with the same token
// stride (a fused product's queries and keys) may lie side by side
bool overlap(const qgemv_heads& x, int heads_x, const qgemv_heads& y, int heads_y, int tokens, int dim) {
  if (!overlap(span(x, tokens, heads_x, dim), span(y, tokens, heads_y, dim))) return false;
  const int64_t t = x.token, ex = (heads_x - 1) * x.head + dim, ey = (heads_y - 1) * y.head + dim;
  const int64_t bytes = (int64_t)((uintptr_t)y.data - (uintptr_t)x.data);
  if (tokens < 2 || t != y.token || t < 1 || ex > t || ey > t || bytes % 2) return true;
  const int64_t d = ((bytes / 2) % t + t) % t;  // where a token of y begins in one of x
  return d < ex || d + ey > t;
}

int kv_append(int dtype, const Cache& c, int layer, int tokens, int heads, const qgemv_heads* q_, const qgemv_heads* k_,
              const qgemv_heads* v_, const int32_t* cu, const int32_t* pos, const float* freqs, int rot, int interleaved,
              const int32_t* at, const qgemv_heads* o_, qgemv_stream_t stream) {
  int rc;
  if (missing(c) || !k_ || !v_ || !k_->data || !v_->data || !cu || !pos || (rot > 0 && !freqs)) return QGEMV_ERR_NULL;
  if (heads > 0 && (!q_ || !o_ || !q_->data || !o_->data)) return QGEMV_ERR_NULL;
  if (dtype != QGEMV_F16 && dtype != QGEMV_BF16) return QGEMV_ERR_UNSUPPORTED;
  if ((rc = check_cache(c, false))) return rc;
  if (rot < 0 || rot > c.head_dim || rot % 16) return QGEMV_ERR_UNSUPPORTED;
  if (layer < 0 || layer >= c.layers || tokens < 0 || heads < 0) return QGEMV_ERR_SHAPE;
  // (waves of a launch: see launch_kv_append; it stays under 2^32 threads)
  const double each = (double)heads + 2.0 * c.heads_kv;
  if ((double)tokens * (each / 8 + 1) + 4.0 * c.rows * c.heads_kv >= 0x1p26 - 8) return QGEMV_ERR_SHAPE;
  const qgemv_heads none{nullptr, 0, 0};
  const qgemv_heads q = heads ? used(*q_, tokens, heads) : none, o = heads ? used(*o_, tokens, heads) : none;
  const qgemv_heads k = used(*k_, tokens, c.heads_kv), v = used(*v_, tokens, c.heads_kv);
  if ((rc = check_heads(q, tokens, heads, c.head_dim, false)) || (rc = check_heads(o, tokens, heads, c.head_dim, true)) ||
      (rc = check_heads(k, tokens, c.heads_kv, c.head_dim, false)) ||
      (rc = check_heads(v, tokens, c.heads_kv, c.head_dim, false)))
    return rc;
  if (!aligned_heads(q) || !aligned_heads(o) || !aligned_heads(k) || !aligned_heads(v) || !aligned(cu, 4) || !aligned(pos, 4) ||
      !aligned(freqs, 16) || !aligned(at, 4))
    return QGEMV_ERR_ALIGN;
  const Pools p = pools(c);
  const Span so = span(o, tokens, heads, c.head_dim);
  const Span small[] = {tables_of(c), lens_of(c), refs_of(c), status_of(c), span(cu, 4 * ((int64_t)c.rows + 1)),
                        span(pos, (int64_t)4 * c.rows), span(freqs, rot > 0 ? (int64_t)2 * rot : 0),
                        span(at, at ? (int64_t)4 * tokens : 0)};
  for (const Span& x : small)
    if (overlap(p, x) || overlap(so, x)) return QGEMV_ERR_VALUE;
  if (!distinct(p)) return QGEMV_ERR_VALUE;
  if (!apart(p, {so, span(q, tokens, heads, c.head_dim), span(k, tokens, c.heads_kv, c.head_dim),
                 span(v, tokens, c.heads_kv, c.head_dim)}))
    return QGEMV_ERR_VALUE;
  if (heads) {
    const bool in_place = o.data == q.data && o.token == q.token && o.head == q.head;
    if ((!in_place && overlap(o, heads, q, heads, tokens, c.head_dim)) ||
        overlap(o, heads, k, c.heads_kv, tokens, c.head_dim) || overlap(o, heads, v, c.heads_kv, tokens, c.head_dim))
      return QGEMV_ERR_VALUE;
  }
  if (!tokens || !c.rows) return QGEMV_OK;
  qg::KvAppendArgs a{};
  a.c = cache_args(c);
  a.bf16 = dtype == QGEMV_BF16;
  a.layer = layer;
  a.tokens = tokens;
  a.heads = heads;
  a.rot = rot;
  a.interleaved = interleaved != 0;
  a.q = q.data, a.q_token = q.token, a.q_head = q.head;
  a.k = k.data, a.k_token = k.token, a.k_head = k.head;
  a.v = v.data, a.v_token = v.token, a.v_head = v.head;
  a.o = o.data, a.o_token = o.token, a.o_head = o.head;
  a.freqs = freqs;
  a.at = rot ? at : nullptr;
  a.cu = cu;
  a.pos = pos;
  return qg::hip_status(qg::launch_kv_append(a, stream_of(stream)));
}

int kv_read(int dtype, const Cache& c, int layer, int tokens, const int32_t* cu, const int32_t* start,
            const qgemv_heads* k_, const qgemv_heads* v_, qgemv_stream_t stream) {
  int rc;
  if (missing(c) || !k_ || !v_ || !k_->data || !v_->data || !cu || !start) return QGEMV_ERR_NULL;
  if (dtype != QGEMV_F16 && dtype != QGEMV_BF16) return QGEMV_ERR_UNSUPPORTED;
  if ((rc = check_cache(c, false))) return rc;
  if (layer < 0 || layer >= c.layers || tokens < 0 || tokens > WRITE_MAX) return QGEMV_ERR_SHAPE;
  const qgemv_heads k = used(*k_, tokens, c.heads_kv), v = used(*v_, tokens, c.heads_kv);
  if ((rc = check_heads(k, tokens, c.heads_kv, c.head_dim, true)) || (rc = check_heads(v, tokens, c.heads_kv, c.head_dim, true)))
    return rc;
  if (!aligned_heads(k) || !aligned_heads(v) || !aligned(cu, 4) || !aligned(start, 4)) return QGEMV_ERR_ALIGN;
  const Pools p = pools(c);
  const Span sk = span(k, tokens, c.heads_kv, c.head_dim), sv = span(v, tokens, c.heads_kv, c.head_dim);
  const Span in[] = {tables_of(c), lens_of(c), refs_of(c), status_of(c), span(cu, 4 * ((int64_t)c.rows + 1)),
                     span(start, (int64_t)4 * c.rows)};
  for (const Span& x : in)
    if (overlap(sk, x) || overlap(sv, x)) return QGEMV_ERR_VALUE;
  if (!apart(p, {sk, sv}) || overlap(k, c.heads_kv, v, c.heads_kv, tokens, c.head_dim)) return QGEMV_ERR_VALUE;
  if (!tokens || !c.rows) return QGEMV_OK;
  qg::KvReadArgs a{cache_args(c), dtype == QGEMV_BF16, layer, tokens, k.data, v.data, k.token, k.head, v.token, v.head, cu, start};
  return qg::hip_status(qg::launch_kv_read(a, stream_of(stream)));
}

}  // namespace

int qgemv_kv_reserve(const qgemv_kv_cache* c, const int32_t* cu, int32_t* pos, void* ws, size_t ws_bytes,
                     qgemv_stream_t stream) {
  return kv_reserve(view(c), cu, pos, ws, ws_bytes, stream);
}
int qgemv_kv8_reserve(const qgemv_kv8_cache* c, const int32_t* cu, int32_t* pos, void* ws, size_t ws_bytes,
                      qgemv_stream_t stream) {
  return kv_reserve(view(c), cu, pos, ws, ws_bytes, stream);
}

int qgemv_kv_write(const qgemv_kv_cache* c_, int layer, int tokens, const qgemv_heads* k_, const qgemv_heads* v_,
                   const int32_t* cu, const int32_t* pos, qgemv_stream_t stream) {
  const Cache c = view(c_);
  int rc = check_cache(c, false);
  if (rc) return rc;
  if (!k_ || !v_ || !k_->data || !v_->data || !cu || !pos) return QGEMV_ERR_NULL;
  if (layer < 0 || layer >= c.layers || tokens < 0 || tokens > WRITE_MAX) return QGEMV_ERR_SHAPE;
  const qgemv_heads k = used(*k_, tokens, c.heads_kv), v = used(*v_, tokens, c.heads_kv);
  if ((rc = check_heads(k, tokens, c.heads_kv, c.head_dim, false)) ||
      (rc = check_heads(v, tokens, c.heads_kv, c.head_dim, false)))
    return rc;
  if (!aligned_heads(k) || !aligned_heads(v) || !aligned(cu, 4) || !aligned(pos, 4)) return QGEMV_ERR_ALIGN;
  const Span in[] = {span(k, tokens, c.heads_kv, c.head_dim), span(v, tokens, c.heads_kv, c.head_dim), tables_of(c),
                     span(cu, 4 * ((int64_t)c.rows + 1)), span(pos, (int64_t)4 * c.rows)};
  for (const Span& r : in)
    if (overlap(pools(c), r)) return QGEMV_ERR_VALUE;
  if (!tokens || !c.rows) return QGEMV_OK;
  qg::KvWriteArgs a{cache_args(c), layer, tokens, k.data, v.data, k.token, k.head, v.token, v.head, cu, pos};
  return qg::hip_status(qg::launch_kv_write(a, stream_of(stream)));
}

int qgemv_kv_append(int dtype, const qgemv_kv_cache* c, int layer, int tokens, int heads, const qgemv_heads* q,
                    const qgemv_heads* k, const qgemv_heads* v, const int32_t* cu, const int32_t* pos, const float* freqs,
                    int rot, int interleaved, const int32_t* at, const qgemv_heads* o, qgemv_stream_t stream) {
  return kv_append(dtype, view(c), layer, tokens, heads, q, k, v, cu, pos, freqs, rot, interleaved, at, o, stream);
}
int qgemv_kv8_append(int dtype, const qgemv_kv8_cache* c, int layer, int tokens, int heads, const qgemv_heads* q,
                     const qgemv_heads* k, const qgemv_heads* v, const int32_t* cu, const int32_t* pos, const float* freqs,
                     int rot, int interleaved, const int32_t* at, const qgemv_heads* o, qgemv_stream_t stream) {
  return kv_append(dtype, view(c), layer, tokens, heads, q, k, v, cu, pos, freqs, rot, interleaved, at, o, stream);
}

int qgemv_kv_read(const qgemv_kv_cache* c, int layer, int tokens, const int32_t* cu, const int32_t* start,
                  const qgemv_heads* k, const qgemv_heads* v, qgemv_stream_t stream) {
  return kv_read(QGEMV_F16, view(c), layer, tokens, cu, start, k, v, stream);  // (16 bits are copied as they are)
}
int qgemv_kv8_read(int dtype, const qgemv_kv8_cache* c, int layer, int tokens, const int32_t* cu, const int32_t* start,
                   const qgemv_heads* k, const qgemv_heads* v, qgemv_stream_t stream) {
  return kv_read(dtype, view(c), layer, tokens, cu, start, k, v, stream);
}

int qgemv_kv_fork(const qgemv_kv_cache* c, const int32_t* parents, const qgemv_kv_cache* out, void* ws,
                  size_t ws_bytes, qgemv_stream_t stream) {
  return kv_fork(view(c), parents, view(out), ws, ws_bytes, stream);
}
int qgemv_kv8_fork(const qgemv_kv8_cache* c, const int32_t* parents, const qgemv_kv8_cache* out, void* ws,
                   size_t ws_bytes, qgemv_stream_t stream) {
  return kv_fork(view(c), parents, view(out), ws, ws_bytes, stream);
}

int qgemv_kv_compact(const qgemv_kv_cache* c, const int32_t* pos, const int32_t* keep, int max_keep,
                     const int32_t* count, void* ws, size_t ws_bytes, qgemv_stream_t stream) {
  return kv_compact(view(c), pos, keep, max_keep, count, ws, ws_bytes, stream);
}
int qgemv_kv8_compact(const qgemv_kv8_cache* c, const int32_t* pos, const int32_t* keep, int max_keep,
                      const int32_t* count, void* ws, size_t ws_bytes, qgemv_stream_t stream) {
  return kv_compact(view(c), pos, keep, max_keep, count, ws, ws_bytes, stream);
}

}  // extern "C"
