// The paged key/value cache: growing rows, writing new tokens, forking rows,
// compacting verified trees.
//
// State: tables[row][i] is the page that holds positions i << shift ..; refs
// counts the rows that hold a page, and a page with 0 is free.  There is no
// other allocator state: a call that needs n pages takes the n lowest-numbered
// free ones, found by one workgroup that scans refs (4 bytes a page, 8192
// pages an iteration, up to the last page it needs).  So the result depends
// on the state alone, never on the order of atomics, and a decode loop needs
// no host between steps.
//
// What moves is copied in 16-byte pieces: in a page, a token's heads are one
// contiguous block (heads_kv * head_dim elements), so a wave's load or store
// is 1 KB of one token (or of neighbouring tokens).  These kernels do no
// arithmetic: they are bound by their launches where little moves, else by
// the memory.
//
// Every page number read from a table is checked against the pool before it is
// used, and every row, slot and count against its range.
//
// In a cache of 8 bits a token's piece holds 16 codes, and the blocks' exponents
// go with their pages.  Compaction there moves tokens between blocks of
// different exponents: a block that gains tokens takes the largest of those that
// its tokens come from.  Measured (32 layers, 8 heads of 128): a fork of 8 rows 5.4 us
// for the pages and 3 for the copies, of 32 rows in pages of 64 5.5 and 14.
#include "attn.hpp"
#include "e4m3.hpp"
#include "rows.hpp"

namespace qg {
namespace {

constexpr int SCAN = 1024;  // threads of the one-workgroup kernels

// Exclusive prefix sum over the workgroup's SCAN threads; total in all.  Sums
// end at 2^32 - 1: rows with offsets that go up and down can need more pages
// together than 32 bits count, and whatever does not fit a pool is too many.
// (The additions saturate by themselves; with sums of 64 bits an append of one
// token to 48 rows takes 11.7 us for 11.3.)
__device__ __forceinline__ uint32_t block_scan(uint32_t v, uint32_t& total, uint32_t* red) {
  auto add = [](uint32_t a, uint32_t b) { return __builtin_elementwise_add_sat(a, b); };
  const int lane = threadIdx.x & 63, w = threadIdx.x >> 6;
  uint32_t s = v;
#pragma unroll
  for (int d = 1; d < 64; d <<= 1) {
    const uint32_t o = __shfl_up(s, d);
    if (lane >= d) s = add(s, o);
  }
  if (lane == 63) red[w] = s;
  __syncthreads();
  uint32_t before = 0, all = 0;
#pragma unroll
  for (int i = 0; i < SCAN / 64; ++i) {
    const uint32_t x = red[i];
    before = add(before, i < w ? x : 0);
    all = add(all, x);
  }
  __syncthreads();
  total = all;
  s = add(before, s);
  return s == UINT32_MAX ? s : s - v;
}

// The lowest `want` free pages into list, in order; returns how many there are
// (<= want).  All threads of the workgroup; ends with a barrier, so list can
// be read by any of them.  A wave takes 512 neighbouring pages, 64 at a time,
// and counts by ballots.
template <typename L>
__device__ __forceinline__ int find_free(const int32_t* refs, int pages, int want, L* list, int* red) {
  constexpr int EACH = 8;
  const int lane = threadIdx.x & 63, w = threadIdx.x >> 6;
  int found = 0;
  for (int p0 = 0; p0 < pages && found < want; p0 += EACH * SCAN) {
    const int p = p0 + w * 64 * EACH + lane;
    int r[EACH];
#pragma unroll
    for (int i = 0; i < EACH; ++i) r[i] = p + 64 * i < pages ? refs[p + 64 * i] : 1;
    uint64_t free[EACH];
    int n = 0;
#pragma unroll
    for (int i = 0; i < EACH; ++i) {
      free[i] = __ballot(r[i] == 0);
      n += __builtin_popcountll(free[i]);
    }
    if (lane == 0) red[w] = n;
    __syncthreads();
    int at = found, total = 0;
#pragma unroll
    for (int i = 0; i < SCAN / 64; ++i) {
      const int x = red[i];
      at += i < w ? x : 0;
      total += x;
    }
#pragma unroll
    for (int i = 0; i < EACH; ++i) {
      const int mine = at + __builtin_popcountll(free[i] & ((1ull << lane) - 1));
      if (free[i] >> lane & 1 && mine < want) list[mine] = p + 64 * i;
      at += __builtin_popcountll(free[i]);
    }
    found += total;
    __syncthreads();
  }
  return found < want ? found : want;
}

__device__ __forceinline__ int pages_of(int tokens, int shift) { return (int)(((int64_t)tokens + (1 << shift) - 1) >> shift); }

// ---------------------------------------------------------------------------
// reserve
// ---------------------------------------------------------------------------

// One workgroup: the pages that all rows need, the free pages, then the
// rows' shares of them in row order.  `need` of a row that cannot grow
// whatever the pool holds (bad count, table too short) is 0 pages, ok false.
__global__ void __launch_bounds__(SCAN) kv_reserve_kernel(KvArgs c, const int32_t* cu, int32_t* pos, KvScratch w) {
  __shared__ int red[SCAN / 64];
  __shared__ uint32_t sums[SCAN / 64];
  __shared__ int at_s[SCAN], need_s[SCAN], have_s[SCAN];
  struct Row {
    int len, n, have, need, bad;
  };
  auto row = [&](int b) {
    Row r{0, 0, 0, 0, 0};
    if (b >= c.rows) return r;
    r.len = c.lens[b];
    const int64_t n = (int64_t)cu[b + 1] - cu[b];
    r.n = (int)n;
    if (n < 0 || n > 0x7fffffff || r.len < 0) {
      r.bad = KV_BAD_INDEX;
    } else if (r.len + n > (int64_t)c.max_pages << c.page_shift) {
      r.bad = KV_TABLE_FULL;
    } else {
      r.have = pages_of(r.len, c.page_shift);
      r.need = pages_of(r.len + r.n, c.page_shift) - r.have;
    }
    return r;
  };
  Row r = row(threadIdx.x);
  uint32_t before, total;  // (the first 1024 rows are read and summed once)
  before = block_scan(r.need, total, sums);
  int64_t want = total;
  for (int b0 = SCAN; b0 < c.rows; b0 += SCAN) {
    uint32_t more;
    block_scan(row(b0 + threadIdx.x).need, more, sums);
    want += more;
  }
  const int got = want ? find_free(c.refs, c.pages, want < c.pages ? (int)want : c.pages, w.free_list, red) : 0;
  int64_t given = 0;
  int status = 0;
  for (int b0 = 0; b0 < c.rows; b0 += SCAN) {
    const int b = b0 + threadIdx.x;
    if (b0) {
      r = row(b);
      before = block_scan(r.need, total, sums);
    }
    const int64_t at = given + before;
    given += total;
    const bool fits = r.need == 0 || at + r.need <= got;
    const bool ok = b < c.rows && !r.bad && fits;
    at_s[threadIdx.x] = (int)at;  // (used where the row fits: at most got)
    need_s[threadIdx.x] = ok ? r.need : 0;
    have_s[threadIdx.x] = r.have;
    if (b < c.rows) {
      status |= r.bad | (fits ? 0 : KV_NO_PAGES);
      pos[b] = ok ? r.len : -1;
      if (ok) c.lens[b] = r.len + r.n;
    }
    __syncthreads();
    // a wave per row, a lane per page
    for (int i = threadIdx.x >> 6; i < SCAN && b0 + i < c.rows; i += SCAN / 64)
      for (int j = threadIdx.x & 63; j < need_s[i]; j += 64) {
        const int p = w.free_list[at_s[i] + j];
        c.tables[(int64_t)(b0 + i) * c.max_pages + have_s[i] + j] = p;
        c.refs[p] = 1;
      }
    __syncthreads();
  }
  if (status) atomicOr(c.status, status);
}

// ---------------------------------------------------------------------------
// write
// ---------------------------------------------------------------------------

// One wave per token: keys and values are read by the strides of their arrays
// (a head is head_dim contiguous elements) and written as one block each.
__global__ void __launch_bounds__(256) kv_write_kernel(KvWriteArgs a) {
  const KvArgs& c = a.c;
  const int lane = threadIdx.x & 63;
  const int t = __builtin_amdgcn_readfirstlane(blockIdx.x * 4 + (threadIdx.x >> 6));
  if (t >= a.tokens) return;
  const int b = find_row(c.rows, t, [&](int i) { return a.cu[i]; });
  const int i = t - a.cu[b], p0 = a.pos[b];
  if (p0 < 0 || i < 0 || t >= a.cu[b + 1]) return;
  const int64_t p = (int64_t)p0 + i;
  const int64_t slot = p >> c.page_shift;
  if (slot >= c.max_pages) return;
  const int page = c.tables[(int64_t)b * c.max_pages + slot];
  if ((unsigned)page >= (unsigned)c.pages) return;
  const int hs = c.head_dim == 128 ? 4 : 3;  // log2 of a head's 16-byte pieces
  const int n = c.heads_kv << hs;
  const int64_t at = ((((int64_t)a.layer * c.pages + page) << c.page_shift) + (p & ((1 << c.page_shift) - 1))) * n;
  u4* dk = reinterpret_cast<u4*>(c.k) + at;
  u4* dv = reinterpret_cast<u4*>(c.v) + at;
  for (int j = lane; j < n; j += 64) {
    const int h = j >> hs, d = (j & ((1 << hs) - 1)) * 8;
    const u4 x = *reinterpret_cast<const u4*>(a.k + t * a.k_token + h * a.k_head + d);
    const u4 y = *reinterpret_cast<const u4*>(a.v + t * a.v_token + h * a.v_head + d);
    dk[j] = x;
    dv[j] = y;
  }
}

// ---------------------------------------------------------------------------
// fork
// ---------------------------------------------------------------------------

// Workgroup x: old row x's references (children - 1 for every full page; a
// childless row's partial page too), and new row x's table, length and the
// page that it has to copy.  Reference counts change by atomic adds, whose
// order does not change the sum.
__global__ void __launch_bounds__(256) kv_fork_rows_kernel(KvArgs c, const int32_t* parents, KvArgs out, KvScratch w) {
  __shared__ int cnt_s, earlier_s;
  const int x = blockIdx.x;
  const int page = 1 << c.page_shift;
  auto parent = [&](int i) {
    const int p = parents[i];
    return (unsigned)p < (unsigned)c.rows ? p : -1;
  };
  const int mine = x < out.rows ? parent(x) : -1;
  if (threadIdx.x == 0) cnt_s = 0, earlier_s = 0;
  __syncthreads();
  int cnt = 0, earlier = 0;
  for (int i = threadIdx.x; i < out.rows; i += 256) {
    const int p = parent(i);
    cnt += p == x;
    earlier += i < x && p == mine;
  }
  if (cnt) atomicAdd(&cnt_s, cnt);
  if (earlier) atomicAdd(&earlier_s, earlier);
  __syncthreads();
  auto whole = [&](int len) { return len < 0 ? 0 : min(len >> c.page_shift, c.max_pages); };
  if (x < c.rows && cnt_s != 1) {
    const int len = c.lens[x], full = whole(len);
    const bool part = len > 0 && (len & (page - 1)) && full < c.max_pages;
    for (int i = threadIdx.x; i < full + (part && cnt_s == 0); i += 256) {
      const int p = c.tables[(int64_t)x * c.max_pages + i];
      if ((unsigned)p < (unsigned)c.pages) atomicAdd(&c.refs[p], cnt_s - 1);
    }
  }
  if (x < out.rows) {
    int len = 0, keep = 0, src = -1;
    if (mine >= 0) {
      len = max(c.lens[mine], 0);
      const int full = whole(len);
      const bool part = (len & (page - 1)) && full < c.max_pages;
      keep = full + (part && !earlier_s);  // table entries taken over
      if (part && earlier_s) {
        const int p = c.tables[(int64_t)mine * c.max_pages + full];
        src = (unsigned)p < (unsigned)c.pages ? p : -1;
        if (src < 0) len = full << c.page_shift;
      }
    }
    for (int i = threadIdx.x; i < out.max_pages; i += 256)
      out.tables[(int64_t)x * out.max_pages + i] = i < keep ? c.tables[(int64_t)mine * c.max_pages + i] : -1;
    if (threadIdx.x == 0) {
      out.lens[x] = len;
      w.src[x] = src;
      if (mine < 0 && parents[x] != -1) atomicOr(c.status, KV_BAD_INDEX);
    }
  }
}

// One workgroup: a fresh page for every row that copies, in row order.
__global__ void __launch_bounds__(SCAN) kv_fork_pages_kernel(KvArgs c, KvArgs out, KvScratch w) {
  __shared__ int red[SCAN / 64];
  __shared__ uint32_t sums[SCAN / 64];
  int want = 0;
  for (int b0 = 0; b0 < out.rows; b0 += SCAN) {
    const int b = b0 + threadIdx.x;
    uint32_t total;
    block_scan(b < out.rows && w.src[b] >= 0, total, sums);
    want += total;
  }
  if (!want) return;
  const int got = find_free(c.refs, c.pages, want, w.free_list, red);
  int given = 0;
  for (int b0 = 0; b0 < out.rows; b0 += SCAN) {
    const int b = b0 + threadIdx.x;
    const bool copy = b < out.rows && w.src[b] >= 0;
    uint32_t total;
    const int at = given + (int)block_scan(copy, total, sums);
    given += total;
    if (copy) {
      const int full = out.lens[b] >> c.page_shift;
      if (at < got) {
        const int p = w.free_list[at];
        w.dst[b] = p;
        c.refs[p] = 1;
        out.tables[(int64_t)b * out.max_pages + full] = p;
      } else {
        w.src[b] = -1;
        out.lens[b] = full << c.page_shift;
      }
    }
  }
  if (threadIdx.x == 0 && got < want) atomicOr(c.status, KV_NO_PAGES);
}

// kv_fork_rows_kernel and kv_fork_pages_kernel in one workgroup, a thread per
// table entry: for few entries, where the second launch costs more.
constexpr int FORK_ROWS = 256;
__global__ void __launch_bounds__(SCAN) kv_fork_small_kernel(KvArgs c, const int32_t* parents, KvArgs out, KvScratch w) {
  __shared__ int red[SCAN / 64];
  __shared__ uint32_t sums[SCAN / 64];
  // of the old rows: children, length; of the new rows: parent, and whether an
  // earlier new row has it too
  __shared__ int kids[FORK_ROWS], lens[FORK_ROWS], par[FORK_ROWS], later[FORK_ROWS], list[FORK_ROWS];
  const int page = 1 << c.page_shift, x = threadIdx.x;
  if (x < FORK_ROWS) {
    kids[x] = 0;
    lens[x] = x < c.rows ? max(c.lens[x], 0) : 0;
    const int p = x < out.rows ? parents[x] : -1;
    par[x] = (unsigned)p < (unsigned)c.rows ? p : -1;
    if (p != -1 && par[x] < 0) atomicOr(c.status, KV_BAD_INDEX);
  }
  __syncthreads();
  if (x < out.rows && par[x] >= 0) {
    atomicAdd(&kids[par[x]], 1);
    int e = 0;
    for (int i = 0; i < x; ++i) e |= par[i] == par[x];
    later[x] = e;
  }
  __syncthreads();
  auto full_of = [&](int len) { return min(len >> c.page_shift, c.max_pages); };
  auto part_of = [&](int len) { return (len & (page - 1)) && full_of(len) < c.max_pages; };
  int len = 0, src = -1;  // of new row x
  if (x < out.rows && par[x] >= 0) {
    len = lens[par[x]];
    if (part_of(len) && later[x]) {
      const int p = c.tables[(int64_t)par[x] * c.max_pages + full_of(len)];
      src = (unsigned)p < (unsigned)c.pages ? p : -1;
      if (src < 0) len = full_of(len) << c.page_shift;
    }
  }
  const int rows = max(c.rows, out.rows), entries = rows * c.max_pages;
  for (int e = x; e < entries; e += SCAN) {
    const int b = e / c.max_pages, i = e - b * c.max_pages;
    if (b < c.rows && kids[b] != 1) {
      const int full = full_of(lens[b]);
      if (i < full || (i == full && part_of(lens[b]) && kids[b] == 0)) {
        const int p = c.tables[e];
        if ((unsigned)p < (unsigned)c.pages) atomicAdd(&c.refs[p], kids[b] - 1);
      }
    }
    if (b < out.rows && !(par[b] >= 0 && later[b] && i == full_of(lens[par[b]]))) {
      int entry = -1;
      if (par[b] >= 0) {
        const int n = lens[par[b]], full = full_of(n);
        if (i < full || (i == full && part_of(n))) entry = c.tables[(int64_t)par[b] * c.max_pages + i];
      }
      out.tables[e] = entry;
    }
  }
  // the counts have to be in memory (this XCD's cache) before they are
  // searched: every wave waits for its atomics, then all for one another
  __builtin_amdgcn_s_waitcnt(0x0F70);  // vmcnt 0
  uint32_t copies;
  const int at = (int)block_scan(src >= 0, copies, sums), want = (int)copies;
  const int got = want ? find_free(c.refs, c.pages, want, list, red) : 0;
  // (a later child's entry for its partial page is written here alone)
  if (x < out.rows) {
    int fresh = -1;
    if (src >= 0) {
      if (at < got) {
        fresh = list[at];
        c.refs[fresh] = 1;
        w.dst[x] = fresh;
      } else {
        src = -1;
        len = full_of(len) << c.page_shift;
      }
    }
    if (par[x] >= 0 && later[x] && full_of(lens[par[x]]) < out.max_pages)
      out.tables[(int64_t)x * out.max_pages + full_of(lens[par[x]])] = fresh;
    out.lens[x] = len;
    w.src[x] = src;
  }
  if (x == 0 && got < want) atomicOr(c.status, KV_NO_PAGES);
}

// Copies the tokens of the pages that kv_fork_pages_kernel gave out: grid
// (pieces of one token over all layers, keys and values; rows).  A thread
// moves its 16-byte piece of every token, four at a time in flight.  Behind the
// pieces, in a cache of 8 bits, a thread per layer, key or value and head moves
// the exponents of the page's blocks.
__global__ void __launch_bounds__(256) kv_fork_copy_kernel(KvArgs c, KvArgs out, KvScratch w, int n) {
  const int b = blockIdx.y, src = w.src[b];
  if (src < 0) return;
  const int64_t j = (int64_t)blockIdx.x * 256 + threadIdx.x;
  const int tokens = out.lens[b] & ((1 << c.page_shift) - 1);
  const int64_t more = j - (int64_t)2 * c.layers * n;
  if (more >= 0) {
    if (!c.k_exps || more >= (int64_t)2 * c.layers * c.heads_kv) return;
    const int r = (int)(more % (2 * c.heads_kv)), blocks = (1 << c.page_shift) / KV_BLOCK;
    uint8_t* exps = (r < c.heads_kv ? c.k_exps : c.v_exps) + r % c.heads_kv;
    const int64_t base = more / (2 * c.heads_kv) * c.pages;
    for (int i = 0; i * KV_BLOCK < tokens; ++i)
      exps[((base + w.dst[b]) * blocks + i) * c.heads_kv] = exps[((base + src) * blocks + i) * c.heads_kv];
    return;
  }
  const int layer = (int)(j / (2 * n)), r = (int)(j % (2 * n));
  u4* pool = reinterpret_cast<u4*>(r < n ? c.k : c.v);
  const int64_t base = (int64_t)layer * c.pages;
  const u4* from = pool + ((base + src) << c.page_shift) * n + (r < n ? r : r - n);
  u4* to = pool + ((base + w.dst[b]) << c.page_shift) * n + (r < n ? r : r - n);
  int t = 0;
  for (; t + 4 <= tokens; t += 4) {
    u4 x[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) x[i] = from[(int64_t)(t + i) * n];
#pragma unroll
    for (int i = 0; i < 4; ++i) to[(int64_t)(t + i) * n] = x[i];
  }
  for (; t < tokens; ++t) to[(int64_t)t * n] = from[(int64_t)t * n];
}

// ---------------------------------------------------------------------------
// compact
// ---------------------------------------------------------------------------

// The kept tokens of a row and whether the row can be compacted at all, from the
// state before the call, so that every wave of a row comes to the same answer.
struct Kept {
  const KvArgs& c;
  const int32_t *keep, *table;
  int pos, count, len, inside;
  bool sound;
  __device__ __forceinline__ Kept(const KvArgs& c, const int32_t* pos_, const int32_t* keep_, int max_keep,
                                  const int32_t* count_, int b)
      : c(c), keep(keep_ + (int64_t)b * max_keep), table(c.tables + (int64_t)b * c.max_pages), pos(pos_[b]), count(count_[b]),
        len(c.lens[b]), inside((1 << c.page_shift) - 1) {
    // (the kept ones are ascending and inside the row, so there are no more of
    // them than tokens, and no position below passes 32 bits)
    sound = pos >= 0 && count >= 0 && count <= max_keep && pos <= len && count <= len - pos &&
            pages_of(len, c.page_shift) <= c.max_pages;
  }
  // token t of the kept ones: its source and destination in the pool (in
  // tokens), and what is wrong with it
  __device__ __forceinline__ int look(int t, int64_t& from, int64_t& to) const {
    from = to = 0;
    if (!sound || t >= count) return 0;
    const int s = keep[t], before = t ? keep[t - 1] : -1, p = pos + t;
    const int dg = p >> c.page_shift;
    const int dst = dg < c.max_pages ? table[dg] : -1;
    if (s <= before || s >= len - pos) return KV_BAD_INDEX;
    // the page of a token that moves, or of the last one where the row ends
    // inside it, may not be another row's too
    const int src = s == t ? dst : table[(pos + s) >> c.page_shift];
    const bool uses = s != t || (t == count - 1 && (p + 1) & inside);
    if (uses && ((unsigned)dst >= (unsigned)c.pages || (unsigned)src >= (unsigned)c.pages)) return KV_BAD_INDEX;
    if (uses && c.refs[dst] > 1) return KV_SHARED;
    from = ((int64_t)src << c.page_shift) + ((pos + s) & inside);
    to = ((int64_t)dst << c.page_shift) + (p & inside);
    return 0;
  }
  // Looks all kept tokens up, a lane each; the first 64 stay looked up.  Returns
  // the bits to report, and whether the row is compacted.
  __device__ __forceinline__ int decide(int lane, int64_t& from, int64_t& to, bool& ok) const {
    int wrong = 0;
    for (int t0 = 64; t0 < count && sound; t0 += 64) wrong |= look(t0 + lane, from, to);
    wrong |= look(lane, from, to);
    if (sound && count == 0 && pos & inside) {  // ends inside a page that stays
      const int page = table[pos >> c.page_shift];
      if ((unsigned)page >= (unsigned)c.pages) wrong |= KV_BAD_INDEX;
      else if (c.refs[page] > 1) wrong |= KV_SHARED;
    }
    int bad = __ballot(wrong & KV_BAD_INDEX) ? KV_BAD_INDEX : __ballot(wrong & KV_SHARED) ? KV_SHARED : 0;
    if (!sound) bad = pos == -1 ? 0 : KV_BAD_INDEX;
    ok = sound && !bad;
    return bad;
  }
};

// Moves the kept tokens: grid (pieces of one token over all layers, keys and
// values; rows).  Lane j of every wave looks up kept token j (64 at a time):
// where it is and goes, and whether the row can be compacted at all; the first
// workgroup of a row leaves that for the next kernel.  Then a thread moves its
// 16-byte piece of every token in order, eight at a time: keep is strictly
// ascending, so the places that a batch writes (up to pos + j + 7) are never
// sources of a later one (from pos + j + 8 on).
__global__ void __launch_bounds__(256) kv_compact_move_kernel(KvArgs c, const int32_t* pos_, const int32_t* keep_,
                                                              int max_keep, const int32_t* count_, KvScratch w, int n) {
  const int b = blockIdx.y, lane = threadIdx.x & 63;
  const Kept kept(c, pos_, keep_, max_keep, count_, b);
  const int count = kept.count;
  int64_t from, to;
  bool ok;
  const int bad = kept.decide(lane, from, to, ok);
  if (blockIdx.x == 0 && threadIdx.x == 0) {
    w.src[b] = ok;
    if (bad) atomicOr(c.status, bad);
  }
  if (!ok) return;
  const int64_t j = (int64_t)blockIdx.x * 256 + threadIdx.x;
  const bool mine = j < (int64_t)2 * c.layers * n;
  const int layer = (int)(j / (2 * n)), r = (int)(j % (2 * n));
  u4* pool = reinterpret_cast<u4*>(r < n ? c.k : c.v) + (((int64_t)(mine ? layer : 0) * c.pages) << c.page_shift) * n +
             (r < n ? r : r - n);
  for (int t0 = 0; t0 < count; t0 += 64) {
    if (t0) kept.look(t0 + lane, from, to);
    const int m = min(64, count - t0);
    for (int i0 = 0; i0 < m; i0 += 8) {
      u4 x[8];
      int64_t f[8], d[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        f[i] = __shfl((long long)from, i0 + i);
        d[i] = __shfl((long long)to, i0 + i);
        if (mine && i0 + i < m && f[i] != d[i]) x[i] = pool[f[i] * n];
      }
#pragma unroll
      for (int i = 0; i < 8; ++i)
        if (mine && i0 + i < m && f[i] != d[i]) pool[d[i] * n] = x[i];
    }
  }
}

// The same for a cache of 8 bits: a wave has `group` heads of the keys or values
// of one layer and row (grid: layer, keys or values, heads in waves; rows), and
// takes the row's blocks from pos on in order, 16 tokens at once: it reads the
// codes of all a block's tokens and the exponents that they are under, then
// writes them under the largest.  Places written lie before all later sources,
// as above.  A block none of whose tokens moves stays.
template <int D>
__global__ void __launch_bounds__(256) kv_compact_move8_kernel(KvArgs c, const int32_t* pos_, const int32_t* keep_,
                                                               int max_keep, const int32_t* count_, KvScratch w, int group) {
  constexpr int U = D / 16, TP = 64 / U, PASSES = KV_BLOCK / TP;
  const int b = blockIdx.y, lane = threadIdx.x & 63;
  const Kept kept(c, pos_, keep_, max_keep, count_, b);
  int64_t from, to;
  bool ok;
  const int bad = kept.decide(lane, from, to, ok);
  if (blockIdx.x == 0 && threadIdx.x == 0) {
    w.src[b] = ok;
    if (bad) atomicOr(c.status, bad);
  }
  if (!ok) return;
  const int parts = (c.heads_kv + group - 1) / group;
  const int64_t wave = (int64_t)blockIdx.x * 4 + __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  if (wave >= (int64_t)2 * c.layers * parts) return;
  const int layer = (int)(wave / (2 * parts)), which = (int)(wave % (2 * parts)) / parts, h0 = (int)(wave % parts) * group;
  const int64_t base = ((int64_t)layer * c.pages) << c.page_shift;
  uint8_t* codes = reinterpret_cast<uint8_t*>(which ? c.v : c.k) + base * c.heads_kv * D;
  uint8_t* exps = (which ? c.v_exps : c.k_exps) + base / KV_BLOCK * c.heads_kv;
  const int end = kept.pos + kept.count;
  for (int first = kept.pos & ~(KV_BLOCK - 1); first < end; first += KV_BLOCK) {
    // the lane's tokens of the block: from, to (-1: none)
    int64_t f[PASSES], t[PASSES];
    bool moves = false;
#pragma unroll
    for (int x = 0; x < PASSES; ++x) {
      const int p = first + TP * x + lane / U;
      f[x] = t[x] = -1;
      if (p < kept.pos) {
        f[x] = t[x] = ((int64_t)kept.table[p >> c.page_shift] << c.page_shift) + (p & kept.inside);
      } else if (p < end) {
        kept.look(p - kept.pos, f[x], t[x]);
        if (kept.keep[p - kept.pos] == p - kept.pos) {  // (looked up only where it has to be)
          f[x] = t[x] = ((int64_t)kept.table[p >> c.page_shift] << c.page_shift) + (p & kept.inside);
        } else {
          moves = true;
        }
      }
    }
    if (!__any(moves)) continue;
    const int64_t pool = (int64_t)c.pages << c.page_shift;
    for (int h = h0; h < min(h0 + group, c.heads_kv); ++h) {
      u4 v[PASSES];
      int e[PASSES], most = 1;
#pragma unroll
      for (int x = 0; x < PASSES; ++x) {
        e[x] = 1;
        if ((uint64_t)f[x] >= (uint64_t)pool || (uint64_t)t[x] >= (uint64_t)pool) continue;
        v[x] = *reinterpret_cast<const u4*>(codes + (f[x] * c.heads_kv + h) * D + 16 * (lane % U));
        e[x] = (int)exp_of(exps[f[x] / KV_BLOCK * c.heads_kv + h]);
        most = max(most, e[x]);
      }
#pragma unroll
      for (int d = U; d < 64; d <<= 1) most = max(most, __shfl_xor(most, d));
#pragma unroll
      for (int x = 0; x < PASSES; ++x) {
        if ((uint64_t)f[x] >= (uint64_t)pool || (uint64_t)t[x] >= (uint64_t)pool) continue;
        const float by = exp_ratio(e[x], most);
#pragma unroll
        for (int i = 0; i < 4; ++i) v[x][i] = e[x] == most ? v[x][i] : rescale4(v[x][i], by);
        if (f[x] != t[x] || e[x] != most) *reinterpret_cast<u4*>(codes + (t[x] * c.heads_kv + h) * D + 16 * (lane % U)) = v[x];
        if (lane % U == 0) exps[t[x] / KV_BLOCK * c.heads_kv + h] = (uint8_t)most;
      }
    }
  }
}

// One workgroup per row: gives back the pages past the row's new end.
__global__ void __launch_bounds__(64) kv_compact_rows_kernel(KvArgs c, const int32_t* pos, const int32_t* count,
                                                             KvScratch w) {
  const int b = blockIdx.x;
  if (!w.src[b]) return;
  const int end = pos[b] + count[b], len = c.lens[b];
  int32_t* table = c.tables + (int64_t)b * c.max_pages;
  for (int i = pages_of(end, c.page_shift) + (int)threadIdx.x; i < pages_of(len, c.page_shift); i += 64) {
    const int p = table[i];
    if ((unsigned)p < (unsigned)c.pages) atomicAdd(&c.refs[p], -1);
    table[i] = -1;
  }
  __syncthreads();
  if (threadIdx.x == 0) c.lens[b] = end;
}

int pieces(const KvArgs& c) { return c.heads_kv * c.head_dim / (c.k_exps ? 16 : 8); }
unsigned piece_blocks(const KvArgs& c) {
  const int64_t exps = c.k_exps ? c.heads_kv : 0;  // (the threads of kv_fork_copy_kernel that move exponents)
  return (unsigned)((2 * c.layers * (pieces(c) + exps) + 255) / 256);
}

}  // namespace

hipError_t launch_kv_reserve(const KvArgs& c, const int32_t* cu, int32_t* pos, const KvScratch& w, hipStream_t s) {
  hipLaunchKernelGGL(kv_reserve_kernel, dim3(1), dim3(SCAN), 0, s, c, cu, pos, w);
  return hipGetLastError();
}

hipError_t launch_kv_write(const KvWriteArgs& a, hipStream_t s) {
  hipLaunchKernelGGL(kv_write_kernel, dim3((unsigned)((a.tokens + 3) / 4)), dim3(256), 0, s, a);
  return hipGetLastError();
}

hipError_t launch_kv_fork(const KvArgs& c, const int32_t* parents, const KvArgs& out, const KvScratch& w,
                          hipStream_t s) {
  const int rows = c.rows > out.rows ? c.rows : out.rows;
  // (up to 16 entries a thread)
  const bool small = rows <= FORK_ROWS && (int64_t)rows * c.max_pages <= 16 * SCAN;
  if (small) hipLaunchKernelGGL(kv_fork_small_kernel, dim3(1), dim3(SCAN), 0, s, c, parents, out, w);
  else hipLaunchKernelGGL(kv_fork_rows_kernel, dim3((unsigned)rows), dim3(256), 0, s, c, parents, out, w);
  if (out.rows) {
    if (!small) hipLaunchKernelGGL(kv_fork_pages_kernel, dim3(1), dim3(SCAN), 0, s, c, out, w);
    hipLaunchKernelGGL(kv_fork_copy_kernel, dim3(piece_blocks(c), (unsigned)out.rows), dim3(256), 0, s, c, out, w,
                       pieces(c));
  }
  return hipGetLastError();
}

hipError_t launch_kv_compact(const KvArgs& c, const int32_t* pos, const int32_t* keep, int max_keep,
                             const int32_t* count, const KvScratch& w, hipStream_t s) {
  if (c.k_exps) {
    // (heads that a wave takes with one look at the kept tokens: as many as
    // leave enough waves.  8 heads: 32 rows of 32 layers 7.9 us, with 1 head a
    // wave 12.7, with 8 9.4; 16 rows of 80 layers 10.8, 18.3 and 15; one row of
    // 32 layers 8 with any)
    int group = 1;
    while (group < 8 && group < c.heads_kv && (int64_t)c.rows * c.layers * c.heads_kv / group >= 4096) group *= 2;
    const int64_t waves = (int64_t)2 * c.layers * ((c.heads_kv + group - 1) / group);
    const dim3 grid((unsigned)((waves + 3) / 4), (unsigned)c.rows);
    if (c.head_dim == 128)
      hipLaunchKernelGGL(kv_compact_move8_kernel<128>, grid, dim3(256), 0, s, c, pos, keep, max_keep, count, w, group);
    else hipLaunchKernelGGL(kv_compact_move8_kernel<64>, grid, dim3(256), 0, s, c, pos, keep, max_keep, count, w, group);
  } else {
    hipLaunchKernelGGL(kv_compact_move_kernel, dim3(piece_blocks(c), (unsigned)c.rows), dim3(256), 0, s, c, pos, keep,
                       max_keep, count, w, pieces(c));
  }
  hipLaunchKernelGGL(kv_compact_rows_kernel, dim3((unsigned)c.rows), dim3(64), 0, s, c, pos, count, w);
  return hipGetLastError();
}

}  // namespace qg
