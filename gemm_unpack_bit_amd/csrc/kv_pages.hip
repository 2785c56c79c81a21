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
#include "attn.hpp"
#include "rows.hpp"

namespace qg {
namespace {

constexpr int SCAN = 1024;  // threads of the one-workgroup kernels

// Exclusive prefix sum over the workgroup's SCAN threads; total in all.
__device__ __forceinline__ int block_scan(int v, int& total, int* red) {
  const int lane = threadIdx.x & 63, w = threadIdx.x >> 6;
  int s = v;
#pragma unroll
  for (int d = 1; d < 64; d <<= 1) {
    const int o = __shfl_up(s, d);
    if (lane >= d) s += o;
  }
  if (lane == 63) red[w] = s;
  __syncthreads();
  int before = 0, all = 0;
#pragma unroll
  for (int i = 0; i < SCAN / 64; ++i) {
    const int x = red[i];
    before += i < w ? x : 0;
    all += x;
  }
  __syncthreads();
  total = all;
  return before + s - v;
}

// The lowest `want` free pages into list, in order; returns how many there are
// (<= want).  All threads of the workgroup; ends with a barrier, so list can
// be read by any of them.
__device__ __forceinline__ int find_free(const int32_t* refs, int pages, int want, int32_t* list, int* red) {
  int found = 0;
  for (int p0 = 0; p0 < pages && found < want; p0 += 8 * SCAN) {
    const int p = p0 + 8 * (int)threadIdx.x;
    uint32_t free = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (p + i < pages && refs[p + i] == 0) free |= 1u << i;
    int total;
    int at = found + block_scan(__builtin_popcount(free), total, red);
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (free >> i & 1) {
        if (at < want) list[at] = p + i;
        ++at;
      }
    found += total;
  }
  __threadfence_block();
  __syncthreads();
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
  int64_t want = 0;
  for (int b0 = 0; b0 < c.rows; b0 += SCAN) {
    int total;
    block_scan(row(b0 + threadIdx.x).need, total, red);
    want += total;
  }
  const int got = want ? find_free(c.refs, c.pages, want < c.pages ? (int)want : c.pages, w.free_list, red) : 0;
  int64_t given = 0;
  int status = 0;
  for (int b0 = 0; b0 < c.rows; b0 += SCAN) {
    const int b = b0 + threadIdx.x;
    const Row r = row(b);
    int total;
    const int64_t at = given + block_scan(r.need, total, red);
    given += total;
    const bool fits = r.need == 0 || at + r.need <= got;
    const bool ok = b < c.rows && !r.bad && fits;
    at_s[threadIdx.x] = (int)at;
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
  int want = 0;
  for (int b0 = 0; b0 < out.rows; b0 += SCAN) {
    const int b = b0 + threadIdx.x;
    int total;
    block_scan(b < out.rows && w.src[b] >= 0, total, red);
    want += total;
  }
  if (!want) return;
  const int got = find_free(c.refs, c.pages, want, w.free_list, red);
  int given = 0;
  for (int b0 = 0; b0 < out.rows; b0 += SCAN) {
    const int b = b0 + threadIdx.x;
    const bool copy = b < out.rows && w.src[b] >= 0;
    int total;
    const int at = given + block_scan(copy, total, red);
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

// Copies the tokens of the pages that kv_fork_pages_kernel gave out: grid
// (pieces of one token over all layers, keys and values; rows).  A thread
// moves its 16-byte piece of every token, four at a time in flight.
__global__ void __launch_bounds__(256) kv_fork_copy_kernel(KvArgs c, KvArgs out, KvScratch w, int n) {
  const int b = blockIdx.y, src = w.src[b];
  if (src < 0) return;
  const int64_t j = (int64_t)blockIdx.x * 256 + threadIdx.x;
  if (j >= (int64_t)2 * c.layers * n) return;
  const int tokens = out.lens[b] & ((1 << c.page_shift) - 1);
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

// Whether row b can be compacted, from the state before the call; every
// thread of the workgroup gets the same answer and `bad` the reason.
__device__ __forceinline__ bool compactable(const KvArgs& c, int b, int pos, int count, const int32_t* keep,
                                            int max_keep, int& bad) {
  bad = 0;
  if (pos < 0) {
    bad = pos < -1 ? KV_BAD_INDEX : 0;
    return false;
  }
  const int len = c.lens[b];
  if (count < 0 || count > max_keep || pos > len || pages_of(len, c.page_shift) > c.max_pages) {
    bad = KV_BAD_INDEX;
    return false;
  }
  int wrong = 0;
  for (int j = threadIdx.x & 63; j < count; j += 64) {
    const int s = keep[j], before = j ? keep[j - 1] : -1;
    if (s <= before || s >= len - pos) wrong |= KV_BAD_INDEX;
    // the page of a token that moves, or of the last one where the row ends
    // inside it, may not be another row's too
    const int p = pos + j;
    if (s != j || (j == count - 1 && (p + 1) & ((1 << c.page_shift) - 1))) {
      const int g = p >> c.page_shift;
      const int page = g < c.max_pages ? c.tables[(int64_t)b * c.max_pages + g] : -1;
      if ((unsigned)page >= (unsigned)c.pages) wrong |= KV_BAD_INDEX;
      else if (c.refs[page] > 1) wrong |= KV_SHARED;
    }
  }
  if (count == 0 && pos & ((1 << c.page_shift) - 1)) {
    const int page = c.tables[(int64_t)b * c.max_pages + (pos >> c.page_shift)];
    if ((unsigned)page >= (unsigned)c.pages) wrong |= KV_BAD_INDEX;
    else if (c.refs[page] > 1) wrong |= KV_SHARED;
  }
  bad = __ballot(wrong & KV_BAD_INDEX) ? KV_BAD_INDEX : __ballot(wrong & KV_SHARED) ? KV_SHARED : 0;
  return !bad;
}

// Moves the kept tokens: grid (pieces of one token over all layers, keys and
// values; rows).  A thread moves its 16-byte piece of every token in order,
// eight at a time: keep is strictly ascending, so the places that a batch
// writes (up to pos + j + 7) are never sources of a later one (from
// pos + j + 8 on).  The first workgroup of a row leaves the decision for the
// next kernel.
__global__ void __launch_bounds__(256) kv_compact_move_kernel(KvArgs c, const int32_t* pos_, const int32_t* keep_,
                                                              int max_keep, const int32_t* count_, KvScratch w, int n) {
  const int b = blockIdx.y;
  const int pos = pos_[b], count = count_[b];
  const int32_t* keep = keep_ + (int64_t)b * max_keep;
  int bad;
  const bool ok = compactable(c, b, pos, count, keep, max_keep, bad);
  if (blockIdx.x == 0 && threadIdx.x == 0) {
    w.src[b] = ok;
    if (bad) atomicOr(c.status, bad);
  }
  const int64_t j = (int64_t)blockIdx.x * 256 + threadIdx.x;
  if (!ok || j >= (int64_t)2 * c.layers * n) return;
  const int layer = (int)(j / (2 * n)), r = (int)(j % (2 * n));
  u4* pool = reinterpret_cast<u4*>(r < n ? c.k : c.v) + (((int64_t)layer * c.pages) << c.page_shift) * n + (r < n ? r : r - n);
  const int32_t* table = c.tables + (int64_t)b * c.max_pages;
  const int inside = (1 << c.page_shift) - 1;
  for (int t0 = 0; t0 < count; t0 += 8) {
    u4 x[8];
    const int m = min(8, count - t0);
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (i < m && keep[t0 + i] != t0 + i) {
        const int p = pos + keep[t0 + i], page = table[p >> c.page_shift];
        if ((unsigned)page < (unsigned)c.pages) x[i] = pool[(((int64_t)page << c.page_shift) + (p & inside)) * n];
      }
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (i < m && keep[t0 + i] != t0 + i) {
        const int p = pos + t0 + i, page = table[p >> c.page_shift];
        if ((unsigned)page < (unsigned)c.pages) pool[(((int64_t)page << c.page_shift) + (p & inside)) * n] = x[i];
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

int pieces(const KvArgs& c) { return c.heads_kv * c.head_dim / 8; }
unsigned piece_blocks(const KvArgs& c) { return (unsigned)(((int64_t)2 * c.layers * pieces(c) + 255) / 256); }

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
  hipLaunchKernelGGL(kv_fork_rows_kernel, dim3((unsigned)rows), dim3(256), 0, s, c, parents, out, w);
  if (out.rows) {
    hipLaunchKernelGGL(kv_fork_pages_kernel, dim3(1), dim3(SCAN), 0, s, c, out, w);
    hipLaunchKernelGGL(kv_fork_copy_kernel, dim3(piece_blocks(c), (unsigned)out.rows), dim3(256), 0, s, c, out, w,
                       pieces(c));
  }
  return hipGetLastError();
}

hipError_t launch_kv_compact(const KvArgs& c, const int32_t* pos, const int32_t* keep, int max_keep,
                             const int32_t* count, const KvScratch& w, hipStream_t s) {
  hipLaunchKernelGGL(kv_compact_move_kernel, dim3(piece_blocks(c), (unsigned)c.rows), dim3(256), 0, s, c, pos, keep,
                     max_keep, count, w, pieces(c));
  hipLaunchKernelGGL(kv_compact_rows_kernel, dim3((unsigned)c.rows), dim3(64), 0, s, c, pos, count, w);
  return hipGetLastError();
}

}  // namespace qg
