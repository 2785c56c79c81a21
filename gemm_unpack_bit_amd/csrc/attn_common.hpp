// Device parts shared by the attention kernels: element types, the split of
// the key axis over workgroups, visibility of keys, and the store of a tile's
// result or partial result.
#pragma once

#include "attn.hpp"
#include "rows.hpp"

namespace qg {

typedef __bf16 b2v __attribute__((ext_vector_type(2)));
typedef __bf16 b8v __attribute__((ext_vector_type(8)));
typedef float f2v __attribute__((ext_vector_type(2)));

// Element types.  LIFT: the softmax weights are held 2^LIFT times too large, as
// are their sums, which cancels in the quotient; in fp16, whose normal numbers
// end at 2^-14, weights down to 2^-24 of the largest then keep all their bits.
// SLACK: the weights' reference m may lie that far (in powers of two) below the
// largest score before sums are rescaled to a new one, so that after the first
// few tiles they hardly ever are; the largest weight, 2^(LIFT + SLACK), still
// is a normal fp16 number.  In bf16 it is 1 (weights down to 2^-118 of it stay
// normal), so that sums of values near the type's largest overflow no sooner
// than with weights from the largest score.
// pack rounds two floats to nearest even; NONFINITE_* find
// halves whose exponent is all ones: ((w & EXP) + ONE) has bit 15 of such a
// half set, and the addition never carries into the next half.
struct F16 {
  static constexpr uint32_t EXP = 0x7C007C00u, ONE = 0x04000400u;
  static constexpr float LIFT = 10.f, SLACK = 5.f;
  static __device__ __forceinline__ uint32_t pack(float a, float b) {
    return __builtin_bit_cast(uint32_t, __builtin_convertvector(f2v{a, b}, h2));
  }
  static __device__ __forceinline__ float value(uint16_t x) { return h2f(x); }
  static __device__ __forceinline__ f4 mfma16(u4 a, u4 b, f4 c) {
    return __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(h8, a), __builtin_bit_cast(h8, b), c, 0, 0, 0);
  }
  static __device__ __forceinline__ f16v mfma32(u4 a, u4 b, f16v c) {
    return __builtin_amdgcn_mfma_f32_32x32x16_f16(__builtin_bit_cast(h8, a), __builtin_bit_cast(h8, b), c, 0, 0, 0);
  }
};
struct BF16 {
  static constexpr uint32_t EXP = 0x7F807F80u, ONE = 0x00800080u;
  static constexpr float LIFT = -8.f, SLACK = 8.f;
  static __device__ __forceinline__ uint32_t pack(float a, float b) {
    return __builtin_bit_cast(uint32_t, __builtin_convertvector(f2v{a, b}, b2v));
  }
  static __device__ __forceinline__ float value(uint16_t x) { return __builtin_bit_cast(float, (uint32_t)x << 16); }
  static __device__ __forceinline__ f4 mfma16(u4 a, u4 b, f4 c) {
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(b8v, a), __builtin_bit_cast(b8v, b), c, 0, 0, 0);
  }
  static __device__ __forceinline__ f16v mfma32(u4 a, u4 b, f16v c) {
    return __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(b8v, a), __builtin_bit_cast(b8v, b), c, 0, 0, 0);
  }
};
template <typename E>
__device__ __forceinline__ uint32_t nonfinite(uint32_t w) {  // bits 15 and 31: the halves that are not finite
  return ((w & E::EXP) + E::ONE) & 0x80008000u;
}

__device__ __forceinline__ float exp2_(float x) { return __builtin_amdgcn_exp2f(x); }
constexpr float NEG_INF = -__builtin_inff();
// Whether scores are multiplied by 0 (the same in the whole wave).  A score of
// -inf then is NaN, but would be taken for an unseen key's; so the kernels put
// score - score in its place: 0, or NaN where it is not finite.
__device__ __forceinline__ bool zero_scale(float scale) { return (__float_as_uint(scale) & 0x7FFFFFFFu) == 0; }

// Weights are 2^(x * scale - m), one fused operation a score; their reference m
// is a rounded product.  From 2^16 on its rounding counts (from 2^24 a score may
// lie whole powers of two off its own reference, which made weights overflow or
// vanish), so there the product of every score is rounded likewise and m taken
// off behind it: the largest score's weight is exact, and the others' errors are
// those of the product.  (m of -inf or +inf: no.)
__device__ __forceinline__ bool far(float m) {
  return (__float_as_uint(m) & 0x7FFFFFFFu) - 0x47800000u < 0x7F800000u - 0x47800000u;
}
__device__ __forceinline__ float far_score(float x, float scale, float m) {
#pragma clang fp contract(off)
  const float product = x * scale;
  return product - m;
}

// max and sum over the lanes l, l ^ 32
__device__ __forceinline__ float half_max(float v) {
  const uint32_t u = __float_as_uint(v);
  const auto a = __builtin_amdgcn_permlane32_swap(u, u, false, false);
  return fmaxf(__uint_as_float(a[0]), __uint_as_float(a[1]));
}
__device__ __forceinline__ float half_sum(float v) {
  const uint32_t u = __float_as_uint(v);
  const auto a = __builtin_amdgcn_permlane32_swap(u, u, false, false);
  return __uint_as_float(a[0]) + __uint_as_float(a[1]);
}
// max over the lanes l % 16 + {0, 16, 32, 48}
__device__ __forceinline__ float quarter_max(float v) {
  const uint32_t u = __float_as_uint(half_max(v));
  const auto a = __builtin_amdgcn_permlane16_swap(u, u, false, false);
  return fmaxf(__uint_as_float(a[0]), __uint_as_float(a[1]));
}

// The kernel's AttnArgs (its first argument), read again from the argument
// segment: code outside a hot loop takes its fields from here, so that they do
// not occupy scalar registers during the loop.
__device__ __forceinline__ AttnArgs args_again() {
  typedef __attribute__((address_space(4))) const uint32_t* words;
  words p = (words)__builtin_amdgcn_kernarg_segment_ptr();
  asm volatile("" : "+s"(p));
  struct W {
    uint32_t w[sizeof(AttnArgs) / 4];
  } x;
#pragma unroll
  for (unsigned i = 0; i < sizeof(AttnArgs) / 4; ++i) x.w[i] = p[i];
  return __builtin_bit_cast(AttnArgs, x);
}

// One row (sequence) as the kernels see it.
struct Row {
  int q0, n;    // first query token, number of query tokens
  int pos;      // keys in front of the query tokens (may be negative for packed keys)
  int k0;       // packed keys: first key token
  int keys;     // keys of the row, 0 or more
};
template <bool PAGED>
__device__ __forceinline__ Row row_of(const AttnArgs& a, int b) {
  Row r;
  auto clamp = [](int x, int hi) { return x < 0 ? 0 : x > hi ? hi : x; };
  r.q0 = clamp(a.cu[b], a.tokens);
  r.n = clamp(a.cu[b + 1], a.tokens) - r.q0;
  if (r.n < 0) r.n = 0;
  if constexpr (PAGED) {
    r.pos = a.pos[b];
    r.k0 = 0;
    const int64_t cap = (int64_t)a.max_pages << a.page_shift, end = (int64_t)r.pos + r.n;
    r.keys = r.pos < 0 ? 0 : (int)(end < cap ? end : cap);
  } else {
    r.k0 = clamp(a.cu_k[b], a.tokens_k);
    r.keys = clamp(a.cu_k[b + 1], a.tokens_k) - r.k0;
    if (r.keys < 0) r.keys = 0;
    r.pos = r.keys - r.n;
  }
  return r;
}

// The pool token (page * page_size + place) of position kb of row b, kb in the
// row's table; a page number outside the pool counts as page 0.  b and kb are
// the same in the whole wave, and tables do not change during the kernel, so
// this is a scalar load.
__device__ __forceinline__ int64_t pool_token(const AttnArgs& a, int b, int kb) {
  typedef __attribute__((address_space(4))) const int32_t* table;
  const int page = ((table)a.tables)[(int64_t)b * a.max_pages + (kb >> a.page_shift)];
  return ((int64_t)((unsigned)page < (unsigned)a.pages ? page : 0) << a.page_shift) + (kb & ((1 << a.page_shift) - 1));
}

// What query token t of a row sees: every key below lim, and of the keys from
// pos up to all those whose bit is set in its mask words.  A token that the row
// does not have (t >= n) sees nothing.  No branch here depends on the lane
// (selects do): around the kernels' many live registers, code that only some
// lanes run is where a compiler is most easily led to keep a register for
// those lanes alone.
template <bool PAGED>
struct Sight {
  int lim, all;
  const uint64_t* words;  // (of some token of the row, also for a token that it does not have)
  __device__ __forceinline__ void init(const AttnArgs& a, const Row& r, int t) {
    const bool live = t < r.n;
    all = live ? r.keys : 0;
    words = nullptr;
    if constexpr (PAGED) {
      words = a.mask + (int64_t)(r.q0 + (live ? t : 0)) * a.mask_words;
      lim = a.mask ? r.pos : r.pos + t + 1;
    } else {
      lim = a.causal ? r.pos + t + 1 : r.keys;
    }
    lim = lim < 0 ? 0 : lim > all ? all : lim;
  }
  // bit i: key kb + i is seen, i < 64
  __device__ __forceinline__ uint64_t window(const AttnArgs& a, const Row& r, int kb) const {
    auto below = [](int n) { return n <= 0 ? 0ull : n >= 64 ? ~0ull : (1ull << n) - 1; };
    uint64_t v = below(lim - kb);
    if constexpr (PAGED)
      if (a.mask) {
        const int i0 = kb - r.pos;
        uint64_t m = 0;
        if (i0 >= 0) {
          const int w = i0 >> 6, s = i0 & 63;
          if (w < a.mask_words) m = words[w] >> s;
          if (s && w + 1 < a.mask_words) m |= words[w + 1] << (64 - s);
        } else if (i0 > -64) {
          m = words[0] << -i0;
        }
        v |= m & below(all - kb);
      }
    return v;
  }
};

// Partial results: [slots][BM] (max, sum), then per slot the sums in groups of
// four columns, each group's 32 rows side by side (a wave's store of its 32
// rows is contiguous): [BM / 32][D / 4][32][4].
template <int BM, int D>
struct Partials {
  float *ml, *o;
  __device__ __forceinline__ Partials(float* ws, int64_t slots) : ml(ws), o(ws + slots * BM * 2) {}
  __device__ __forceinline__ float* ml_at(int64_t slot, int row) const { return ml + (slot * BM + row) * 2; }
  // columns 4 c .. 4 c + 3 of a row
  __device__ __forceinline__ f4* o_at(int64_t slot, int row, int c) const {
    return reinterpret_cast<f4*>(o + slot * BM * D) + ((row >> 5) * (D / 4) + c) * 32 + (row & 31);
  }
};

// Joins the partial results of 32 query rows (row0 .. row0 + 31 of the tile) in
// the order of their slots: o = sum 2^(m_i - M) o_i / sum 2^(m_i - M) l_i.  A
// workgroup of 256 threads: a thread has one row and every eighth group of four
// columns of it, so a wave's load is two runs of 512 bytes.
// out(row) is where the row's result goes, NULL if nowhere.
template <typename E, int BM, int D, typename F, typename O>
__device__ __forceinline__ void join_rows(const Partials<BM, D>& p, int row0, int parts, F&& slot, O&& out) {
  constexpr int G = D / 32;  // column groups of a thread
  const int row = row0 + (threadIdx.x & 31), c0 = threadIdx.x >> 5;
  uint16_t* to = out(row);
  if (!to) return;
  float m = NEG_INF, l = 0.f;
  f4 acc[G];
#pragma unroll
  for (int e = 0; e < G; ++e) acc[e] = f4{0.f, 0.f, 0.f, 0.f};
  for (int i = 0; i < parts; i += 2) {
    float mi[2], li[2];
    f4 oi[2][G];
#pragma unroll
    for (int x = 0; x < 2; ++x) {
      const int64_t s = slot(i + x < parts ? i + x : i);
      const float* ml = p.ml_at(s, row);
      mi[x] = i + x < parts ? ml[0] : NEG_INF;
      li[x] = i + x < parts ? ml[1] : 0.f;
#pragma unroll
      for (int e = 0; e < G; ++e) oi[x][e] = *p.o_at(s, row, c0 + 8 * e);
    }
    const float mn = fmaxf(m, fmaxf(mi[0], mi[1]));
    const float base = mn == NEG_INF ? 0.f : mn, w = exp2_(m - base);
    l *= w;
#pragma unroll
    for (int e = 0; e < G; ++e) acc[e] *= w;
#pragma unroll
    for (int x = 0; x < 2; ++x) {
      const float wx = exp2_(mi[x] - base);
      l += wx * li[x];
#pragma unroll
      for (int e = 0; e < G; ++e)
#pragma unroll
        for (int y = 0; y < 4; ++y) acc[e][y] += li[x] == 0.f ? 0.f : wx * oi[x][e][y];  // (no weights: o may be anything)
    }
    m = mn;
  }
  const float inv = l == 0.f ? 0.f : 1.f / l;
#pragma unroll
  for (int e = 0; e < G; ++e)
    *reinterpret_cast<u2*>(to + 4 * (c0 + 8 * e)) =
        u2{E::pack(acc[e][0] * inv, acc[e][1] * inv), E::pack(acc[e][2] * inv, acc[e][3] * inv)};
}

// inclusive sums over the wave's lanes of values < 2^24 (row shifts, then
// broadcasts of the rows' last lanes)
__device__ __forceinline__ uint32_t scan24(uint32_t v) {
#define QG_SCAN(CTRL, ROWS) v += __builtin_amdgcn_update_dpp(0, (int)v, CTRL, ROWS, 0xF, false)
  QG_SCAN(0x111, 0xF);  // row_shr:1
  QG_SCAN(0x112, 0xF);
  QG_SCAN(0x114, 0xF);
  QG_SCAN(0x118, 0xF);
  QG_SCAN(DPP_BCAST15, 0xA);
  QG_SCAN(DPP_BCAST31, 0xC);
#undef QG_SCAN
  return v;
}

// The split of the key axis.  An item is a tile of BM query rows (row
// t * group + g: query token t, head g of the key head's group) of one row and
// key head; its keys are cut into units of KB.  The units of all items, in the
// order row, key head, tile, unit, are shared out evenly: workgroup c takes
// units [c * per, (c + 1) * per), per = ceil(total / workgroups).
// So a long row is worked on by many workgroups and short ones share one,
// whatever the mix, and no workgroup waits for another.  An item that lies in
// one workgroup is finished there; of the others every workgroup leaves a
// partial result (the part that starts with the workgroup's share in slot
// 2 c, one that starts later in slot 2 c + 1), and they are joined in key order.
//
// Neighbouring shares read the same keys (the tiles of a row and key head come
// one after the other) at about the same time, so they belong on one XCD, where
// the second one finds them in the cache: workgroups go to the XCDs round robin,
// and share_of gives each XCD a run of shares.
//
// A wave keeps 64 rows at a time, one per lane, with the running sum of their
// units; up to 64 rows are read once.
constexpr int NXCD = 8;
// (`shares` of them have work; a result past them means none)
__device__ __forceinline__ int share_of(int workgroup, int shares) {
  const int run = (shares + NXCD - 1) / NXCD, in = workgroup / NXCD;
  return in < run ? (workgroup % NXCD) * run + in : shares;
}

// Where one workgroup joins an item's parts, a part costs it some of a unit's
// time, and an item of n units is done soonest in parts of sqrt(n * that): per
// is at least so much, up to LEAST (1: a join that is itself shared out).
template <int BM, int KB, bool PAGED, int LEAST>
struct Walk {
  int64_t total, per;
  int b0;           // the first row held
  Row mine;         // the lane's row
  int64_t incl;     // units of the rows held up to and with the lane's
  int64_t cost;     // units of the lane's row
  int64_t before, all;  // units in front of the rows held, and of the rows held

  static __device__ __forceinline__ int tiles(const AttnArgs& a, const Row& r) { return (r.n * a.group + BM - 1) / BM; }
  // key units of an item; one without keys still has an output to write
  static __device__ __forceinline__ int units(const Row& r) { return r.keys ? (r.keys + KB - 1) / KB : 1; }
  static __device__ __forceinline__ int uniform(int x) { return __builtin_amdgcn_readfirstlane(x); }
  static __device__ __forceinline__ int64_t lane64(int64_t v, int lane) {
    const uint32_t lo = __builtin_amdgcn_readlane((uint32_t)v, lane);
    const uint32_t hi = __builtin_amdgcn_readlane((uint32_t)((uint64_t)v >> 32), lane);
    return (int64_t)((uint64_t)hi << 32 | lo);
  }
  __device__ __forceinline__ void hold(const AttnArgs& a, int first, int64_t sum) {
    b0 = first;
    before = sum;
    const int b = b0 + (threadIdx.x & 63);
    mine = Row{0, 0, 0, 0, 0};
    cost = 0;
    if (b < a.rows) {
      mine = row_of<PAGED>(a, b);
      cost = (int64_t)tiles(a, mine) * a.heads_kv * units(mine);
    }
    incl = ((int64_t)scan24((uint32_t)(cost >> 24)) << 24) + scan24((uint32_t)cost & 0xFFFFFF);
    all = lane64(incl, 63);
  }
  __device__ __forceinline__ void init(const AttnArgs& a, int workgroups) {
    hold(a, 0, 0);
    total = all;
    for (int first = 64; first < a.rows; first += 64) {
      hold(a, first, total);
      total += all;
    }
    per = (total + workgroups - 1) / workgroups;
    if (LEAST > 1 && per < LEAST) {
      const float joined = __builtin_amdgcn_sqrtf((float)(uint32_t)min(total, (int64_t)UINT32_MAX) * a.join_cost);
      const int least = uniform((int)fminf(joined, (float)LEAST));
      if (per < least) per = least;
    }
    if (per < 1) per = 1;
  }
  __device__ __forceinline__ int shares() const { return (int)((total + per - 1) / per); }
  __device__ __forceinline__ Row row(int lane) const {
    Row r;
    r.q0 = __builtin_amdgcn_readlane(mine.q0, lane);
    r.n = __builtin_amdgcn_readlane(mine.n, lane);
    r.pos = __builtin_amdgcn_readlane(mine.pos, lane);
    r.k0 = __builtin_amdgcn_readlane(mine.k0, lane);
    r.keys = __builtin_amdgcn_readlane(mine.keys, lane);
    return r;
  }
  __device__ __forceinline__ int64_t first_of(int lane) const { return before + lane64(incl - cost, lane); }
  // unit u (< total) and what follows it in its item, up to unit u_end: row b,
  // key head h, tile, units [k0, k1) of the item's `of`
  struct Piece {
    Row r;
    int b, h, tile, k0, k1, of;
  };
  __device__ __forceinline__ Piece seek(const AttnArgs& a, int64_t u, int64_t u_end) {
    if (u < before) hold(a, 0, 0);
    while (u >= before + all && b0 + 64 < a.rows) hold(a, b0 + 64, before + all);
    const int lane = __builtin_ctzll(__ballot(u < before + incl) | 1ull << 63);
    Piece p;
    p.b = uniform(b0 + lane);
    p.r = row(lane);
    p.of = uniform(units(p.r));
    const int64_t in = u - first_of(lane), item = in / p.of, left = u_end - u;
    p.k0 = uniform((int)(in - item * p.of));
    p.k1 = uniform((int)(p.k0 + left < p.of ? p.k0 + left : p.of));
    const int n = tiles(a, p.r);
    p.h = uniform((int)(item / n));
    p.tile = uniform((int)(item % n));
    return p;
  }
  // row b, and its first unit
  __device__ __forceinline__ void seek_row(const AttnArgs& a, int b, Row& r, int64_t& first) {
    if (b < b0) hold(a, 0, 0);
    while (b >= b0 + 64) hold(a, b0 + 64, before + all);
    r = row(b - b0);
    first = first_of(b - b0);
  }
  // the row of highest number whose key (ascending over rows, key(0) <= x) is
  // at most x; held(row) gives the key of a row held, key(b) of any row
  template <typename H, typename K>
  __device__ __forceinline__ int find(const AttnArgs& a, int x, H&& held, K&& key) const {
    if (a.rows <= 64) {
      const int b = threadIdx.x & 63;
      const uint64_t m = __ballot(b < a.rows && held(mine, b) <= x);
      return m ? 63 - __builtin_clzll(m) : 0;
    }
    return find_row(a.rows, x, key);
  }
  // the parts of an item whose first unit is u0: how many (1: it lies in one
  // workgroup), the first one's workgroup, and whether it is that workgroup's
  // second slot
  struct Parts {
    int n;
    int64_t c0;
    bool late;
    __device__ __forceinline__ int64_t slot(int i) const { return 2 * (c0 + i) + (i == 0 && late); }
  };
  __device__ __forceinline__ Parts parts(int64_t u0, int of) const {
    Parts p;
    p.c0 = u0 / per;
    p.n = (int)((u0 + of - 1) / per - p.c0) + 1;
    p.late = u0 != p.c0 * per;
    return p;
  }
};

}  // namespace qg
