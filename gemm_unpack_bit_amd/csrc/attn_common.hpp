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
// is a normal fp16 number.
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
  static constexpr float LIFT = 0.f, SLACK = 8.f;
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

// What query token t of a row sees: every key below lim, and of the keys from
// pos on those whose bit is set in its mask words.
template <bool PAGED>
struct Sight {
  int lim;
  const uint64_t* words;  // NULL: lim alone
  __device__ __forceinline__ void init(const AttnArgs& a, const Row& r, int t) {
    words = nullptr;
    if (t >= r.n) {
      lim = 0;
      return;
    }
    if constexpr (PAGED) {
      if (a.mask) {
        lim = r.pos;
        words = a.mask + (int64_t)(r.q0 + t) * a.mask_words;
      } else {
        lim = r.pos + t + 1;
      }
    } else {
      lim = a.causal ? r.pos + t + 1 : r.keys;
    }
    lim = lim < 0 ? 0 : lim > r.keys ? r.keys : lim;
  }
  // bit i: key kb + i is seen, i < 64
  __device__ __forceinline__ uint64_t window(const AttnArgs& a, const Row& r, int kb) const {
    auto below = [](int n) { return n <= 0 ? 0ull : n >= 64 ? ~0ull : (1ull << n) - 1; };
    uint64_t v = below(lim - kb);
    if (PAGED && words) {
      const int i0 = kb - r.pos;
      uint64_t m = 0;
      if (i0 >= 0) {
        const int w = i0 >> 6, s = i0 & 63;
        if (w < a.mask_words) m = words[w] >> s;
        if (s && w + 1 < a.mask_words) m |= words[w + 1] << (64 - s);
      } else if (i0 > -64) {
        m = words[0] << -i0;
      }
      v |= m & below(r.keys - kb);
    }
    return v;
  }
};

// partial results: [slots][BM] (max, sum), then [slots][BM][D] sums
template <int BM, int D>
struct Partials {
  float *ml, *o;
  __device__ __forceinline__ Partials(float* ws, int64_t slots) : ml(ws), o(ws + slots * BM * 2) {}
  __device__ __forceinline__ float* ml_at(int64_t slot, int row) const { return ml + (slot * BM + row) * 2; }
  __device__ __forceinline__ float* o_at(int64_t slot, int row) const { return o + (slot * BM + row) * D; }
};

// Joins the partial results of one query row (one wave; lane l holds outputs
// EPL * l ..): o = sum 2^(m_i - M) o_i / sum 2^(m_i - M) l_i over parts i,
// slot(i) naming the part's slot.
template <typename E, int BM, int D, typename F>
__device__ __forceinline__ void join_row(const Partials<BM, D>& p, int row, int parts, F&& slot, uint16_t* out) {
  constexpr int EPL = D / 64;
  const int lane = threadIdx.x & 63;
  float M = NEG_INF;
  for (int i = lane; i < parts; i += 64) M = fmaxf(M, p.ml_at(slot(i), row)[0]);
  M = quarter_max(M);
#pragma unroll
  for (int d = 1; d < 16; d <<= 1) M = fmaxf(M, __shfl_xor(M, d));
  const float base = M == NEG_INF ? 0.f : M;
  float l = 0.f, acc[EPL] = {};
#pragma unroll 4
  for (int i = 0; i < parts; ++i) {
    const int64_t s = slot(i);
    const float* ml = p.ml_at(s, row);
    const float w = exp2_(ml[0] - base), li = ml[1];
    l += w * li;
    const float* o = p.o_at(s, row) + EPL * lane;
#pragma unroll
    for (int e = 0; e < EPL; ++e) acc[e] += li == 0.f ? 0.f : w * o[e];
  }
  const float inv = l == 0.f ? 0.f : 1.f / l;
  if constexpr (EPL == 2) reinterpret_cast<uint32_t*>(out)[lane] = E::pack(acc[0] * inv, acc[1] * inv);
  else out[lane] = (uint16_t)E::pack(acc[0] * inv, 0.f);
}

// The split of the key axis.  An item is a tile of BM query rows (row
// t * group + g: query token t, head g of the key head's group) of one row and
// key head; its keys are cut into units of KB.  The units of all items, in the
// order row, tile, key head, unit, are shared out evenly: workgroup c takes
// units [c * per, (c + 1) * per), per = max(least, ceil(total / workgroups)).
// So a long row is worked on by many workgroups and short ones share one,
// whatever the mix, and no workgroup waits for another.  An item that lies in
// one workgroup is finished there; of the others every workgroup leaves a
// partial result (the part that starts with the workgroup's share in slot
// 2 c, one that starts later in slot 2 c + 1), which a second kernel joins in
// key order.
struct Split {
  int64_t per, total;
};
struct Place {  // of one unit
  int b;
  int64_t first;  // the row's first unit
};
template <int BM, int KB, bool PAGED>
struct Units {
  static __device__ __forceinline__ int tiles(const AttnArgs& a, const Row& r) { return (r.n * a.group + BM - 1) / BM; }
  // key units of an item; one without keys still has an output to write
  static __device__ __forceinline__ int units(const Row& r) { return r.keys ? (r.keys + KB - 1) / KB : 1; }
  static __device__ __forceinline__ int64_t cost(const AttnArgs& a, int b) {
    if (b >= a.rows) return 0;
    const Row r = row_of<PAGED>(a, b);
    return (int64_t)tiles(a, r) * a.heads_kv * units(r);
  }
  static __device__ __forceinline__ int64_t scan64(int64_t v) {  // inclusive, over the wave
    const int lane = threadIdx.x & 63;
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) {
      const int64_t o = __shfl_up((long long)v, d);
      if (lane >= d) v += o;
    }
    return v;
  }
  static __device__ __forceinline__ int64_t uniform64(int64_t v, int lane) {
    const uint32_t lo = __builtin_amdgcn_readlane((uint32_t)v, lane);
    const uint32_t hi = __builtin_amdgcn_readlane((uint32_t)((uint64_t)v >> 32), lane);
    return (int64_t)((uint64_t)hi << 32 | lo);
  }
  static __device__ __forceinline__ Split split(const AttnArgs& a, int workgroups, int least) {
    Split s;
    s.total = 0;
    for (int b0 = 0; b0 < a.rows; b0 += 64) s.total += uniform64(scan64(cost(a, b0 + (threadIdx.x & 63))), 63);
    const int64_t even = (s.total + workgroups - 1) / workgroups;
    s.per = even > least ? even : least;
    return s;
  }
  // the row that unit u (< total) belongs to
  static __device__ __forceinline__ Place place(const AttnArgs& a, int64_t u) {
    int64_t before = 0;
    for (int b0 = 0; b0 < a.rows; b0 += 64) {
      const int64_t c = cost(a, b0 + (threadIdx.x & 63)), s = scan64(c);
      const int64_t all = uniform64(s, 63);
      if (u < before + all) {
        const int l = __builtin_ctzll(__ballot(u < before + s));
        return Place{b0 + l, before + uniform64(s - c, l)};
      }
      before += all;
    }
    return Place{a.rows - 1, before};
  }
  // one wave: query token w / heads of head w % heads, where its item lay in
  // several workgroups
  template <typename E, int D>
  static __device__ __forceinline__ void join(const AttnArgs& a, int w, int workgroups, int least) {
    const int token = w / a.heads, head = w - token * a.heads, h = head / a.group;
    const Split sp = split(a, workgroups, least);
    const int b = find_row(a.rows, token, [&](int i) { return a.cu[i]; });
    const Row r = row_of<PAGED>(a, b);
    const int t = token - r.q0;
    if (t < 0 || t >= r.n) return;
    int64_t first = 0;
    for (int b0 = 0; b0 < b; b0 += 64) {
      const int x = b0 + (threadIdx.x & 63);
      first += uniform64(scan64(x < b ? cost(a, x) : 0), 63);
    }
    const int qr = t * a.group + head - h * a.group;
    const int tile = qr / BM;
    const int64_t u0 = first + (int64_t)(tile * a.heads_kv + h) * units(r), u1 = u0 + units(r);
    const int64_t c0 = u0 / sp.per, c1 = (u1 - 1) / sp.per;
    if (c0 == c1) return;
    const Partials<BM, D> parts(a.ws, 2 * (int64_t)workgroups);
    const bool late = u0 != c0 * sp.per;
    join_row<E>(parts, qr - tile * BM, (int)(c1 - c0 + 1), [&](int i) { return 2 * (c0 + i) + (i == 0 && late); },
                a.o + (int64_t)token * a.o_token + (int64_t)head * a.o_head);
  }
};

}  // namespace qg
