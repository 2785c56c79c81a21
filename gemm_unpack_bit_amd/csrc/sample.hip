// The next token of every row from its logits: temperature, top-k, top-p, min-p
// and a given random number.
//
// Mathematics.  With M the row's largest logit and w_i = exp((l_i - M) / T), the
// tokens in the order of falling logits, equal ones by index, keep a prefix:
//   top-k  the first k,
//   top-p  of those, with S the sum of their weights, every one with less than
//          p S in front of it,
//   min-p  of those, every one with w_i >= min_p.
// The result is the first token, now in the order of the vocabulary, up to which
// the kept weights add up to more than u times their sum.
//
// Weights are held in fixed point, 2^-42 of the largest, and worked out in 64
// bits: their sums are whole numbers, so they do not depend on the order in which
// threads add them, and a draw that falls near the border of two tokens falls on
// the same side as in the definition.  (In 32 bits, of 128000 tokens kept about
// one draw in a thousand would not.)
//
// A prefix of the order ends at one logit and index.  No row is sorted to find
// them: a histogram of 1024 bins of equal width, from the row's largest logit to
// its smallest, says in which bin it ends, and the elements of that bin alone
// (with top-k, where they are few, of all bins up to it) are listed and sorted.
//
// Kernels.  `slices` of the vocabulary, each a workgroup, do what touches every
// logit: sample_scan_kernel (largest and smallest), sample_bins_kernel (the
// histogram, where a row has top-k or top-p), sample_draw_kernel (the list, and the
// sums of what is kept for certain); of each row, the workgroup that is the last one
// with this does the rest.
//
// Bound: for one row the launches and what waits for one another (the largest logit,
// the bin, the list, the draw); for many the three times that a logit is read (once
// from memory, then from the caches), and a weight's 50 instructions, 18 of them of
// 64 bits, at 4.5 cycles each, twice with top-p.
//
// Measured: one row of 128256 fp16 logits with top-p 18.6 us; 72 rows of 151643 fp32
// ones, settings of all kinds, 46.2 us: scan 10, bins 13, draw 20.  In the last a
// row's summing takes 2 us where little is kept and 5 to 9 where much is, its end
// 2 us for one token of the list, 4 up to 256, 8 above.
#include "attn_common.hpp"
#include "step.hpp"

namespace qg {
namespace {

constexpr int BINS = 1024;  // and at most so many chunks, of which a slice has one per wave
constexpr int CAP = 2032;   // elements listed (so that four workgroups' LDS fits a CU)
constexpr int T = 256;      // threads of every workgroup
constexpr int WAVES = T / 64, PIECE = 8, STEP = PIECE * T, MOST_SLICES = BINS / WAVES;
constexpr int OWN = BINS / T;  // bins (or chunks) of a thread
constexpr float LOWEST = -3.402823466e38f;

// what a slice of a row leaves: its largest logit's key and place (the first
// one), its smallest finite logit
struct Part {
  uint32_t key;
  int at;
  float least;
  int pad;
};
// how the end of a row's prefix is found: it has none, all that is left is in
// the list, it lies in the bin `bin` whose elements are in the list, or neither
// (the list is not used)
enum : int { CUT_NONE = 0, CUT_FEW = 1, CUT_BIN = 2, CUT_MANY = 3 };
struct Plan {
  int mode, bin;
  unsigned long long before;  // weights in front of the bin (by weight)
  double goal;                // p S
  unsigned long long total;   // S
};
// the end of a prefix: keys above `key`, and of those equal the ones up to
// index `at`
struct Cut {
  uint32_t key;
  int at;
};

struct Work {
  unsigned long long *bins, *list, *sums;  // [rows][BINS], [rows][CAP], [rows][slices * WAVES]
  int *listed, *done;                      // [rows]
  Part* parts;                             // [rows][slices]
  __device__ __forceinline__ Work(void* ws, int64_t rows, int slices) {
    char* p = reinterpret_cast<char*>(ws);
    bins = reinterpret_cast<unsigned long long*>(p), p += rows * BINS * 8;
    list = reinterpret_cast<unsigned long long*>(p), p += rows * CAP * 8;
    parts = reinterpret_cast<Part*>(p), p += rows * slices * 16;
    sums = reinterpret_cast<unsigned long long*>(p), p += rows * slices * (8 * WAVES);
    listed = reinterpret_cast<int*>(p), p += rows * 4;
    done = reinterpret_cast<int*>(p);
  }
};
constexpr size_t work_bytes(int64_t rows, int slices) {
  return (size_t)(rows * (BINS * 8 + CAP * 8 + 8) + rows * slices * (16 + 8 * WAVES));
}

// Keys: floats in their order as unsigned numbers; NaN as -infinity, -0 as 0.
__device__ __forceinline__ float clean(float v) { return v == v ? v + 0.f : NEG_INF; }
__device__ __forceinline__ uint32_t key_of(float v) {
  const uint32_t b = __float_as_uint(v);
  return b ^ ((uint32_t)((int)b >> 31) | 0x80000000u);
}
__device__ __forceinline__ float logit_of(uint32_t key) {
  return __uint_as_float(key & 0x80000000u ? key ^ 0x80000000u : ~key);
}

template <int TYPE>
__device__ __forceinline__ float logit_at(const void* row, int64_t i) {
  if constexpr (TYPE == 0) return F16::value(static_cast<const uint16_t*>(row)[i]);
  else if constexpr (TYPE == 1) return BF16::value(static_cast<const uint16_t*>(row)[i]);
  else return static_cast<const float*>(row)[i];
}
// PIECE logits from i on, as they are in memory, and as floats.  (Rows may begin
// at any element.)
template <int TYPE>
struct Raw {
  u4 w[TYPE == 2 ? 2 : 1];
  __device__ __forceinline__ void load(const void* row, int i) {
    if constexpr (TYPE == 2) {
      typedef uint32_t loose __attribute__((ext_vector_type(4), aligned(4)));
      const uint32_t* p = static_cast<const uint32_t*>(row) + i;
      w[0] = *reinterpret_cast<const loose*>(p);
      w[1] = *reinterpret_cast<const loose*>(p + 4);
    } else {
      typedef uint32_t loose __attribute__((ext_vector_type(4), aligned(2)));
      w[0] = *reinterpret_cast<const loose*>(static_cast<const uint16_t*>(row) + i);
    }
  }
  template <bool CLEAN>
  __device__ __forceinline__ void get(float (&v)[PIECE]) const {
#pragma unroll
    for (int e = 0; e < PIECE; ++e) {
      if constexpr (TYPE == 2) {
        v[e] = __uint_as_float(w[e / 4][e & 3]);
      } else {
        const uint16_t h = (uint16_t)(w[0][e / 2] >> (16 * (e & 1)));
        v[e] = TYPE == 0 ? F16::value(h) : BF16::value(h);
      }
      if constexpr (CLEAN) v[e] = clean(v[e]);
    }
  }
};
// the same where the row may end inside the piece: those from `end` on are
// -infinity
template <int TYPE>
__device__ __forceinline__ void load_piece(const void* row, int i, int end, float (&v)[PIECE]) {
  if (i + PIECE <= end) {
    Raw<TYPE> r;
    r.load(row, i);
    r.template get<true>(v);
  } else {
#pragma unroll
    for (int e = 0; e < PIECE; ++e) v[e] = i + e < end ? clean(logit_at<TYPE>(row, i + e)) : NEG_INF;
  }
}
// The pieces of [begin, end), THREADS at a time, this one's first at begin + PIECE
// * thread; four of a thread are on their way at once, the first ones from the
// construction on.  Without CLEAN they may hold NaN and -0.
template <int TYPE, int THREADS, bool CLEAN>
struct Pieces {
  static constexpr int AT_ONCE = 4, ROUND = PIECE * THREADS;
  const void* row;
  int i, end;
  Raw<TYPE> raw[AT_ONCE];
  __device__ __forceinline__ Pieces(const void* row, int begin, int end, int thread)
      : row(row), i(begin + PIECE * thread), end(end) {
#pragma unroll
    for (int k = 0; k < AT_ONCE; ++k)
      if (i + k * ROUND + PIECE <= end) raw[k].load(row, i + k * ROUND);
  }
  // f(piece, its first index)
  template <typename F>
  __device__ __forceinline__ void each(F&& f) {
    while (i + PIECE <= end) {
#pragma unroll
      for (int k = 0; k < AT_ONCE; ++k) {
        if (i + PIECE > end) continue;
        float v[PIECE];
        raw[k].template get<CLEAN>(v);
        if (i + AT_ONCE * ROUND + PIECE <= end) raw[k].load(row, i + AT_ONCE * ROUND);
        f(v, i);
        i += ROUND;
      }
    }
    if (i < end) {  // (the last one)
      float v[PIECE];
      load_piece<TYPE>(row, i, end, v);
      f(v, i);
    }
  }
};

// Weights.  x = (l - M) log2(e) / T <= 0 is split into its nearest whole number
// n and f; 2^f is a polynomial through 2^f at the ten Chebyshev points of
// [-1/2, 1/2], off by 3e-14 of it at most (2^-42 is 2.3e-13); n goes into the
// exponent.  The additions of 1.5 * 2^52 round to whole numbers and leave these in
// the sum's low bits.
struct Weigh {
  double top, by;  // M, log2(e) / T
  __device__ __forceinline__ double operator()(float l) const {
    constexpr double ROUND = 0x1.8p52;
    const double x = l == (float)top ? 0.0 : ((double)l - top) * by, r = x + ROUND, f = x - (r - ROUND);
    double p = 1.0205905413765595e-07;
    p = fma(p, f, 1.325964524488711e-06);
    p = fma(p, f, 1.5252672924850737e-05);
    p = fma(p, f, 1.540343375125101e-04);
    p = fma(p, f, 1.3333558200794592e-03);
    p = fma(p, f, 9.618129193934313e-03);
    p = fma(p, f, 5.550410866465167e-02);
    p = fma(p, f, 2.402265069564034e-01);
    p = fma(p, f, 6.931471805599462e-01);
    p = fma(p, f, 1.0);
    const uint64_t n = __builtin_bit_cast(uint64_t, r) << 52;
    // (below 2^-64, and where x is NaN, as of -infinity at an infinite T: none)
    return x > -64.0 ? __builtin_bit_cast(double, __builtin_bit_cast(uint64_t, p) + n) : 0.0;
  }
};
// as a whole number of 2^-42, rounded to nearest
__device__ __forceinline__ unsigned long long fixed(double w) {
  return __builtin_bit_cast(unsigned long long, fma(w, 0x1p42, 0x1p52)) & ((1ull << 52) - 1);
}

// What the row's settings ask for.
struct Settings {
  double by, p, least;
  int k;
  bool greedy;
  __device__ __forceinline__ Settings(const SampleArgs& a, int row) {
    const float t = a.temperature ? a.temperature[row] : 1.f;
    greedy = !(t > 0.f);
    by = 1.4426950408889634 / (double)t;
    k = a.top_k ? a.top_k[row] : 0;
    const float q = a.top_p ? a.top_p[row] : 1.f;
    p = q < 1.f ? (q > 0.f ? (double)q : 0.0) : 1.0;  // (NaN: off)
    const float m = a.min_p ? a.min_p[row] : 0.f;
    least = m > 0.f ? (m < 1.f ? (double)m : 1.0) : 0.0;
  }
  // finite, and at most as large as every logit whose weight passes min-p
  __device__ __forceinline__ float under(float most) const {
    const float l = (float)((double)most + ((double)__builtin_log2f((float)least) - 0.01) / by);
    return least > 0.0 && fabsf(l) < __builtin_inff() ? l : LOWEST;
  }
  __device__ __forceinline__ bool by_count(int vocab) const { return k > 0 && k < vocab; }
  __device__ __forceinline__ bool by_weight() const { return p < 1.0; }
};

// Lane moves of 64-bit values without a detour through LDS: the value of lane
// ^ J, and sums over the wave's lanes up to and with the lane's.
template <int CTRL, int ROWS = 0xF>
__device__ __forceinline__ uint32_t dpp32(uint32_t v) {
  return (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, CTRL, ROWS, 0xF, false);
}
template <int J>
__device__ __forceinline__ uint32_t lane_xor32(uint32_t v) {
  if constexpr (J == 1) return dpp32<DPP_QP_XOR1>(v);
  else if constexpr (J == 2) return dpp32<DPP_QP_XOR2>(v);
  else if constexpr (J == 4) return dpp32<0x1B>(dpp32<0x141>(v));  // mirrored in 8 lanes, then in 4
  else if constexpr (J == 8) return dpp32<DPP_ROR8>(v);
  else {
    const auto r = J == 16 ? __builtin_amdgcn_permlane16_swap(v, v, false, false)
                           : __builtin_amdgcn_permlane32_swap(v, v, false, false);
    return threadIdx.x & J ? r[0] : r[1];
  }
}
template <int J>
__device__ __forceinline__ unsigned long long lane_xor(unsigned long long v) {
  return (unsigned long long)lane_xor32<J>((uint32_t)(v >> 32)) << 32 | lane_xor32<J>((uint32_t)v);
}
__device__ __forceinline__ unsigned long long wave_max64(unsigned long long v) {
  auto most = [](unsigned long long x, unsigned long long y) { return x > y ? x : y; };
  v = most(v, lane_xor<1>(v));
  v = most(v, lane_xor<2>(v));
  v = most(v, lane_xor<4>(v));
  v = most(v, lane_xor<8>(v));
  v = most(v, lane_xor<16>(v));
  return most(v, lane_xor<32>(v));
}
template <int CTRL, int ROWS>
__device__ __forceinline__ unsigned long long dpp64(unsigned long long v) {
  return (unsigned long long)dpp32<CTRL, ROWS>((uint32_t)(v >> 32)) << 32 | dpp32<CTRL, ROWS>((uint32_t)v);
}
__device__ __forceinline__ unsigned long long wave_scan64(unsigned long long v) {
  v += dpp64<0x111, 0xF>(v);  // row_shr:1, 2, 4, 8, then the rows' last lanes
  v += dpp64<0x112, 0xF>(v);
  v += dpp64<0x114, 0xF>(v);
  v += dpp64<0x118, 0xF>(v);
  v += dpp64<DPP_BCAST15, 0xA>(v);
  v += dpp64<DPP_BCAST31, 0xC>(v);
  return v;
}

// A workgroup's threads: sums up to and with the thread's, and of all.
__device__ __forceinline__ unsigned long long block_scan64(unsigned long long v, unsigned long long& total,
                                                           unsigned long long* red) {
  const int lane = threadIdx.x & 63, w = threadIdx.x >> 6;
  v = wave_scan64(v);
  if (lane == 63) red[w] = v;
  __syncthreads();
  unsigned long long before = 0, all = 0;
#pragma unroll
  for (int i = 0; i < WAVES; ++i) {
    before += i < w ? red[i] : 0;
    all += red[i];
  }
  __syncthreads();
  total = all;
  return before + v;
}

// The row's largest logit's key and first place (as key << 32 | ~place), and
// its smallest finite logit, from the slices' parts (a thread each); the whole
// workgroup.
struct Top {
  unsigned long long best;
  float least;
  __device__ __forceinline__ float most() const { return logit_of((uint32_t)(best >> 32)); }
  __device__ __forceinline__ int place() const { return (int)~(uint32_t)best; }
};
__device__ __forceinline__ Part part_of(const Part* parts, int slices) {
  return (int)threadIdx.x < slices ? parts[threadIdx.x] : Part{0, -1, __builtin_inff(), 0};
}
__device__ __forceinline__ Top top_of(const Part& p, unsigned long long* red) {
  unsigned long long best = wave_max64((unsigned long long)p.key << 32 | (uint32_t)~p.at);
  unsigned long long low = wave_max64((uint32_t)~key_of(p.least));
  if ((threadIdx.x & 63) == 0) red[threadIdx.x >> 6] = best, red[WAVES + (threadIdx.x >> 6)] = low;
  __syncthreads();
#pragma unroll
  for (int i = 0; i < WAVES; ++i) {
    best = red[i] > best ? red[i] : best;
    low = red[WAVES + i] > low ? red[WAVES + i] : low;
  }
  __syncthreads();
  return {best, logit_of(~(uint32_t)low)};
}

// The bin of a logit l <= M: the same or a later one for every smaller l.  Bins
// go from the largest logit to the smallest, or to where weights are 0 (2^-44 of
// the largest; `ends`: the last bin then has no weights), so that a row masked
// with large negative numbers has fine bins too.
struct Binning {
  float most, by;
  bool ends;
  __device__ __forceinline__ Binning(const Top& t, const Settings& set) : most(t.most()) {
    const float width = most - t.least, all = (float)fmin(44.0 / set.by, 3e38);
    ends = !(width <= all);
    const float used = ends ? all : width;
    by = used > 0.f ? (float)BINS / used : 0.f;
  }
  // in bins from the largest logit on; past the last one the last one
  __device__ __forceinline__ float at(float l) const {
    // (NaN, of infinities: the middle one of three numbers is then the least of
    // the other two)
    return __builtin_amdgcn_fmed3f((most - l) * by, 0.f, (float)BINS - 0.001f);
  }
  __device__ __forceinline__ int operator()(float l) const { return (int)at(l); }
  // finite, and at most as large as every logit in the bins up to `last` that is
  // not -infinity (half a bin lower: more than the roundings)
  __device__ __forceinline__ float under(int last) const {
    const float l = most - ((float)last + 1.5f) / by;
    return last < BINS - 1 && fabsf(l) < __builtin_inff() ? l : LOWEST;
  }
  // one of 1024 parts of the bins [first, last], the same order, for l in them
  __device__ __forceinline__ int part(float l, int first, int last) const {
    const float d = (at(l) - (float)first) * ((float)BINS / (float)(last + 1 - first));
    return d < (float)(BINS - 1) ? (int)d : BINS - 1;
  }
};

// What follows from a row's histogram (a thread's bins: mine), the same in every
// workgroup of the row; all threads.
__device__ __forceinline__ Plan plan_of(const SampleArgs& a, const Settings& set, const unsigned long long (&mine)[OWN],
                                        bool ends, unsigned long long* red, Plan* shared) {
  const bool by_count = set.by_count(a.vocab), by_weight = set.by_weight();
  if (!by_count && !by_weight) return Plan{CUT_NONE, BINS, 0, 0.0, 0};
  unsigned long long sum = 0, total;
#pragma unroll
  for (int e = 0; e < OWN; ++e) sum += mine[e];
  if (threadIdx.x == 0) *shared = Plan{CUT_NONE, BINS, 0, 0.0, 0};
  unsigned long long before = block_scan64(sum, total, red) - sum;
  // by count: the first bin with k elements up to it (all may be fewer; among
  // elements without weight it does not matter which stay); by weight: the first
  // up to which the weights reach p S
  const double goal = by_count ? (double)set.k : set.p * (double)total;
#pragma unroll
  for (int e = 0; e < OWN; ++e) {
    const unsigned long long upto = before + mine[e];
    const int b = OWN * threadIdx.x + e;
    if ((double)upto >= goal && (b == 0 || (double)before < goal)) {
      Plan p{CUT_BIN, b, before, goal, total};
      if (by_count) p.mode = upto <= CAP ? CUT_FEW : by_weight ? CUT_MANY : ends && b == BINS - 1 ? CUT_NONE : CUT_BIN;
      *shared = p;
    }
    before = upto;
  }
  __syncthreads();
  Plan p = *shared;
  // (fewer logits above -infinity than k: no end by count)
  if (by_count && p.mode == CUT_NONE && by_weight) p.mode = total <= CAP ? CUT_FEW : CUT_MANY;
  return p;
}
__device__ __forceinline__ void own_bins(const SampleArgs& a, const unsigned long long* bins, unsigned long long (&mine)[OWN]) {
#pragma unroll
  for (int e = 0; e < OWN; ++e) mine[e] = a.top_k || a.top_p ? bins[OWN * threadIdx.x + e] : 0;
}

// ---------------------------------------------------------------------------
// slices
// ---------------------------------------------------------------------------

template <int TYPE>
__global__ void __launch_bounds__(T) sample_scan_kernel(SampleArgs a, int slices, int slice) {
  __shared__ unsigned long long red[2 * WAVES];
  const int row = blockIdx.x / slices, s = blockIdx.x % slices;
  const Work w(a.ws, a.rows, slices);
  const int begin = s * slice, end = min(begin + slice, a.vocab);
  const void* x = static_cast<const char*>(a.logits) + (int64_t)row * a.row_bytes;
  float most = NEG_INF, least = __builtin_inff();
  int at = begin;
  // (maxima and minima pass over NaN)
  Pieces<TYPE, T, false>(x, begin, end, threadIdx.x).each([&](const float (&v)[PIECE], int i) {
    float hi = v[0], lo = v[0];
#pragma unroll
    for (int e = 1; e < PIECE; ++e) hi = fmaxf(hi, v[e]), lo = fminf(lo, v[e]);
    // (seldom, after the first pieces; elements come by rising index, so the
    // first of equal ones stays)
    if (hi > most) {
      most = hi;
#pragma unroll
      for (int e = PIECE - 1; e >= 0; --e) at = v[e] == hi ? i + e : at;
    }
    if (lo == NEG_INF) {
      lo = __builtin_inff();
#pragma unroll
      for (int e = 0; e < PIECE; ++e) lo = v[e] > NEG_INF ? fminf(lo, v[e]) : lo;
    }
    least = fminf(least, lo);
  });
  unsigned long long best = wave_max64((unsigned long long)key_of(clean(most)) << 32 | (uint32_t)~at);
  least = logit_of(~(uint32_t)wave_max64((uint32_t)~key_of(least)));
  if ((threadIdx.x & 63) == 0) {
    red[threadIdx.x >> 6] = best;
    red[WAVES + (threadIdx.x >> 6)] = __float_as_uint(least);
  }
  __syncthreads();
  if (threadIdx.x == 0) {
#pragma unroll
    for (int i = 0; i < WAVES; ++i) {
      best = red[i] > best ? red[i] : best;
      least = fminf(least, __uint_as_float((uint32_t)red[WAVES + i]));
    }
    w.parts[(int64_t)row * slices + s] = Part{(uint32_t)(best >> 32), (int)~(uint32_t)best, least, 0};
    if (s == 0) w.listed[row] = w.done[row] = 0;
  }
  // the row's histogram starts at 0, a part of it by each slice
  if (a.top_k || a.top_p)
    for (int i = s * T + threadIdx.x; i < BINS; i += slices * T) w.bins[(int64_t)row * BINS + i] = 0;
}

// Counts (with top-k) or weights (with top-p alone) by bins.
template <int TYPE>
__global__ void __launch_bounds__(T) sample_bins_kernel(SampleArgs a, int slices, int slice) {
  __shared__ unsigned long long red[2 * WAVES];
  __shared__ unsigned long long bins[BINS];
  const int row = blockIdx.x / slices, s = blockIdx.x % slices;
  const Settings set(a, row);
  const bool by_count = set.by_count(a.vocab);
  if (set.greedy || !(by_count || set.by_weight())) return;
  const Work w(a.ws, a.rows, slices);
  const int begin = s * slice, end = min(begin + slice, a.vocab);
  Pieces<TYPE, T, false> pieces(static_cast<const char*>(a.logits) + (int64_t)row * a.row_bytes, begin, end, threadIdx.x);
  for (int i = threadIdx.x; i < BINS; i += T) bins[i] = 0;
  const Top top = top_of(part_of(w.parts + (int64_t)row * slices, slices), red);  // (with barriers)
  const Binning bin(top, set);
  const Weigh weigh{(double)top.most(), set.by};
  uint32_t* counts = reinterpret_cast<uint32_t*>(bins);
  pieces.each([&](const float (&v)[PIECE], int) {
    if (by_count) {
#pragma unroll
      for (int e = 0; e < PIECE; ++e)
        if (v[e] > NEG_INF) atomicAdd(&counts[bin(v[e])], 1u);
    } else {
#pragma unroll
      for (int e = 0; e < PIECE; ++e) {
        const unsigned long long f = fixed(weigh(v[e]));
        if (f) atomicAdd(&bins[bin(v[e])], f);
      }
    }
  });
  __syncthreads();
  for (int i = threadIdx.x; i < BINS; i += T) {
    const unsigned long long f = by_count ? counts[i] : bins[i];
    if (f) atomicAdd(&w.bins[(int64_t)row * BINS + i], f);
  }
}

// ---------------------------------------------------------------------------
// rows
// ---------------------------------------------------------------------------

// the place of a draw in a sum of weights, below it (u past the numbers below 1
// counts as the last of these, NaN as 0)
__device__ __forceinline__ unsigned long long target_of(float u, unsigned long long total) {
  const double t = (double)(u < 1.f ? u : 0x1.fffffep-1f) * (double)total;
  return u > 0.f ? (unsigned long long)t : 0;
}

__device__ __forceinline__ int power_of_two(int n) { return n < 2 ? 1 : 1 << (32 - __builtin_clz(n - 1)); }

struct Shared {
  unsigned long long list[CAP];
  union {  // (counts are looked at before elements are picked)
    unsigned long long few[2048];
    uint32_t counts[BINS];
  };
  unsigned long long bins[BINS];  // of weights or chunks' sums
  unsigned long long red[2 * WAVES];
  unsigned long long found;
  Plan plan;
  uint32_t key0, key1;
  int n, at;
};

// Sorts list[0 .. n) (n a power of two up to 2048) upwards; the whole workgroup,
// barriers on both sides.  Up to an entry a thread they stay in registers:
// partners within a wave change places by lanes, others through the list.
__device__ __forceinline__ void sort(unsigned long long* list, int n) {
  __syncthreads();
  if (n <= T) {
    const int t = threadIdx.x;
    unsigned long long v = t < n ? list[t] : 0;
    for (int k = 2; k <= n; k <<= 1) {
      // this place takes the smaller one of a pair, or the larger
      auto take = [&](unsigned long long o, int j) { v = (o < v) == (((t & j) == 0) == ((t & k) == 0)) ? o : v; };
      for (int j = k >> 1; j >= 64; j >>= 1) {
        __syncthreads();
        if (t < n) list[t] = v;
        __syncthreads();
        if (t < n) take(list[t ^ j], j);
      }
      if (k >= 64) take(lane_xor<32>(v), 32);
      if (k >= 32) take(lane_xor<16>(v), 16);
      if (k >= 16) take(lane_xor<8>(v), 8);
      if (k >= 8) take(lane_xor<4>(v), 4);
      if (k >= 4) take(lane_xor<2>(v), 2);
      take(lane_xor<1>(v), 1);
    }
    __syncthreads();
    if (t < n) list[t] = v;
  } else {
    for (int k = 2; k <= n; k <<= 1)
      for (int j = k >> 1; j > 0; j >>= 1) {
        __syncthreads();
        for (int t = threadIdx.x; t < n / 2; t += T) {
          const int i = ((t & ~(j - 1)) << 1) | (t & (j - 1)), o = i | j;
          const unsigned long long x = list[i], y = list[o];
          if ((x > y) == ((i & k) == 0)) list[i] = y, list[o] = x;
        }
      }
  }
  __syncthreads();
}

// A row with all that its workgroup needs.  List entries: ~key << 32 | index, so
// rising entries are falling logits, equal ones by index.
template <int TYPE>
struct OneRow {
  const SampleArgs& a;
  const Settings& set;
  Shared& sh;
  const void* x;
  const Binning bin;
  const Weigh weigh;

  __device__ __forceinline__ static uint32_t key_in(unsigned long long entry) { return ~(uint32_t)(entry >> 32); }
  __device__ __forceinline__ unsigned long long weight_of(uint32_t key) const { return fixed(weigh(logit_of(key))); }
  __device__ __forceinline__ unsigned long long scan(unsigned long long v, unsigned long long& total) const {
    return block_scan64(v, total, sh.red);
  }

  // f(logit, index) for the row's elements that are not -infinity
  template <typename F>
  __device__ __forceinline__ void each(F&& f) const {
    Pieces<TYPE, T, true>(x, 0, a.vocab, threadIdx.x).each([&](const float (&v)[PIECE], int i) {
#pragma unroll
      for (int e = 0; e < PIECE; ++e)
        if (v[e] != NEG_INF) f(v[e], i + e);
    });
  }

  // Sorts the n entries that are in `few`.
  __device__ __forceinline__ void order(int n) const {
    const int m = power_of_two(n);
    for (int i = n + threadIdx.x; i < m; i += T) sh.few[i] = ~0ull;
    sort(sh.few, m);
  }
  // The last of the n sorted entries of `few` that stays.  By count: the `want`th (from
  // 1).  By weight: the last with less than `goal` in front of it, `before` of
  // that in front of them (the first one, if none has).  `upto`: the weights
  // up to and with it.
  __device__ __forceinline__ int last_of(int n, bool by_weight, uint32_t want, unsigned long long before, double goal,
                                         unsigned long long& upto) const {
    const int each = (n + T - 1) / T, j0 = each * (int)threadIdx.x, j1 = min(j0 + each, n);  // a thread's entries
    unsigned long long total, sum = 0;
    for (int j = j0; j < j1; ++j) sum += weight_of(key_in(sh.few[j]));
    if (threadIdx.x == 0) sh.at = by_weight ? 0 : max((int)min(want, (uint32_t)n) - 1, 0);
    sum = scan(sum, total) - sum;
    if (by_weight) {
      int last = 0;
      unsigned long long at = before + sum;
      for (int j = j0; j < j1; ++j) {
        last = (double)at < goal ? j : last;
        at += weight_of(key_in(sh.few[j]));
      }
      if (last) atomicMax(&sh.at, last);
      __syncthreads();
    }
    const int l = sh.at;
    if (j0 <= l && l < j1) {
      for (int j = j0; j <= l; ++j) sum += weight_of(key_in(sh.few[j]));
      sh.found = sum;
    }
    __syncthreads();
    upto = n ? sh.found : 0;
    __syncthreads();
    return l;
  }

  // Sums over sh.bins or sh.counts (a thread's OWN ones side by side), in place.
  template <typename N>
  __device__ __forceinline__ void sum_up(N* bins) const {
    unsigned long long mine[OWN], sum = 0, total;
#pragma unroll
    for (int e = 0; e < OWN; ++e) mine[e] = sum += bins[OWN * threadIdx.x + e];
    const unsigned long long before = scan(sum, total) - sum;
#pragma unroll
    for (int e = 0; e < OWN; ++e) bins[OWN * threadIdx.x + e] = (N)(before + mine[e]);
    __syncthreads();
  }
  // The first bin up to which sums reach a goal, as reaches(bin) says (false,
  // ..., false, true, ...), or the last one.
  template <typename F>
  __device__ __forceinline__ int first_bin(F&& reaches) const {
    if (threadIdx.x == 0) sh.at = BINS - 1;
    __syncthreads();
#pragma unroll
    for (int e = 0; e < OWN; ++e) {
      const int b = OWN * threadIdx.x + e;
      if (reaches(b) && (b == 0 || !reaches(b - 1))) sh.at = b;
    }
    __syncthreads();
    const int r = sh.at;
    __syncthreads();
    return r;
  }

  // Chunks of the vocabulary: at most as many as bins, of at most STEP elements.
  __device__ __forceinline__ int chunk_shift() const {
    const int q = (a.vocab - 1) / BINS;
    return q ? 32 - __builtin_clz(q) : 0;
  }

  // The end of a prefix in the bin `only` (-1: anywhere) among keys from `low` on, with
  // the weights `inside` in front, by the row itself: where the list cannot say
  // (thousands of elements in one bin, or both criteria over as many).  Counts or
  // weights by ranges of keys, each about a 1000th of the last, until the range in
  // which the prefix ends has few elements, or one key.
  __device__ __forceinline__ Cut search(bool by_weight, uint32_t want, double goal, int only, uint32_t low,
                                        unsigned long long inside, unsigned long long& upto) const {
    uint32_t high = ~0u;
    auto in = [&](float l) {
      const uint32_t k = key_of(l);
      return k >= low && k <= high && (only < 0 || bin(l) == only);
    };
    uint32_t n = 0;
    for (;;) {
      __syncthreads();
      if (threadIdx.x == 0) sh.key0 = ~0u, sh.key1 = 0, sh.n = 0;
      for (int i = threadIdx.x; i < BINS; i += T) sh.counts[i] = 0, sh.bins[i] = 0;
      __syncthreads();
      uint32_t k0 = ~0u, k1 = 0;
      int mine = 0;
      each([&](float l, int) {
        if (in(l)) k0 = min(k0, key_of(l)), k1 = max(k1, key_of(l)), ++mine;
      });
      if (mine) atomicMin(&sh.key0, k0), atomicMax(&sh.key1, k1), atomicAdd(&sh.n, mine);
      __syncthreads();
      low = sh.key0, high = sh.key1, n = sh.n;
      only = -1;  // (keys between two of a bin are in it)
      want = min(want, n);
      if (n <= CAP || low == high) break;
      const int shift = max(0, 32 - __builtin_clz(high - low) - 10);
      each([&](float l, int) {
        if (!in(l)) return;
        const uint32_t r = (high - key_of(l)) >> shift;
        atomicAdd(&sh.counts[r], 1u);
        atomicAdd(&sh.bins[r], fixed(weigh(l)));
      });
      __syncthreads();
      sum_up(sh.bins);
      sum_up(sh.counts);
      const int r = first_bin([&](int i) {
        return by_weight ? (double)(inside + sh.bins[i]) >= goal : sh.counts[i] >= want;
      });
      want -= r ? sh.counts[r - 1] : 0;
      inside += r ? sh.bins[r - 1] : 0;
      const uint32_t h = high - ((uint32_t)r << shift), l = h - ((1u << shift) - 1);
      high = h;
      low = l > h || l < low ? low : l;
    }
    if (n <= CAP) {
      __syncthreads();  // (every wave has read the number before it starts again at 0)
      if (threadIdx.x == 0) sh.n = 0;
      __syncthreads();
      each([&](float l, int i) {
        if (in(l)) sh.few[atomicAdd(&sh.n, 1)] = (unsigned long long)~key_of(l) << 32 | (uint32_t)i;
      });
      __syncthreads();
      order(n);
      const int j = last_of(n, by_weight, want, inside, goal, upto);
      upto += inside;
      const unsigned long long entry = sh.few[j];
      __syncthreads();
      return Cut{key_in(entry), (int)(uint32_t)entry};
    }
    // all equal: the one of their number `m`, in the order of the vocabulary
    const unsigned long long w = weight_of(high);
    uint32_t m = want;
    if (by_weight) {
      const double need = goal - (double)inside;
      m = need > 0.0 ? (w ? (uint32_t)fmin(ceil(need / (double)w), (double)n) : n) : 1;
    }
    m = max(1u, min(m, n));
    const int shift = chunk_shift();
    for (int i = threadIdx.x; i < BINS; i += T) sh.counts[i] = 0;
    __syncthreads();
    each([&](float l, int i) {
      if (key_of(l) == high) atomicAdd(&sh.counts[i >> shift], 1u);
    });
    __syncthreads();
    sum_up(sh.counts);
    const int c = first_bin([&](int i) { return sh.counts[i] >= m; });
    const int end = min((c + 1) << shift, a.vocab), i = (c << shift) + PIECE * threadIdx.x;
    float v[PIECE];
    uint32_t mine = 0;
    if (i < end) {
      load_piece<TYPE>(x, i, end, v);
#pragma unroll
      for (int e = 0; e < PIECE; ++e) mine += v[e] != NEG_INF && key_of(v[e]) == high;
    }
    unsigned long long all;
    uint32_t at = (c ? sh.counts[c - 1] : 0) + (uint32_t)scan(mine, all) - mine;
    if (mine)
#pragma unroll
      for (int e = 0; e < PIECE; ++e)
        if (v[e] != NEG_INF && key_of(v[e]) == high && ++at == m) sh.at = i + e;
    __syncthreads();
    const int place = sh.at;
    __syncthreads();
    upto = inside + (unsigned long long)m * w;
    return Cut{high, place};
  }

  // Counts and weights of the n listed elements, which are in the bins [first,
  // last], up to each of 1024 parts of these.
  __device__ __forceinline__ void parts(int n, int first, int last) const {
    for (int i = threadIdx.x; i < BINS; i += T) sh.bins[i] = 0, sh.counts[i] = 0;
    __syncthreads();
    for (int j = threadIdx.x; j < n; j += T) {
      const uint32_t key = key_in(sh.list[j]);
      const int p = bin.part(logit_of(key), first, last);
      atomicAdd(&sh.bins[p], weight_of(key));
      atomicAdd(&sh.counts[p], 1u);
    }
    __syncthreads();
    sum_up(sh.bins);
    sum_up(sh.counts);
  }
  // Puts those of the n listed elements that `in` accepts into `few`, made into
  // entries by `as`, and sorts them; how many.
  template <typename F, typename G>
  __device__ __forceinline__ int pick(int n, F&& in, G&& as) const {
    if (threadIdx.x == 0) sh.n = 0;
    __syncthreads();
    for (int j = threadIdx.x; j < n; j += T) {
      const unsigned long long entry = sh.list[j];
      if (in(entry)) sh.few[atomicAdd(&sh.n, 1)] = as(entry);
    }
    __syncthreads();
    const int m = sh.n;
    order(m);
    return m;
  }
  // The end of a prefix among them: the part in which it lies, then its sorted
  // elements.  By count: the `want`th (from 1); by weight: as last_of, `before` in
  // front of all.  `upto`: the weights up to and with it.
  __device__ __forceinline__ Cut end_in(int n, int first, int last, bool by_weight, uint32_t want, unsigned long long before,
                                        double goal, unsigned long long& upto) const {
    const int r = first_bin([&](int i) { return by_weight ? (double)(before + sh.bins[i]) >= goal : sh.counts[i] >= want; });
    const unsigned long long inside = r ? sh.bins[r - 1] : 0;
    want -= r ? min(sh.counts[r - 1], want) : 0;
    const int m = pick(n, [&](unsigned long long e) { return bin.part(logit_of(key_in(e)), first, last) == r; },
                       [](unsigned long long e) { return e; });
    const int l = last_of(m, by_weight, want, before + inside, goal, upto);
    upto += inside;
    const unsigned long long entry = sh.few[l];
    __syncthreads();
    return Cut{key_in(entry), (int)(uint32_t)entry};
  }
  // The weight that an entry adds to what is kept.
  __device__ __forceinline__ unsigned long long kept(unsigned long long entry, Cut cut) const {
    const uint32_t key = key_in(entry);
    if (key < cut.key || (key == cut.key && (int)(uint32_t)entry > cut.at)) return 0;
    const double p = weigh(logit_of(key));
    return p >= set.least ? fixed(p) : 0;
  }
  // The chunk (of sh.bins, a thread's OWN ones side by side) in which the draw
  // falls, its place there and what is in front of it.
  __device__ __forceinline__ int chunk_of(float u, unsigned long long& before, unsigned long long& t) const {
    unsigned long long sum = 0, own[OWN], total;
#pragma unroll
    for (int e = 0; e < OWN; ++e) sum += own[e] = sh.bins[OWN * threadIdx.x + e];
    if (threadIdx.x == 0) sh.at = 0, sh.found = 0;
    unsigned long long at = scan(sum, total) - sum;
    t = target_of(u, total);
#pragma unroll
    for (int e = 0; e < OWN; ++e) {
      if (at <= t && t < at + own[e]) sh.at = OWN * threadIdx.x + e, sh.found = at;
      at += own[e];
    }
    __syncthreads();
    before = sh.found;
    return sh.at;
  }

  // The token, among elements [begin, end): the first up to which the kept
  // weights, `before` in front, pass t; returns the weights up to the end.  (Where
  // they do not pass it nothing is written.)
  __device__ __forceinline__ unsigned long long draw(int begin, int end, Cut cut, unsigned long long before,
                                                     unsigned long long t, int32_t* out) const {
    for (int i0 = begin; i0 < end && before <= t; i0 += STEP) {
      const int i = i0 + PIECE * threadIdx.x;
      unsigned long long w[PIECE], sum = 0, all;
      float v[PIECE];
      if (i < end) load_piece<TYPE>(x, i, end, v);
#pragma unroll
      for (int e = 0; e < PIECE; ++e) {
        w[e] = 0;
        if (i + e >= end || v[e] == NEG_INF) continue;
        const uint32_t key = key_of(v[e]);
        if (key < cut.key || (key == cut.key && i + e > cut.at)) continue;
        const double p = weigh(v[e]);
        w[e] = p >= set.least ? fixed(p) : 0;
        sum += w[e];
      }
      unsigned long long at = before + scan(sum, all) - sum;
#pragma unroll
      for (int e = 0; e < PIECE; ++e) {
        if (at <= t && t < at + w[e]) *out = i + e;
        at += w[e];
      }
      before += all;
    }
    return before;
  }

  // Up to T entries, one a thread (~0: none), sorted: the thread's is the one of its
  // number.
  __device__ __forceinline__ unsigned long long sorted(unsigned long long entry, int n) const {
    const int m = power_of_two(n);
    if ((int)threadIdx.x < m) sh.few[threadIdx.x] = entry;
    sort(sh.few, m);
    return (int)threadIdx.x < n ? sh.few[threadIdx.x] : ~0ull;
  }
  // The token, where all that the prefix by count can hold are n <= T entries, one a
  // thread (~0: none).
  __device__ __forceinline__ void among(unsigned long long entry, int n, bool by_weight, float u, int32_t* out) const {
    const int j = threadIdx.x;
    entry = sorted(entry, n);
    const bool live = j < n && j < set.k;
    const double p = weigh(logit_of(key_in(entry)));
    unsigned long long w = live ? fixed(p) : 0, total;
    const unsigned long long before = scan(w, total) - w;
    if (!live || (by_weight && j > 0 && !((double)before < set.p * (double)total)) || !(p >= set.least)) w = 0;
    // in the order of the vocabulary
    sh.bins[j] = w;
    const unsigned long long place = sorted(j < n ? entry << 32 | (uint32_t)j : ~0ull, n);
    w = j < n ? sh.bins[(uint32_t)place] : 0;
    const unsigned long long at = scan(w, total) - w, t = target_of(u, total);
    if (at <= t && t < at + w) *out = (int)(place >> 32);
  }
  // The end of a prefix among n <= T entries, one a thread (~0: none), that follow
  // `plan.before` of it; what stays of them goes into the chunks' sums, sh.bins.
  __device__ __forceinline__ Cut end_among(unsigned long long entry, int n, bool by_count, const Plan& plan, int chunk) const {
    const int j = threadIdx.x;
    entry = sorted(entry, n);
    const double p = weigh(logit_of(key_in(entry)));
    unsigned long long w = j < n ? fixed(p) : 0, total;
    const unsigned long long before = plan.before + scan(w, total) - w;
    auto stays = [&](int j, unsigned long long before) {
      return j < n && (j == 0 || (by_count ? j < set.k - (int)plan.before : (double)before < plan.goal));
    };
    if (stays(j, before)) {
      if (!stays(j + 1, before + w)) sh.found = entry;
      if (w && p >= set.least) atomicAdd(&sh.bins[(uint32_t)entry / (uint32_t)chunk], w);
    }
    __syncthreads();
    const unsigned long long last = sh.found;
    __syncthreads();
    return Cut{key_in(last), (int)(uint32_t)last};
  }

  // The token, from the row's logits alone.
  __device__ __forceinline__ void alone(bool by_count, bool by_weight, const Plan& plan, float u, int32_t* out) const {
    Cut cut{0, 0};
    unsigned long long upto = 0, total, before, t;
    if (by_count) {
      const bool some = plan.bin < BINS;  // (otherwise all stay)
      unsigned long long front = 0;
      if (some && by_weight) {
        each([&](float l, int) {
          if (bin(l) < plan.bin) front += fixed(weigh(l));
        });
        scan(front, total);
        front = total;
      }
      cut = search(false, (uint32_t)set.k - (some ? (uint32_t)plan.before : 0), 0.0, some ? plan.bin : -1, 0, front, upto);
    }
    if (by_weight)
      cut = search(true, 1, by_count ? set.p * (double)upto : plan.goal, by_count ? -1 : plan.bin, cut.key,
                   by_count ? 0 : plan.before, upto);
    const int shift = chunk_shift();
    for (int i = threadIdx.x; i < BINS; i += T) sh.bins[i] = 0;
    __syncthreads();
    each([&](float l, int i) {
      const unsigned long long w = kept((unsigned long long)~key_of(l) << 32 | (uint32_t)i, cut);
      if (w) atomicAdd(&sh.bins[i >> shift], w);
    });
    __syncthreads();
    const int c = chunk_of(u, before, t);
    draw(c << shift, min((c + 1) << shift, a.vocab), cut, before, t, out);
  }
};

// Across the workgroups of a row, which sit on different XCDs whose caches do not
// see each other: past these.
template <typename V>
__device__ __forceinline__ void put(V* p, V v) {
  __hip_atomic_store(p, v, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}
template <typename V>
__device__ __forceinline__ V get(const V* p) {
  return __hip_atomic_load(p, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}

// The slice's elements of the bin in which the prefix ends go into the list (or
// those of all bins up to it); the weights that it keeps of the bins in front of
// it are summed, by chunks: a wave has a run of the slice.  The row's workgroup
// that is the last one with this then finds the token; none waits for another.
template <int TYPE>
__global__ void __launch_bounds__(T, 4) sample_draw_kernel(SampleArgs a, int slices, int slice) {
  __shared__ Shared sh;
  __shared__ int mine_s, place_s;
  const int row = blockIdx.x / slices, s = blockIdx.x % slices;
  if (threadIdx.x == 0) mine_s = 0;
  const Work w(a.ws, a.rows, slices);
  const Part part = part_of(w.parts + (int64_t)row * slices, slices);
  unsigned long long mine[OWN];
  own_bins(a, w.bins + (int64_t)row * BINS, mine);
  const Settings set(a, row);
  int32_t* out = a.out + row;
  const float u = a.u[row];
  const void* x = static_cast<const char*>(a.logits) + (int64_t)row * a.row_bytes;
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int begin = s * slice + wave * (slice / WAVES), end = min(begin + slice / WAVES, a.vocab);
  Pieces<TYPE, 64, false> pieces(x, begin, end, lane);
  const Top top = top_of(part, sh.red);  // (with barriers)
  if (set.greedy || top.most() == NEG_INF) {
    if (s == 0 && threadIdx.x == 0) *out = top.most() == NEG_INF ? -1 : top.place();
    return;
  }
  const Weigh weigh{(double)top.most(), set.by};
  const Binning bin(top, set);
  const OneRow<TYPE> r{a, set, sh, x, bin, weigh};
  const bool by_count = set.by_count(a.vocab), by_weight = set.by_weight();
  const Plan plan = plan_of(a, set, mine, bin.ends, sh.red, &sh.plan);
  if (plan.mode == CUT_MANY) {
    if (s == 0) r.alone(by_count, by_weight, plan, u, out);
    return;
  }

  // The logits up to the plan's bin are above this, and few others: most pieces are
  // passed over.  So are those that min-p takes out, but where top-p counts them.
  float near = plan.mode == CUT_NONE ? LOWEST : bin.under(plan.bin);
  if (plan.mode != CUT_FEW) near = fmaxf(near, set.under(top.most()));
  unsigned long long sum = 0;
  pieces.each([&](const float (&v)[PIECE], int i) {
    const float hi = fmaxf(fmaxf(fmaxf(v[0], v[1]), fmaxf(v[2], v[3])), fmaxf(fmaxf(v[4], v[5]), fmaxf(v[6], v[7])));
    if (!(hi >= near)) return;
#pragma unroll
    for (int e = 0; e < PIECE; ++e) {
      if (!(v[e] >= near)) continue;
      const int b = plan.mode == CUT_NONE ? 0 : bin(v[e]);
      if (plan.mode != CUT_FEW && b < plan.bin) {
        const double p = weigh(v[e]);
        sum += p >= set.least ? fixed(p) : 0;
      } else if (b <= plan.bin) {
        const int at = atomicAdd(&mine_s, 1);
        if (at < CAP) sh.few[at] = (unsigned long long)~key_of(clean(v[e])) << 32 | (uint32_t)(i + e);
      }
    }
  });
  sum = wave_scan64(sum);
  if (lane == 63) put(&w.sums[((int64_t)row * slices + s) * WAVES + wave], sum);
  if (plan.mode != CUT_NONE) {
    __syncthreads();
    if (threadIdx.x == 0 && mine_s) place_s = atomicAdd(&w.listed[row], mine_s);
    __syncthreads();
    // (more than CAP in all: the list is not used, and not filled past its end)
    for (int j = threadIdx.x; j < min(mine_s, CAP) && place_s + j < CAP; j += T)
      put(&w.list[(int64_t)row * CAP + place_s + j], sh.few[j]);
  }
  asm volatile("s_waitcnt vmcnt(0)" ::: "memory");  // this wave's stores have reached the device's memory
  __syncthreads();                                  // ... and every wave's
  if (threadIdx.x == 0) sh.n = atomicAdd(&w.done[row], 1);
  __syncthreads();
  if (sh.n != slices - 1) return;

  // (asked for at once, with the list's first places, whether filled or not)
  const int n = plan.mode == CUT_NONE ? 0 : get(&w.listed[row]);
  unsigned long long sums[OWN], upto, before, t;
#pragma unroll
  for (int e = 0; e < OWN; ++e) {
    const int c = OWN * threadIdx.x + e;
    sums[e] = c < slices * WAVES ? get(&w.sums[(int64_t)row * slices * WAVES + c]) : 0;
  }
  const unsigned long long* list = w.list + (int64_t)row * CAP;
  const unsigned long long l0 = get(&list[threadIdx.x]), l1 = get(&list[T + threadIdx.x]);
  if (n > CAP) {
    r.alone(by_count, by_weight, plan, u, out);
    return;
  }
  sh.list[threadIdx.x] = l0, sh.list[T + threadIdx.x] = l1;
  for (int j = 2 * T + threadIdx.x; j < n; j += T) sh.list[j] = get(&list[j]);
  __syncthreads();
  Cut cut{0, 0};
  if (plan.mode == CUT_FEW) {
    if (n <= T) {
      r.among((int)threadIdx.x < n ? l0 : ~0ull, n, by_weight, u, out);
      return;
    }
    // everything from the list: the ends, then the draw by chunks of the
    // vocabulary
    const int last = min(plan.bin, BINS - 1);
    r.parts(n, 0, last);
    cut = r.end_in(n, 0, last, false, (uint32_t)min(set.k, n), 0, 0.0, upto);
    if (by_weight) cut = r.end_in(n, 0, last, true, 1, 0, set.p * (double)upto, upto);
    const uint32_t chunk = (uint32_t)(a.vocab + BINS - 1) / BINS;
    for (int i = threadIdx.x; i < BINS; i += T) sh.bins[i] = 0;
    __syncthreads();
    for (int j = threadIdx.x; j < n; j += T) {
      const unsigned long long w = r.kept(sh.list[j], cut);
      if (w) atomicAdd(&sh.bins[(uint32_t)sh.list[j] / chunk], w);
    }
    __syncthreads();
    const uint32_t c = (uint32_t)r.chunk_of(u, before, t);
    const int m = r.pick(n, [&](unsigned long long e) { return (uint32_t)e / chunk == c && r.kept(e, cut); },
                         [](unsigned long long e) { return e << 32 | e >> 32; });
    if (threadIdx.x == 0)
      for (int j = 0; j < m; ++j) {  // (a chunk has few)
        const unsigned long long w = r.weight_of(~(uint32_t)sh.few[j]);
        if (before <= t && t < before + w) *out = (int)(sh.few[j] >> 32);
        before += w;
      }
    return;
  }

  // the chunks' sums, and to each what it keeps of the list
  const int chunk = slice / WAVES;
  if (n > T) {
    r.parts(n, plan.bin, plan.bin);
    cut = r.end_in(n, plan.bin, plan.bin, !by_count, by_count ? (uint32_t)(set.k - (int)plan.before) : 1,
                   by_count ? 0 : plan.before, plan.goal, upto);
  }
#pragma unroll
  for (int e = 0; e < OWN; ++e) sh.bins[OWN * threadIdx.x + e] = sums[e];
  if (n > T) {
    __syncthreads();
    for (int j = threadIdx.x; j < n; j += T) {
      const unsigned long long w = r.kept(sh.list[j], cut);
      if (w) atomicAdd(&sh.bins[(uint32_t)sh.list[j] / (uint32_t)chunk], w);
    }
  } else if (n) {
    cut = r.end_among((int)threadIdx.x < n ? l0 : ~0ull, n, by_count, plan, chunk);
  }
  __syncthreads();
  const int at = r.chunk_of(u, before, t) * chunk;
  r.draw(at, min(at + chunk, a.vocab), cut, before, t, out);
}

// Logits of a slice: about 1024 workgroups over all rows, between 2048 and 16384
// logits each.  Measured with 512, 1024, 2048 and 4096 of them, half of the rows with
// top-k, half with top-p: 72 rows of 151643 fp32 62, 60, 65, 97 us; 512 of 32000 fp16 71,
// 77, 75, 132; 2000 of 8192 bf16 90, 85, 103, 135; 4096 of 1000 fp32 85, 78, 79, 79;
// 300 of 128256 fp16 112, 112, 112, 116; 8 of 128256 and 32 of 32000 30 and 25 with any.
int slice_of(int64_t rows, int vocab) {
  const int64_t each = rows * vocab / (1024 * STEP) * STEP;
  const int64_t least = ((int64_t)vocab + MOST_SLICES * STEP - 1) / (MOST_SLICES * STEP) * STEP;
  const int64_t s = each < 8 * STEP ? each : 8 * STEP;
  return (int)(s < least ? least : s);
}
int slices_of(int64_t rows, int vocab) {
  const int s = slice_of(rows, vocab);
  return (vocab + s - 1) / s;
}

template <int TYPE>
hipError_t launch(const SampleArgs& a, hipStream_t s) {
  const int slice = slice_of(a.rows, a.vocab), slices = slices_of(a.rows, a.vocab);
  const dim3 grid((unsigned)a.rows * (unsigned)slices), threads(T);
  hipLaunchKernelGGL(sample_scan_kernel<TYPE>, grid, threads, 0, s, a, slices, slice);
  if (a.top_k || a.top_p) hipLaunchKernelGGL(sample_bins_kernel<TYPE>, grid, threads, 0, s, a, slices, slice);
  hipLaunchKernelGGL(sample_draw_kernel<TYPE>, grid, threads, 0, s, a, slices, slice);
  return hipGetLastError();
}

}  // namespace

// (Past 2^24 logits a slice has 16384, and with fewer there are at most 2048 slices
// and one a row: fewer than 2^23 are asked for where rows * ceil(vocab / 16384) is.)
bool sample_fits(int rows, int vocab) { return (int64_t)rows * slices_of(rows, vocab) < 1 << 23 && rows < 1 << 21; }
size_t sample_ws_bytes(int rows, int vocab) { return work_bytes(rows, slices_of(rows, vocab)); }

hipError_t launch_sample(const SampleArgs& a, hipStream_t s) {
  return a.type == 0 ? launch<0>(a, s) : a.type == 1 ? launch<1>(a, s) : launch<2>(a, s);
}

}  // namespace qg
