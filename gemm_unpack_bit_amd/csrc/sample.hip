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
// histogram, where a row has top-k or top-p), sample_sums_kernel (the list, and
// the sum of what is kept for certain); a workgroup per row does the rest
// (sample_draw_kernel).
//
// Bound: for one row the launches; for many the three times that a logit is read
// (once from memory, then from the caches) and a weight's 20 operations of 64
// bits, twice with top-p.
#include <type_traits>

#include "attn_common.hpp"
#include "step.hpp"

namespace qg {
namespace {

constexpr int BINS = 1024;  // and at most so many chunks, of which a slice has one per wave
constexpr int CAP = 4096;   // elements listed
constexpr int T = 256;      // threads of every workgroup
constexpr int WAVES = T / 64, PIECE = 8, STEP = PIECE * T, MOST_SLICES = BINS / WAVES;
constexpr int OWN = BINS / T;  // bins (or chunks) of a thread

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
  int* listed;                             // [rows]
  Part* parts;                             // [rows][slices]
  __device__ __forceinline__ Work(void* ws, int64_t rows, int slices) {
    char* p = reinterpret_cast<char*>(ws);
    bins = reinterpret_cast<unsigned long long*>(p), p += rows * BINS * 8;
    list = reinterpret_cast<unsigned long long*>(p), p += rows * CAP * 8;
    parts = reinterpret_cast<Part*>(p), p += rows * slices * 16;
    sums = reinterpret_cast<unsigned long long*>(p), p += rows * slices * (8 * WAVES);
    listed = reinterpret_cast<int*>(p);
  }
};
constexpr size_t work_bytes(int64_t rows, int slices) {
  return (size_t)(rows * (BINS * 8 + CAP * 8 + 4) + rows * slices * (16 + 8 * WAVES));
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
// PIECE logits from i on; those from `end` on are -infinity.  (Rows may begin at
// any element.)
template <int TYPE>
__device__ __forceinline__ void load_piece(const void* row, int i, int end, float (&v)[PIECE]) {
  if (i + PIECE <= end) {
    if constexpr (TYPE == 2) {
      typedef float loose4 __attribute__((ext_vector_type(4), aligned(4)));
      const float* p = static_cast<const float*>(row) + i;
      const f4 a = *reinterpret_cast<const loose4*>(p), b = *reinterpret_cast<const loose4*>(p + 4);
#pragma unroll
      for (int e = 0; e < 4; ++e) v[e] = a[e], v[4 + e] = b[e];
    } else {
      typedef uint32_t loose __attribute__((ext_vector_type(4), aligned(2)));
      const u4 a = *reinterpret_cast<const loose*>(static_cast<const uint16_t*>(row) + i);
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const uint16_t h = (uint16_t)(a[e / 2] >> (16 * (e & 1)));
        v[e] = TYPE == 0 ? F16::value(h) : BF16::value(h);
      }
    }
#pragma unroll
    for (int e = 0; e < PIECE; ++e) v[e] = clean(v[e]);
  } else {
#pragma unroll
    for (int e = 0; e < PIECE; ++e) v[e] = i + e < end ? clean(logit_at<TYPE>(row, i + e)) : NEG_INF;
  }
}

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

// The bin of a logit l <= M: the same or a later one for every smaller l.
struct Binning {
  float most, by;
  __device__ __forceinline__ Binning(const Top& t) : most(t.most()) {
    const float width = most - t.least;
    by = width > 0.f && width < 3e38f ? (float)BINS / width : 0.f;
  }
  // in bins from the largest logit on; past the last one (and NaN, of
  // infinities) the last one
  __device__ __forceinline__ float at(float l) const {
    const float d = (most - l) * by;
    return l == most ? 0.f : d < (float)BINS - 0.001f ? d : (float)BINS - 0.001f;
  }
  __device__ __forceinline__ int operator()(float l) const { return (int)at(l); }
  // a 1024th part of its bin, the same order
  __device__ __forceinline__ int part(float l) const {
    const float d = at(l);
    return (int)((d - (float)(int)d) * (float)BINS);
  }
};

// What follows from a row's histogram (a thread's bins: mine), the same in every
// workgroup of the row; all threads.
__device__ __forceinline__ Plan plan_of(const SampleArgs& a, const Settings& set, const unsigned long long (&mine)[OWN],
                                        unsigned long long* red, Plan* shared) {
  const bool by_count = set.by_count(a.vocab), by_weight = set.by_weight();
  if (!by_count && !by_weight) return Plan{CUT_NONE, BINS, 0, 0.0, 0};
  unsigned long long sum = 0, total;
#pragma unroll
  for (int e = 0; e < OWN; ++e) sum += mine[e];
  if (threadIdx.x == 0) *shared = Plan{CUT_NONE, BINS, 0, 0.0, 0};
  unsigned long long before = block_scan64(sum, total, red) - sum;
  // by count: the first bin with k elements up to it (all may be fewer); by
  // weight: the first up to which the weights reach p S
  const double goal = by_count ? (double)set.k : set.p * (double)total;
#pragma unroll
  for (int e = 0; e < OWN; ++e) {
    const unsigned long long upto = before + mine[e];
    const int b = OWN * threadIdx.x + e;
    if ((double)upto >= goal && (b == 0 || (double)before < goal)) {
      Plan p{CUT_BIN, b, before, goal, total};
      if (by_count) p.mode = upto <= CAP ? CUT_FEW : by_weight ? CUT_MANY : CUT_BIN;
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
#pragma unroll 4
  for (int i = begin + PIECE * threadIdx.x; i < end; i += STEP) {
    float v[PIECE];
    load_piece<TYPE>(x, i, end, v);
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
  }
  unsigned long long best = wave_max64((unsigned long long)key_of(most) << 32 | (uint32_t)~at);
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
    if (s == 0) w.listed[row] = 0;
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
  for (int i = threadIdx.x; i < BINS; i += T) bins[i] = 0;
  const Top top = top_of(part_of(w.parts + (int64_t)row * slices, slices), red);  // (with barriers)
  const Binning bin(top);
  const Weigh weigh{(double)top.most(), set.by};
  const int begin = s * slice, end = min(begin + slice, a.vocab);
  const void* x = static_cast<const char*>(a.logits) + (int64_t)row * a.row_bytes;
  uint32_t* counts = reinterpret_cast<uint32_t*>(bins);
#pragma unroll 2
  for (int i = begin + PIECE * threadIdx.x; i < end; i += STEP) {
    float v[PIECE];
    load_piece<TYPE>(x, i, end, v);
    if (by_count) {
#pragma unroll
      for (int e = 0; e < PIECE; ++e)
        if (v[e] != NEG_INF) atomicAdd(&counts[bin(v[e])], 1u);
    } else {
#pragma unroll
      for (int e = 0; e < PIECE; ++e) {
        const unsigned long long f = fixed(weigh(v[e]));
        if (f) atomicAdd(&bins[bin(v[e])], f);
      }
    }
  }
  __syncthreads();
  for (int i = threadIdx.x; i < BINS; i += T) {
    const unsigned long long f = by_count ? counts[i] : bins[i];
    if (f) atomicAdd(&w.bins[(int64_t)row * BINS + i], f);
  }
}

// The slice's elements of the bin in which the prefix ends go into the list (or
// those of all bins up to it); the weights that it keeps of the bins in front of
// it are summed, by chunks: a wave has a run of the slice.
template <int TYPE>
__global__ void __launch_bounds__(T) sample_sums_kernel(SampleArgs a, int slices, int slice) {
  __shared__ unsigned long long red[2 * WAVES];
  __shared__ Plan plan_s;
  __shared__ uint16_t list[CAP];  // places in the slice
  __shared__ int listed, place;
  const int row = blockIdx.x / slices, s = blockIdx.x % slices;
  if (threadIdx.x == 0) listed = 0;
  const Work w(a.ws, a.rows, slices);
  const Part part = part_of(w.parts + (int64_t)row * slices, slices);
  unsigned long long mine[OWN];
  own_bins(a, w.bins + (int64_t)row * BINS, mine);
  const Settings set(a, row);
  if (set.greedy) return;
  const Plan plan = plan_of(a, set, mine, red, &plan_s);
  if (plan.mode == CUT_MANY) return;
  const Top top = top_of(part, red);  // (with barriers)
  const Binning bin(top);
  const Weigh weigh{(double)top.most(), set.by};
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int first = s * slice, begin = first + wave * (slice / WAVES), end = min(begin + slice / WAVES, a.vocab);
  const void* x = static_cast<const char*>(a.logits) + (int64_t)row * a.row_bytes;
  unsigned long long sum = 0;
#pragma unroll 2
  for (int i = begin + PIECE * lane; i < end; i += PIECE * 64) {
    float v[PIECE];
    load_piece<TYPE>(x, i, end, v);
#pragma unroll
    for (int e = 0; e < PIECE; ++e) {
      const int b = plan.mode == CUT_NONE ? 0 : bin(v[e]);
      if (plan.mode != CUT_FEW && b < plan.bin) {
        const double p = weigh(v[e]);
        sum += p >= set.least ? fixed(p) : 0;
      }
      if (plan.mode != CUT_NONE && (plan.mode == CUT_FEW ? b <= plan.bin : b == plan.bin) && v[e] != NEG_INF) {
        const int at = atomicAdd(&listed, 1);
        if (at < CAP) list[at] = (uint16_t)(i + e - first);
      }
    }
  }
  sum = wave_scan64(sum);
  if (lane == 63) w.sums[((int64_t)row * slices + s) * WAVES + wave] = sum;
  if (plan.mode == CUT_NONE) return;
  __syncthreads();
  if (threadIdx.x == 0 && listed) place = atomicAdd(&w.listed[row], listed);
  __syncthreads();
  // (more than CAP in all: the list is not used, and not filled past its end)
  for (int j = threadIdx.x; j < min(listed, CAP) && place + j < CAP; j += T) {
    const int i = first + list[j];
    w.list[(int64_t)row * CAP + place + j] = (unsigned long long)~key_of(clean(logit_at<TYPE>(x, i))) << 32 | (uint32_t)i;
  }
}

// ---------------------------------------------------------------------------
// rows
// ---------------------------------------------------------------------------

// the place of a draw in a sum of weights
__device__ __forceinline__ unsigned long long target_of(float u, unsigned long long total) {
  const double t = (double)u * (double)total;
  if (!(t > 0.0)) return 0;
  return t < (double)total ? (unsigned long long)t : total - 1;
}

__device__ __forceinline__ int power_of_two(int n) { return n < 2 ? 1 : 1 << (32 - __builtin_clz(n - 1)); }

struct Shared {
  unsigned long long list[CAP];
  unsigned long long bins[BINS];  // of counts, weights or chunks' sums
  uint32_t counts[BINS];
  unsigned long long red[2 * WAVES];
  unsigned long long found;
  Plan plan;
  uint32_t key0, key1;
  int n, at;
};

// Sorts E entries a thread upwards (entry T e + thread, n of them, a power of
// two): partners within a wave change places by lanes, others within a thread or
// through the list.
template <int E>
__device__ __forceinline__ void sort_held(unsigned long long* list, int n) {
  const int t = threadIdx.x;
  unsigned long long v[E];
#pragma unroll
  for (int e = 0; e < E; ++e) v[e] = T * e + t < n ? list[T * e + t] : 0;
  for (int k = 2; k <= n; k <<= 1) {
    // a place takes the smaller one of a pair, or the larger
    auto take = [&](int e, unsigned long long o, int j) {
      const int i = T * e + t;
      v[e] = (o < v[e]) == (((i & j) == 0) == ((i & k) == 0)) ? o : v[e];
    };
    auto lanes = [&](auto by) {
      constexpr int J = decltype(by)::value;
#pragma unroll
      for (int e = 0; e < E; ++e) take(e, lane_xor<J>(v[e]), J);
    };
#pragma unroll
    for (int j = E / 2; j > 0; j >>= 1)
      if (k > T * j) {
#pragma unroll
        for (int e = 0; e < E; ++e)
          if (!(e & j)) {
            const unsigned long long x = v[e], y = v[e | j];
            take(e, y, T * j);
            take(e | j, x, T * j);
          }
      }
    for (int j = min(k, T) >> 1; j >= 64; j >>= 1) {
      __syncthreads();
#pragma unroll
      for (int e = 0; e < E; ++e)
        if (T * e + t < n) list[T * e + t] = v[e];
      __syncthreads();
#pragma unroll
      for (int e = 0; e < E; ++e)
        if (T * e + t < n) take(e, list[(T * e + t) ^ j], j);
    }
    if (k >= 64) lanes(std::integral_constant<int, 32>{});
    if (k >= 32) lanes(std::integral_constant<int, 16>{});
    if (k >= 16) lanes(std::integral_constant<int, 8>{});
    if (k >= 8) lanes(std::integral_constant<int, 4>{});
    if (k >= 4) lanes(std::integral_constant<int, 2>{});
    lanes(std::integral_constant<int, 1>{});
  }
  __syncthreads();
#pragma unroll
  for (int e = 0; e < E; ++e)
    if (T * e + t < n) list[T * e + t] = v[e];
}

// Sorts list[0 .. n) (n a power of two up to CAP) upwards; the whole workgroup,
// barriers on both sides.
__device__ __forceinline__ void sort(unsigned long long* list, int n) {
  __syncthreads();
  if (n <= T) {
    sort_held<1>(list, n);
  } else if (n <= 4 * T) {
    sort_held<4>(list, n);
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
#pragma unroll 2
    for (int i = PIECE * threadIdx.x; i < a.vocab; i += STEP) {
      float v[PIECE];
      load_piece<TYPE>(x, i, a.vocab, v);
#pragma unroll
      for (int e = 0; e < PIECE; ++e)
        if (v[e] != NEG_INF) f(v[e], i + e);
    }
  }

  // Sorts the n entries that are in the list.
  __device__ __forceinline__ void order(int n) const {
    const int m = power_of_two(n);
    for (int i = n + threadIdx.x; i < m; i += T) sh.list[i] = ~0ull;
    sort(sh.list, m);
  }
  // The last of the n sorted entries that stays.  By count: the `want`th (from
  // 1).  By weight: the last with less than `goal` in front of it, `before` of
  // that in front of the list (the first one, if none has).  `upto`: the weights
  // up to and with it.
  __device__ __forceinline__ int last_of(int n, bool by_weight, uint32_t want, unsigned long long before, double goal,
                                         unsigned long long& upto) const {
    const int each = (n + T - 1) / T, j0 = each * (int)threadIdx.x, j1 = min(j0 + each, n);  // a thread's entries
    unsigned long long total, sum = 0;
    for (int j = j0; j < j1; ++j) sum += weight_of(key_in(sh.list[j]));
    if (threadIdx.x == 0) sh.at = by_weight ? 0 : max((int)min(want, (uint32_t)n) - 1, 0);
    sum = scan(sum, total) - sum;
    if (by_weight) {
      int last = 0;
      unsigned long long at = before + sum;
      for (int j = j0; j < j1; ++j) {
        last = (double)at < goal ? j : last;
        at += weight_of(key_in(sh.list[j]));
      }
      if (last) atomicMax(&sh.at, last);
      __syncthreads();
    }
    const int l = sh.at;
    if (j0 <= l && l < j1) {
      for (int j = j0; j <= l; ++j) sum += weight_of(key_in(sh.list[j]));
      sh.found = sum;
    }
    __syncthreads();
    upto = n ? sh.found : 0;
    __syncthreads();
    return l;
  }

  // Sums over sh.bins (a thread's OWN ones side by side), in place.
  __device__ __forceinline__ void sum_bins() const {
    unsigned long long mine[OWN], sum = 0, total;
#pragma unroll
    for (int e = 0; e < OWN; ++e) mine[e] = sum += sh.bins[OWN * threadIdx.x + e];
    const unsigned long long before = scan(sum, total) - sum;
#pragma unroll
    for (int e = 0; e < OWN; ++e) sh.bins[OWN * threadIdx.x + e] = before + mine[e];
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

  // The end of a prefix anywhere in the row, by the row itself: where the list
  // cannot say (thousands of elements in one bin, or both criteria over as many).
  // Counts or weights by ranges of keys, each about a 1000th of the last, until
  // the range in which the prefix ends has few elements, or one key.
  __device__ __forceinline__ Cut search(bool by_weight, uint32_t want, double goal, unsigned long long& upto) const {
    uint32_t low = 0, high = ~0u;
    unsigned long long inside = 0;  // weights above `high`
    auto in = [&](float l) {
      const uint32_t k = key_of(l);
      return k >= low && k <= high;
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
      sum_bins();
      {  // counts likewise
        uint32_t mine[OWN], sum = 0;
#pragma unroll
        for (int e = 0; e < OWN; ++e) mine[e] = sum += sh.counts[OWN * threadIdx.x + e];
        unsigned long long total;
        const uint32_t before = (uint32_t)scan(sum, total) - sum;
#pragma unroll
        for (int e = 0; e < OWN; ++e) sh.counts[OWN * threadIdx.x + e] = before + mine[e];
        __syncthreads();
      }
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
      if (threadIdx.x == 0) sh.n = 0;
      __syncthreads();
      each([&](float l, int i) {
        if (in(l)) sh.list[atomicAdd(&sh.n, 1)] = (unsigned long long)~key_of(l) << 32 | (uint32_t)i;
      });
      __syncthreads();
      order(n);
      const int j = last_of(n, by_weight, want, inside, goal, upto);
      upto += inside;
      const unsigned long long entry = sh.list[j];
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
    uint32_t seen = 0;
    for (int i0 = 0; i0 < a.vocab && seen < m; i0 += STEP) {
      const int i = i0 + PIECE * threadIdx.x;
      float v[PIECE];
      uint32_t mine = 0;
      if (i < a.vocab) {
        load_piece<TYPE>(x, i, a.vocab, v);
#pragma unroll
        for (int e = 0; e < PIECE; ++e) mine += v[e] != NEG_INF && key_of(v[e]) == high;
      }
      unsigned long long all;
      uint32_t at = seen + (uint32_t)scan(mine, all) - mine;
      if (mine)
#pragma unroll
        for (int e = 0; e < PIECE; ++e)
          if (v[e] != NEG_INF && key_of(v[e]) == high && ++at == m) sh.at = i + e;
      seen += (uint32_t)all;
    }
    __syncthreads();
    const int place = sh.at;
    __syncthreads();
    upto = inside + (unsigned long long)m * w;
    return Cut{high, place};
  }

  // The end of a prefix among the n listed elements of one bin, `before` (counts
  // or weights) in front of them: first by 1024 parts of the bin, then by the
  // sorted elements of one part.  The entries that stay are those up to the cut.
  __device__ __forceinline__ Cut end_in_bin(int n, bool by_weight, unsigned long long before, double goal) const {
    for (int i = threadIdx.x; i < BINS; i += T) sh.bins[i] = 0;
    if (threadIdx.x == 0) sh.n = 0;
    __syncthreads();
    for (int j = threadIdx.x; j < n; j += T) {
      const uint32_t key = key_in(sh.list[j]);
      atomicAdd(&sh.bins[bin.part(logit_of(key))], by_weight ? weight_of(key) : 1ull);
    }
    __syncthreads();
    sum_bins();
    const int r = first_bin([&](int i) { return (double)(before + sh.bins[i]) >= goal; });
    before += r ? sh.bins[r - 1] : 0;
    // that part's entries in front of the others (which stay where they are
    // listed in global memory)
    constexpr int MORE = CAP / T;
    unsigned long long mine[MORE];
    uint32_t are = 0;
#pragma unroll
    for (int e = 0; e < MORE; ++e) {
      const int j = T * e + threadIdx.x;
      if (T * e >= n) break;
      mine[e] = j < n ? sh.list[j] : 0;
      are |= j < n && bin.part(logit_of(key_in(mine[e]))) == r ? 1u << e : 0u;
    }
    __syncthreads();
#pragma unroll
    for (int e = 0; e < MORE; ++e)
      if (are >> e & 1) sh.list[atomicAdd(&sh.n, 1)] = mine[e];
    __syncthreads();
    const int m = sh.n;
    order(m);
    unsigned long long upto;
    const int l = last_of(m, by_weight, by_weight ? 1 : (uint32_t)(goal - (double)before), before, goal, upto);
    const unsigned long long entry = sh.list[l];
    __syncthreads();
    return Cut{key_in(entry), (int)(uint32_t)entry};
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
};

template <int TYPE>
__global__ void __launch_bounds__(T) sample_draw_kernel(SampleArgs a, int slices, int slice) {
  __shared__ Shared sh;
  const int row = blockIdx.x;
  const Work wk(a.ws, a.rows, slices);
  // (all that is needed of memory is asked for at once)
  const Part part = part_of(wk.parts + (int64_t)row * slices, slices);
  unsigned long long mine[OWN], sums[OWN];
  own_bins(a, wk.bins + (int64_t)row * BINS, mine);
#pragma unroll
  for (int e = 0; e < OWN; ++e) {
    const int c = OWN * threadIdx.x + e;
    sums[e] = c < slices * WAVES ? wk.sums[(int64_t)row * slices * WAVES + c] : 0;
  }
  const int listed = wk.listed[row];
  const unsigned long long* list = wk.list + (int64_t)row * CAP;
  const Settings set(a, row);
  int32_t* out = a.out + row;
  const float u = a.u[row];
  const Top top = top_of(part, sh.red);
  if (set.greedy || top.most() == NEG_INF) {
    if (threadIdx.x == 0) *out = top.most() == NEG_INF ? -1 : top.place();
    return;
  }
  const OneRow<TYPE> r{a, set, sh, static_cast<const char*>(a.logits) + (int64_t)row * a.row_bytes, Binning(top),
                       Weigh{(double)top.most(), set.by}};
  const bool by_count = set.by_count(a.vocab), by_weight = set.by_weight();
  if (by_count || by_weight)
    for (int j = threadIdx.x; j < min(listed, CAP); j += T) sh.list[j] = list[j];
  const Plan plan = plan_of(a, set, mine, sh.red, &sh.plan);  // (with barriers)
  unsigned long long total, upto;

  if (plan.mode == CUT_MANY || (plan.mode != CUT_NONE && listed > CAP)) {
    // the row alone, from its logits
    Cut cut{0, 0};
    double goal = plan.goal;
    if (by_count) {
      cut = r.search(false, (uint32_t)set.k, 0.0, upto);
      goal = set.p * (double)upto;
    }
    if (by_weight) cut = r.search(true, 1, goal, upto);
    total = r.draw(0, a.vocab, cut, 0, ~0ull >> 1, out);
    r.draw(0, a.vocab, cut, 0, target_of(u, total), out);
    return;
  }

  const int n = plan.mode == CUT_NONE ? 0 : listed;
  if (plan.mode == CUT_FEW) {
    r.order(n);
    int kept = by_count ? min(set.k, n) : n;
    if (by_weight) {
      r.last_of(n, false, (uint32_t)kept, 0, 0.0, upto);
      kept = min(kept, 1 + r.last_of(n, true, 1, 0, set.p * (double)upto, upto));
    }
    // (min-p keeps a prefix of these; then by index)
    const int m = power_of_two(kept);
    __syncthreads();
    for (int j = threadIdx.x; j < m; j += T) {
      const unsigned long long entry = sh.list[j];
      const bool stays = j < kept && (j == 0 || r.weigh(logit_of(r.key_in(entry))) >= set.least);
      sh.list[j] = stays ? entry << 32 | entry >> 32 : ~0ull;
    }
    sort(sh.list, m);
    const int each = (m + T - 1) / T, j0 = min(each * (int)threadIdx.x, m), j1 = min(j0 + each, m);
    unsigned long long sum = 0;
    auto weight_at = [&](int j) { return sh.list[j] == ~0ull ? 0ull : r.weight_of(~(uint32_t)sh.list[j]); };
    for (int j = j0; j < j1; ++j) sum += weight_at(j);
    sum = r.scan(sum, total) - sum;
    const unsigned long long t = target_of(u, total);
    for (int j = j0; j < j1; ++j) {
      const unsigned long long w = weight_at(j);
      if (sum <= t && t < sum + w) *out = (int)(sh.list[j] >> 32);
      sum += w;
    }
    return;
  }

  // the chunks' sums, and to each what it keeps of the list
  Cut cut{0, 0};
  if (n) cut = r.end_in_bin(n, !by_count, plan.before, plan.goal);
#pragma unroll
  for (int e = 0; e < OWN; ++e) sh.bins[OWN * threadIdx.x + e] = sums[e];
  __syncthreads();
  const int chunk = slice / WAVES;
  for (int j = threadIdx.x; j < n; j += T) {
    const unsigned long long entry = list[j];
    const uint32_t key = r.key_in(entry), i = (uint32_t)entry;
    if (key < cut.key || (key == cut.key && (int)i > cut.at)) continue;
    const double p = r.weigh(logit_of(key));
    if (p >= set.least) atomicAdd(&sh.bins[i / (uint32_t)chunk], fixed(p));
  }
  __syncthreads();
  unsigned long long sum = 0, own[OWN];
#pragma unroll
  for (int e = 0; e < OWN; ++e) sum += own[e] = sh.bins[OWN * threadIdx.x + e];
  unsigned long long at = r.scan(sum, total) - sum;
  const unsigned long long t = target_of(u, total);
  if (threadIdx.x == 0) sh.key0 = 0, sh.found = 0;
  __syncthreads();
#pragma unroll
  for (int e = 0; e < OWN; ++e) {
    if (at <= t && t < at + own[e]) sh.key0 = OWN * threadIdx.x + e, sh.found = at;
    at += own[e];
  }
  __syncthreads();
  const int begin = (int)sh.key0 * chunk, end = min(begin + chunk, a.vocab);
  r.draw(begin, end, cut, sh.found, t, out);
}

// Logits of a slice: about 1024 workgroups over all rows, between 2048 and
// 16384 of them each.
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
  const dim3 grid((unsigned)a.rows * (unsigned)slices), rows((unsigned)a.rows), threads(T);
  hipLaunchKernelGGL(sample_scan_kernel<TYPE>, grid, threads, 0, s, a, slices, slice);
  if (a.top_k || a.top_p) hipLaunchKernelGGL(sample_bins_kernel<TYPE>, grid, threads, 0, s, a, slices, slice);
  hipLaunchKernelGGL(sample_sums_kernel<TYPE>, grid, threads, 0, s, a, slices, slice);
  hipLaunchKernelGGL(sample_draw_kernel<TYPE>, rows, threads, 0, s, a, slices, slice);
  return hipGetLastError();
}

}  // namespace

bool sample_fits(int rows, int vocab) { return (int64_t)rows * slices_of(rows, vocab) < 1 << 23 && rows < 1 << 21; }
size_t sample_ws_bytes(int rows, int vocab) { return work_bytes(rows, slices_of(rows, vocab)); }

hipError_t launch_sample(const SampleArgs& a, hipStream_t s) {
  return a.type == 0 ? launch<0>(a, s) : a.type == 1 ? launch<1>(a, s) : launch<2>(a, s);
}

}  // namespace qg
