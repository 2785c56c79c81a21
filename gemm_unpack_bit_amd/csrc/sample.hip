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
// its smallest, with counts and weights, says in which bin the prefix ends; the
// row is searched for the elements of that bin alone (or, where they are few, of
// all bins up to it), and these are sorted.
//
// Bound: the logits are read once from memory and up to three times more from
// the caches, and every weight takes about 20 operations of 64 bits; for one row
// it is the launches.  Kernels: `slices` of the vocabulary for what touches every
// logit (scan, histogram, sums), a workgroup per row for what follows from it
// (cut, draw).
#include "attn_common.hpp"
#include "step.hpp"

namespace qg {
namespace {

constexpr int BINS = 1024, THREADS = 1024;  // (a thread a bin)
constexpr int CAP = 4096;                   // elements sorted at once
constexpr int SLICE_THREADS = 256, PIECE = 8;
constexpr double ONE = 0x1p42;  // the largest logit's weight

// what a slice of a row leaves: its largest logit's key and place (the first
// one), its smallest finite logit
struct Part {
  uint32_t key;
  int at;
  float least;
  int pad;
};
// where the kept prefix ends: keys above `key`, and of those equal the ones up
// to index `at`; done: the row's token is chosen
struct Cut {
  uint32_t key;
  int at, done, pad;
};

struct Work {
  unsigned long long *weights, *sums;  // [rows][BINS], [rows][slices]
  uint32_t* counts;                    // [rows][BINS]
  Cut* cuts;                           // [rows]
  Part* parts;                         // [rows][slices]
  __device__ __host__ __forceinline__ Work(void* ws, int64_t rows, int slices) {
    char* p = reinterpret_cast<char*>(ws);
    weights = reinterpret_cast<unsigned long long*>(p), p += rows * BINS * 8;
    sums = reinterpret_cast<unsigned long long*>(p), p += (rows * slices * 8 + 15) / 16 * 16;
    counts = reinterpret_cast<uint32_t*>(p), p += rows * BINS * 4;
    cuts = reinterpret_cast<Cut*>(p), p += rows * 16;
    parts = reinterpret_cast<Part*>(p);
  }
};
constexpr size_t work_bytes(int64_t rows, int slices) {
  return (size_t)(rows * BINS * 12 + (rows * slices * 8 + 15) / 16 * 16 + rows * 16 + rows * slices * 16);
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

// Weights.  2^x for x <= 0 by its power series around the nearest whole number:
// |f ln 2| <= 0.347, so the 12th power's term, the first left out, is 2^-47.
struct Weigh {
  double top, by;  // M, log2(e) / T
  __device__ __forceinline__ double operator()(float l) const {
    const double x = l == (float)top ? 0.0 : ((double)l - top) * by;
    const double n = __builtin_rint(x), f = x - n;
    double p = 4.44553827187081e-10;  // ln(2)^11 / 11!
    p = fma(p, f, 7.054911620801121e-09);
    p = fma(p, f, 1.0178086009239696e-07);
    p = fma(p, f, 1.3215486790144305e-06);
    p = fma(p, f, 1.5252733804059838e-05);
    p = fma(p, f, 1.5403530393381606e-04);
    p = fma(p, f, 1.3333558146428441e-03);
    p = fma(p, f, 9.618129107628477e-03);
    p = fma(p, f, 5.5504108664821576e-02);
    p = fma(p, f, 2.402265069591007e-01);
    p = fma(p, f, 6.931471805599453e-01);
    p = fma(p, f, 1.0);
    // (below 2^-64, and where x is NaN, as of -infinity at an infinite T: none)
    return x > -64.0 ? __builtin_ldexp(p, (int)n) : 0.0;
  }
};
// as a whole number of 2^-42, rounded to nearest
__device__ __forceinline__ unsigned long long fixed(double w) {
  return __builtin_bit_cast(unsigned long long, fma(w, ONE, 0x1p52)) - __builtin_bit_cast(unsigned long long, 0x1p52);
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
  __device__ __forceinline__ bool cuts() const { return !greedy && (k > 0 || p < 1.0); }
};

// max over a wave; sums over the wave's lanes up to and with the lane's
__device__ __forceinline__ unsigned long long wave_max64(unsigned long long v) {
#pragma unroll
  for (int d = 32; d > 0; d >>= 1) {
    const unsigned long long o = __shfl_xor(v, d);
    v = o > v ? o : v;
  }
  return v;
}
__device__ __forceinline__ unsigned long long wave_scan64(unsigned long long v) {
  const int lane = threadIdx.x & 63;
#pragma unroll
  for (int d = 1; d < 64; d <<= 1) {
    const unsigned long long o = __shfl_up(v, d);
    if (lane >= d) v += o;
  }
  return v;
}

// A workgroup's THREADS threads: sums up to and with the thread's, and of all.
__device__ __forceinline__ unsigned long long block_scan64(unsigned long long v, unsigned long long& total,
                                                           unsigned long long* red) {
  const int lane = threadIdx.x & 63, w = threadIdx.x >> 6;
  v = wave_scan64(v);
  if (lane == 63) red[w] = v;
  __syncthreads();
  unsigned long long before = 0, all = 0;
#pragma unroll
  for (int i = 0; i < THREADS / 64; ++i) {
    before += i < w ? red[i] : 0;
    all += red[i];
  }
  __syncthreads();
  total = all;
  return before + v;
}

// The row's largest logit's key and first place (as key << 32 | ~place), and
// its smallest finite logit, from the slices' parts; the whole workgroup.
struct Top {
  unsigned long long best;
  float least;
  __device__ __forceinline__ float most() const { return logit_of((uint32_t)(best >> 32)); }
  __device__ __forceinline__ int place() const { return (int)~(uint32_t)best; }
};
template <int T>
__device__ __forceinline__ Top top_of(const Part* parts, int slices, unsigned long long* red) {
  unsigned long long best = 0, low = 0;
  for (int i = threadIdx.x; i < slices; i += T) {
    const Part p = parts[i];
    const unsigned long long b = (unsigned long long)p.key << 32 | (uint32_t)~p.at;
    best = b > best ? b : best;
    const unsigned long long l = (uint32_t)~key_of(p.least);
    low = l > low ? l : low;
  }
  best = wave_max64(best);
  low = wave_max64(low);
  if ((threadIdx.x & 63) == 0) red[threadIdx.x >> 6] = best, red[T / 64 + (threadIdx.x >> 6)] = low;
  __syncthreads();
#pragma unroll
  for (int i = 0; i < T / 64; ++i) {
    best = red[i] > best ? red[i] : best;
    low = red[T / 64 + i] > low ? red[T / 64 + i] : low;
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
  __device__ __forceinline__ int operator()(float l) const {
    const float d = (most - l) * by;
    return l == most ? 0 : d < (float)(BINS - 1) ? (int)d : BINS - 1;  // (NaN, of infinities: the last)
  }
};

// ---------------------------------------------------------------------------
// slices
// ---------------------------------------------------------------------------

template <int TYPE>
__global__ void __launch_bounds__(SLICE_THREADS) sample_scan_kernel(SampleArgs a, int slices, int slice) {
  __shared__ unsigned long long red[2 * SLICE_THREADS / 64];
  const int row = blockIdx.x / slices, s = blockIdx.x % slices;
  const Work w(a.ws, a.rows, slices);
  const int begin = s * slice, end = min(begin + slice, a.vocab);
  const void* x = static_cast<const char*>(a.logits) + (int64_t)row * a.row_bytes;
  unsigned long long best = 0;
  float least = __builtin_inff();
#pragma unroll 2
  for (int i = begin + PIECE * threadIdx.x; i < end; i += PIECE * SLICE_THREADS) {
    float v[PIECE];
    load_piece<TYPE>(x, i, end, v);
#pragma unroll
    for (int e = 0; e < PIECE; ++e) {
      const unsigned long long b = (unsigned long long)key_of(v[e]) << 32 | (uint32_t)~(i + e);
      best = b > best ? b : best;
      least = v[e] > NEG_INF ? fminf(least, v[e]) : least;
    }
  }
  best = wave_max64(best);
#pragma unroll
  for (int d = 32; d > 0; d >>= 1) least = fminf(least, __shfl_xor(least, d));
  if ((threadIdx.x & 63) == 0) {
    red[threadIdx.x >> 6] = best;
    red[SLICE_THREADS / 64 + (threadIdx.x >> 6)] = __float_as_uint(least);
  }
  __syncthreads();
  if (threadIdx.x == 0) {
#pragma unroll
    for (int i = 0; i < SLICE_THREADS / 64; ++i) {
      best = red[i] > best ? red[i] : best;
      least = fminf(least, __uint_as_float((uint32_t)red[SLICE_THREADS / 64 + i]));
    }
    w.parts[(int64_t)row * slices + s] = Part{(uint32_t)(best >> 32), (int)~(uint32_t)best, least, 0};
  }
  // the row's histogram starts at 0, a part of it by each slice
  if (a.top_k || a.top_p)
    for (int i = s * SLICE_THREADS + threadIdx.x; i < BINS; i += slices * SLICE_THREADS) {
      w.weights[(int64_t)row * BINS + i] = 0;
      w.counts[(int64_t)row * BINS + i] = 0;
    }
}

template <int TYPE>
__global__ void __launch_bounds__(SLICE_THREADS) sample_histogram_kernel(SampleArgs a, int slices, int slice) {
  __shared__ unsigned long long red[2 * SLICE_THREADS / 64];
  __shared__ unsigned long long weights[BINS];
  __shared__ uint32_t counts[BINS];
  const int row = blockIdx.x / slices, s = blockIdx.x % slices;
  const Settings set(a, row);
  if (!set.cuts()) return;
  const Work w(a.ws, a.rows, slices);
  for (int i = threadIdx.x; i < BINS; i += SLICE_THREADS) weights[i] = 0, counts[i] = 0;
  const Top top = top_of<SLICE_THREADS>(w.parts + (int64_t)row * slices, slices, red);  // (with barriers)
  const Binning bin(top);
  const Weigh weigh{(double)top.most(), set.by};
  const int begin = s * slice, end = min(begin + slice, a.vocab);
  const void* x = static_cast<const char*>(a.logits) + (int64_t)row * a.row_bytes;
  for (int i = begin + PIECE * threadIdx.x; i < end; i += PIECE * SLICE_THREADS) {
    float v[PIECE];
    load_piece<TYPE>(x, i, end, v);
#pragma unroll
    for (int e = 0; e < PIECE; ++e) {
      if (v[e] == NEG_INF) continue;
      const int b = bin(v[e]);
      atomicAdd(&counts[b], 1u);
      if (set.p < 1.0) {
        const unsigned long long f = fixed(weigh(v[e]));
        if (f) atomicAdd(&weights[b], f);
      }
    }
  }
  __syncthreads();
  for (int i = threadIdx.x; i < BINS; i += SLICE_THREADS) {
    if (counts[i]) atomicAdd(&w.counts[(int64_t)row * BINS + i], counts[i]);
    if (weights[i]) atomicAdd(&w.weights[(int64_t)row * BINS + i], weights[i]);
  }
}

// the weights that a slice keeps
template <int TYPE>
__global__ void __launch_bounds__(SLICE_THREADS) sample_sums_kernel(SampleArgs a, int slices, int slice) {
  __shared__ unsigned long long red[2 * SLICE_THREADS / 64];
  const int row = blockIdx.x / slices, s = blockIdx.x % slices;
  const Work w(a.ws, a.rows, slices);
  const Settings set(a, row);
  if (set.greedy) return;
  Cut cut{0, 0, 0, 0};
  if (a.top_k || a.top_p) cut = w.cuts[row];
  if (cut.done) return;
  const Top top = top_of<SLICE_THREADS>(w.parts + (int64_t)row * slices, slices, red);
  const Weigh weigh{(double)top.most(), set.by};
  const int begin = s * slice, end = min(begin + slice, a.vocab);
  const void* x = static_cast<const char*>(a.logits) + (int64_t)row * a.row_bytes;
  unsigned long long sum = 0;
  for (int i = begin + PIECE * threadIdx.x; i < end; i += PIECE * SLICE_THREADS) {
    float v[PIECE];
    load_piece<TYPE>(x, i, end, v);
#pragma unroll
    for (int e = 0; e < PIECE; ++e) {
      const uint32_t key = key_of(v[e]);
      if (v[e] == NEG_INF || key < cut.key || (key == cut.key && i + e > cut.at)) continue;
      const double p = weigh(v[e]);
      sum += p >= set.least ? fixed(p) : 0;
    }
  }
  sum = wave_scan64(sum);
  if ((threadIdx.x & 63) == 63) red[threadIdx.x >> 6] = sum;
  __syncthreads();
  if (threadIdx.x == 0) {
    sum = 0;
#pragma unroll
    for (int i = 0; i < SLICE_THREADS / 64; ++i) sum += red[i];
    w.sums[(int64_t)row * slices + s] = sum;
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

// Sorts list[0 .. n) (n a power of two) upwards; the whole workgroup.
__device__ __forceinline__ void sort(unsigned long long* list, int n) {
  for (int k = 2; k <= n; k <<= 1)
    for (int j = k >> 1; j > 0; j >>= 1) {
      __syncthreads();
      for (int t = threadIdx.x; t < n / 2; t += THREADS) {
        const int i = ((t & ~(j - 1)) << 1) | (t & (j - 1)), o = i | j;
        const unsigned long long x = list[i], y = list[o];
        if ((x > y) == ((i & k) == 0)) list[i] = y, list[o] = x;
      }
    }
  __syncthreads();
}
__device__ __forceinline__ int power_of_two(int n) { return n < 2 ? 1 : 1 << (32 - __builtin_clz(n - 1)); }

struct Shared {
  unsigned long long list[CAP];
  unsigned long long weights[BINS];  // up to and with the bin
  uint32_t counts[BINS];
  unsigned long long red[2 * THREADS / 64];
  unsigned long long found;
  uint32_t key0, key1;
  int n, bin;
};

constexpr int EACH = CAP / THREADS;  // entries of a thread

template <int TYPE>
struct RowCut {
  const SampleArgs& a;
  Shared& sh;
  const void* x;
  const Binning bin;
  const Weigh weigh;

  // f(logit, index) for the row's elements that are not -infinity
  template <typename F>
  __device__ __forceinline__ void each(F&& f) const {
#pragma unroll 2
    for (int i = PIECE * threadIdx.x; i < a.vocab; i += PIECE * THREADS) {
      float v[PIECE];
      load_piece<TYPE>(x, i, a.vocab, v);
#pragma unroll
      for (int e = 0; e < PIECE; ++e)
        if (v[e] != NEG_INF) f(v[e], i + e);
    }
  }
  // Sorted entries: ~key << 32 | index, so falling logits, rising indexes.
  __device__ __forceinline__ static uint32_t key_in(unsigned long long entry) { return ~(uint32_t)(entry >> 32); }
  __device__ __forceinline__ unsigned long long weight_in(unsigned long long entry) const {
    return fixed(weigh(logit_of(key_in(entry))));
  }

  // The first bin up to which sums(bin) reaches what is wanted (reaches: false,
  // ..., false, true, ...), or the last one.
  template <typename F>
  __device__ __forceinline__ int first_bin(F&& reaches) const {
    if (threadIdx.x == 0) sh.bin = BINS - 1;
    __syncthreads();
    const int b = threadIdx.x;
    if (reaches(b) && (b == 0 || !reaches(b - 1))) sh.bin = b;
    __syncthreads();
    const int r = sh.bin;
    __syncthreads();
    return r;
  }
  // Turns the bins' own counts and weights (a bin a thread) into sums up to them.
  __device__ __forceinline__ void sum_bins(uint32_t count, unsigned long long weight) const {
    unsigned long long all;
    const unsigned long long c = block_scan64(count, all, sh.red), s = block_scan64(weight, all, sh.red);
    sh.counts[threadIdx.x] = (uint32_t)c;
    sh.weights[threadIdx.x] = s;
    __syncthreads();
  }

  // Puts the elements that `in` accepts into the list (at most CAP) and sorts
  // them; the entries behind them are the largest.
  template <typename F>
  __device__ __forceinline__ int gather(F&& in) const {
    if (threadIdx.x == 0) sh.n = 0;
    __syncthreads();
    each([&](float l, int i) {
      if (in(l)) {
        const int at = atomicAdd(&sh.n, 1);
        if (at < CAP) sh.list[at] = (unsigned long long)~key_of(l) << 32 | (uint32_t)i;
      }
    });
    __syncthreads();
    const int n = min(sh.n, CAP), m = power_of_two(n);
    for (int i = n + threadIdx.x; i < m; i += THREADS) sh.list[i] = ~0ull;
    sort(sh.list, m);
    return n;
  }
  // the weights of a thread's entries EACH * t .. and the sum in front of them
  __device__ __forceinline__ unsigned long long scan_list(int n, unsigned long long (&w)[EACH], unsigned long long& total) const {
    unsigned long long mine = 0;
#pragma unroll
    for (int e = 0; e < EACH; ++e) {
      const int j = EACH * threadIdx.x + e;
      w[e] = j < n ? weight_in(sh.list[j]) : 0;
      mine += w[e];
    }
    return block_scan64(mine, total, sh.red) - mine;
  }

  // The end of a prefix inside bin b.  By count: its `want`th element (from 1).
  // By weight: the last element in front of which the weights, `before` in front
  // of the bin, are less than `goal` (the bin's first, where goal is 0).  Returns
  // the cut and, in `upto`, the bin's weights up to and with it.
  __device__ __forceinline__ Cut end_in(int b, bool by_weight, uint32_t want, unsigned long long before, double goal,
                                        unsigned long long& upto) const {
    uint32_t low = 0, high = ~0u;  // keys looked at
    uint32_t n = sh.counts[b] - (b ? sh.counts[b - 1] : 0);
    unsigned long long inside = 0;  // weights of the bin above `high`
    auto in = [&](float l) {
      const uint32_t k = key_of(l);
      return bin(l) == b && k >= low && k <= high;
    };
    while (n > CAP) {
      // too many: bins of key ranges, until few are left or all are equal
      __syncthreads();
      if (threadIdx.x == 0) sh.key0 = ~0u, sh.key1 = 0;
      __syncthreads();
      uint32_t k0 = ~0u, k1 = 0;
      each([&](float l, int) {
        if (in(l)) k0 = min(k0, key_of(l)), k1 = max(k1, key_of(l));
      });
      if (k0 <= k1) atomicMin(&sh.key0, k0), atomicMax(&sh.key1, k1);
      __syncthreads();
      low = sh.key0, high = sh.key1;
      if (low == high) break;
      const int shift = max(0, 32 - __builtin_clz(high - low) - 10);
      sh.counts[threadIdx.x] = 0;
      sh.weights[threadIdx.x] = 0;
      __syncthreads();
      each([&](float l, int) {
        if (!in(l)) return;
        const uint32_t r = (high - key_of(l)) >> shift;
        atomicAdd(&sh.counts[r], 1u);
        atomicAdd(&sh.weights[r], fixed(weigh(l)));
      });
      __syncthreads();
      const uint32_t c = sh.counts[threadIdx.x];
      const unsigned long long s = sh.weights[threadIdx.x];
      __syncthreads();
      sum_bins(c, s);
      const int r = first_bin([&](int i) {
        return by_weight ? (double)(before + inside + sh.weights[i]) >= goal : sh.counts[i] >= want;
      });
      n = sh.counts[r] - (r ? sh.counts[r - 1] : 0);
      want -= r ? sh.counts[r - 1] : 0;
      inside += r ? sh.weights[r - 1] : 0;
      const uint32_t h = high - ((uint32_t)r << shift), l = h - ((1u << shift) - 1);
      high = h;
      low = l > h || l < low ? low : l;
    }
    if (n <= CAP) {
      n = gather(in);
      unsigned long long w[EACH], total;
      unsigned long long sum = scan_list(n, w, total);
      if (threadIdx.x == 0) sh.bin = by_weight ? 0 : (int)min(want, n) - 1;
      __syncthreads();
      int last = 0;  // the last entry that the weights in front of it leave in
      unsigned long long at = sum;
#pragma unroll
      for (int e = 0; e < EACH; ++e) {
        const int j = EACH * threadIdx.x + e;
        last = j < (int)n && (double)(before + inside + at) < goal ? j : last;
        at += w[e];
      }
      if (by_weight && last) atomicMax(&sh.bin, last);
      __syncthreads();
      const int j = max(sh.bin, 0);
#pragma unroll
      for (int e = 0; e < EACH; ++e) {
        sum += w[e];
        if (EACH * (int)threadIdx.x + e == j) sh.found = sum;
      }
      __syncthreads();
      upto = inside + sh.found;
      const unsigned long long entry = sh.list[j];
      __syncthreads();
      return Cut{key_in(entry), (int)(uint32_t)entry, 0, 0};
    }
    // all equal: the one of their number `m`, in the order of the vocabulary
    const unsigned long long w = fixed(weigh(logit_of(high)));
    uint32_t m = want;
    if (by_weight) {
      const double need = goal - (double)(before + inside);
      m = need > 0.0 ? (w ? (uint32_t)fmin(ceil(need / (double)w), (double)n) : n) : 1;
    }
    m = max(1u, min(m, n));
    uint32_t seen = 0;
    for (int i0 = 0; i0 < a.vocab && seen < m; i0 += PIECE * THREADS) {
      const int i = i0 + PIECE * threadIdx.x;
      float v[PIECE];
      uint32_t mine = 0;
      if (i < a.vocab) {
        load_piece<TYPE>(x, i, a.vocab, v);
#pragma unroll
        for (int e = 0; e < PIECE; ++e) mine += v[e] != NEG_INF && key_of(v[e]) == high;
      }
      unsigned long long all;
      uint32_t at = seen + (uint32_t)block_scan64(mine, all, sh.red) - mine;
      if (mine)
#pragma unroll
        for (int e = 0; e < PIECE; ++e)
          if (v[e] != NEG_INF && key_of(v[e]) == high && ++at == m) sh.bin = i + e;
      seen += (uint32_t)all;
    }
    __syncthreads();
    const int place = sh.bin;
    __syncthreads();
    upto = inside + (unsigned long long)m * w;
    return Cut{high, place, 0, 0};
  }
};

// Where the row's prefix ends, or, where it has few elements, its token.
template <int TYPE>
__global__ void __launch_bounds__(THREADS) sample_cut_kernel(SampleArgs a, int slices) {
  __shared__ Shared sh;
  const int row = blockIdx.x;
  const Settings set(a, row);
  if (set.greedy) return;
  const Work wk(a.ws, a.rows, slices);
  if (!set.cuts()) {
    if (threadIdx.x == 0) wk.cuts[row] = Cut{0, 0, 0, 0};
    return;
  }
  const Top top = top_of<THREADS>(wk.parts + (int64_t)row * slices, slices, sh.red);
  const RowCut<TYPE> r{a, sh, static_cast<const char*>(a.logits) + (int64_t)row * a.row_bytes, Binning(top),
                       Weigh{(double)top.most(), set.by}};
  r.sum_bins(wk.counts[(int64_t)row * BINS + threadIdx.x], wk.weights[(int64_t)row * BINS + threadIdx.x]);
  const uint32_t all = sh.counts[BINS - 1];
  const bool by_count = set.k > 0 && (uint32_t)set.k < all, by_weight = set.p < 1.0;
  if (!by_count && !by_weight) {
    if (threadIdx.x == 0) wk.cuts[row] = Cut{0, 0, 0, 0};
    return;
  }
  // the last bin that the prefix can reach
  int last = BINS - 1;
  if (by_count) last = r.first_bin([&](int b) { return sh.counts[b] >= (uint32_t)set.k; });
  if (by_weight && !by_count) {
    const double goal = set.p * (double)sh.weights[BINS - 1];
    last = r.first_bin([&](int b) { return (double)sh.weights[b] >= goal; });
  }
  if (sh.counts[last] <= CAP) {
    // few: all of them in the list, and the token from it
    const int n = r.gather([&](float l) { return r.bin(l) <= last; });
    unsigned long long w[EACH], total, sum;
    if (n == 0) {  // (no logit above -infinity)
      if (threadIdx.x == 0) wk.cuts[row] = Cut{0, 0, 0, 0};
      return;
    }
    sum = r.scan_list(n, w, total);
    const int nk = by_count ? min(set.k, n) : n;
    if (by_count) {  // the sum of the first nk
      unsigned long long s = sum;
#pragma unroll
      for (int e = 0; e < EACH; ++e) {
        s += w[e];
        if (EACH * (int)threadIdx.x + e == nk - 1) sh.found = s;
      }
      __syncthreads();
      total = sh.found;
    } else {
      total = sh.weights[BINS - 1];  // (of the row, not of the list)
    }
    const double goal = set.p * (double)total;
    if (threadIdx.x == 0) sh.n = 1;
    __syncthreads();
    int kept = 0;
#pragma unroll
    for (int e = 0; e < EACH; ++e) {
      const int j = EACH * threadIdx.x + e;
      const bool keep = j < nk && (j == 0 || !by_weight || (double)sum < goal) &&
                        r.weigh(logit_of(r.key_in(sh.list[j < n ? j : 0]))) >= set.least;
      kept = keep ? j + 1 : kept;
      sum += w[e];
    }
    if (kept) atomicMax(&sh.n, kept);
    __syncthreads();
    const int m = sh.n, m2 = power_of_two(m);
    // ... in the order of the vocabulary
    unsigned long long entry[EACH];
#pragma unroll
    for (int e = 0; e < EACH; ++e) entry[e] = sh.list[EACH * threadIdx.x + e];
    __syncthreads();
#pragma unroll
    for (int e = 0; e < EACH; ++e) {
      const int j = EACH * threadIdx.x + e;
      if (j < m2) sh.list[j] = j < m ? entry[e] << 32 | entry[e] >> 32 : ~0ull;
    }
    sort(sh.list, m2);
    unsigned long long mine = 0;
#pragma unroll
    for (int e = 0; e < EACH; ++e) {
      const int j = EACH * threadIdx.x + e;
      entry[e] = j < m ? sh.list[j] : 0;
      w[e] = j < m ? fixed(r.weigh(logit_of(~(uint32_t)entry[e]))) : 0;
      mine += w[e];
    }
    sum = block_scan64(mine, total, sh.red) - mine;
    const unsigned long long t = target_of(a.u[row], total);
#pragma unroll
    for (int e = 0; e < EACH; ++e) {
      if (sum <= t && t < sum + w[e]) a.out[row] = (int)(entry[e] >> 32);
      sum += w[e];
    }
    if (threadIdx.x == 0) wk.cuts[row] = Cut{0, 0, 1, 0};
    return;
  }
  // many: where the prefix ends
  Cut cut{0, 0, 0, 0};
  unsigned long long total = sh.weights[BINS - 1], upto;
  const unsigned long long upto_last = last ? sh.weights[last - 1] : 0;
  const unsigned long long mine_w = sh.weights[threadIdx.x];  // (end_in may use the bins for its own)
  const uint32_t mine_c = sh.counts[threadIdx.x];
  if (by_count) {
    cut = r.end_in(last, false, (uint32_t)set.k - (last ? sh.counts[last - 1] : 0), upto_last, 0.0, upto);
    total = upto_last + upto;
    sh.weights[threadIdx.x] = mine_w;
    sh.counts[threadIdx.x] = mine_c;
    __syncthreads();
  }
  if (by_weight) {
    const double goal = set.p * (double)total;
    const int b = min(last, r.first_bin([&](int i) { return (double)sh.weights[i] >= goal; }));
    cut = r.end_in(b, true, 1, b ? sh.weights[b - 1] : 0, goal, upto);
  }
  if (threadIdx.x == 0) wk.cuts[row] = cut;
}

// The token of a row whose prefix is known: the slice in which the draw falls,
// then the element.
template <int TYPE>
__global__ void __launch_bounds__(THREADS) sample_draw_kernel(SampleArgs a, int slices, int slice) {
  __shared__ unsigned long long red[2 * THREADS / 64];
  __shared__ unsigned long long before_s;
  __shared__ int slice_s;
  const int row = blockIdx.x;
  const Work wk(a.ws, a.rows, slices);
  const Settings set(a, row);
  Cut cut{0, 0, 0, 0};
  if (!set.greedy && (a.top_k || a.top_p)) cut = wk.cuts[row];
  if (cut.done) return;
  if (threadIdx.x == 0) slice_s = 0, before_s = 0;
  const Top top = top_of<THREADS>(wk.parts + (int64_t)row * slices, slices, red);  // (with barriers)
  if (set.greedy || top.most() == NEG_INF) {
    if (threadIdx.x == 0) a.out[row] = top.most() == NEG_INF ? -1 : top.place();
    return;
  }
  const Weigh weigh{(double)top.most(), set.by};
  unsigned long long total;
  const unsigned long long mine = (int)threadIdx.x < slices ? wk.sums[(int64_t)row * slices + threadIdx.x] : 0;
  const unsigned long long upto = block_scan64(mine, total, red);
  const unsigned long long t = target_of(a.u[row], total);
  if (upto - mine <= t && t < upto) slice_s = threadIdx.x, before_s = upto - mine;
  __syncthreads();
  const int begin = slice_s * slice, end = min(begin + slice, a.vocab);
  unsigned long long before = before_s;
  const void* x = static_cast<const char*>(a.logits) + (int64_t)row * a.row_bytes;
  for (int i0 = begin; i0 < end; i0 += PIECE * THREADS) {
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
    unsigned long long at = before + block_scan64(sum, all, red) - sum;
#pragma unroll
    for (int e = 0; e < PIECE; ++e) {
      if (at <= t && t < at + w[e]) a.out[row] = i + e;
      at += w[e];
    }
    before += all;
    if (before > t) break;
  }
}

// Logits of a slice: about 1024 workgroups over all rows, between 2048 and
// 16384 of them each.
int slice_of(int64_t rows, int vocab) {
  const int64_t step = PIECE * SLICE_THREADS, each = rows * vocab / (1024 * step) * step;
  return (int)(each < step ? step : each > 8 * step ? 8 * step : each);
}
int slices_of(int64_t rows, int vocab) {
  const int s = slice_of(rows, vocab);
  return (vocab + s - 1) / s;
}

template <int TYPE>
hipError_t launch(const SampleArgs& a, hipStream_t s) {
  const int slice = slice_of(a.rows, a.vocab), slices = slices_of(a.rows, a.vocab);
  const dim3 grid((unsigned)a.rows * (unsigned)slices), rows((unsigned)a.rows);
  hipLaunchKernelGGL(sample_scan_kernel<TYPE>, grid, dim3(SLICE_THREADS), 0, s, a, slices, slice);
  if (a.top_k || a.top_p) {
    hipLaunchKernelGGL(sample_histogram_kernel<TYPE>, grid, dim3(SLICE_THREADS), 0, s, a, slices, slice);
    hipLaunchKernelGGL(sample_cut_kernel<TYPE>, rows, dim3(THREADS), 0, s, a, slices);
  }
  hipLaunchKernelGGL(sample_sums_kernel<TYPE>, grid, dim3(SLICE_THREADS), 0, s, a, slices, slice);
  hipLaunchKernelGGL(sample_draw_kernel<TYPE>, rows, dim3(THREADS), 0, s, a, slices, slice);
  return hipGetLastError();
}

}  // namespace

bool sample_fits(int rows, int vocab) { return (int64_t)rows * slices_of(rows, vocab) < 1 << 23 && rows < 1 << 21; }
size_t sample_ws_bytes(int rows, int vocab) { return work_bytes(rows, slices_of(rows, vocab)); }

hipError_t launch_sample(const SampleArgs& a, hipStream_t s) {
  return a.type == 0 ? launch<0>(a, s) : a.type == 1 ? launch<1>(a, s) : launch<2>(a, s);
}

}  // namespace qg
