// Attention for many query rows per key head: whole prompts over packed keys
// and drafted trees over a paged cache.
//
// Mathematics as in attn_narrow.hip (query rows r = t * group + g, running
// maximum and sums, powers of two).
//
// Bound: the matrix cores (2 * head_dim multiplications for each of the two
// products a score), with the exponentials close behind; under 256 query rows
// a key head, the arrival of the keys.  A workgroup takes 32 query rows a wave
// (four waves: 128 rows; eight where a tree has more) and walks the keys in
// tiles of 64; a wave owns 32 rows and all keys of the tile.
//
// Measured (fp16, head_dim 128): a causal prompt of 16384 tokens, 64 heads over
// 8 key heads, 4200 us: 1047 TFLOP/s of the visible pairs, against 1130 for a
// dense product of 8192 x 8192 x 8192 in fp16 on the same card.  64-token bf16 trees
// of 16 rows over 4000 tokens, 32 heads over 8: 99 us, 676 TFLOP/s, 2.7 TB/s
// of keys and values.
// - S^T = K Q^T by 32 x 32 x 16 products: K fragments from LDS, the wave's
//   queries in registers.  A lane then holds 16 scores of ONE query row
//   (lane % 32) per 32 keys, so maximum, exponentials and sum are lane-local;
//   one swap joins the two lane halves.
// - O^T = V^T P^T: the lane's scores of 16 keys, rounded, are its B operand as
//   they stand (the product may take the keys in any order if both operands
//   agree: half h of the lanes holds the keys 4 h + {0..3} and 8 + 4 h +
//   {0..3}).  The A operand, 8 keys of one value column, comes from the
//   row-major tile in LDS by transposing reads (4 keys of 16 columns each).
//   The output sums are per lane of one query row too, so rescaling is a
//   multiplication by a lane's own factor.
// - K and V tiles go from global memory straight into LDS (16 bytes a lane, no
//   registers), the next tile's while this one is computed.  A tile's row is
//   stored in 16-byte pieces whose place is xor-ed with a permutation of the
//   row's low bits, so that both the reads of one piece of many rows and the
//   transposing reads of four neighbouring rows spread over the banks.
#include <type_traits>

#include "attn_common.hpp"

namespace qg {
namespace {

constexpr int KB = 64;   // keys of a tile
constexpr int rows_of(int waves) { return 32 * waves; }  // query rows of a workgroup's tile (BM)

__device__ __forceinline__ f16v zero16() {
  f16v z;
#pragma unroll
  for (int i = 0; i < 16; ++i) z[i] = 0.f;
  return z;
}

typedef short s4v __attribute__((ext_vector_type(4)));
typedef __attribute__((address_space(3))) s4v* lds_s4;

// A segment: key tiles [u0, u1) of `units` of one item, and where the result
// goes (slot < 0: the output).
struct Segment {
  Row r;
  int b, h, tile, u0, u1;
  int64_t slot;
};

template <int D, int WAVES>
struct Tiles {
  static constexpr int PC = D / 8;                // 16-byte pieces of a row
  static constexpr int RPL = 64 / PC;             // rows of one wave-wide load
  static constexpr int RW = KB / WAVES;           // rows of a tile that a wave loads
  static constexpr int LOADS = RW / RPL;          // ... for one tile of K or V
  // 256 bytes of LDS are read at a time: one piece each of 16 rows (K), or four
  // pieces of four rows (V).  A row of 64 elements is half of that, so there
  // rows of one parity have to differ.  (Bank conflicts at D = 64, eight prompts
  // of 61 to 1100 tokens behind 2990: 0.1 million cycles; where rows 0 and 2
  // differ in the lowest piece bit only, 9.3 million, and 1% more time.)
  static __device__ __forceinline__ int swz(int row) {
    return D == 128 ? ((row & 3) << 2 | (row >> 2 & 3)) : ((row >> 1 & 1) << 2 | (row >> 2 & 3));
  }
};

// K and V tiles, two buffers each: separate arrays, so that reading one does
// not wait for loads into another
template <int D>
struct __attribute__((aligned(16))) Buffers {
  uint16_t t[KB * D];
};

template <typename E, int D, bool PAGED, int WAVES>
__device__ __forceinline__ void run_segment(const Segment& g, int64_t slots, Buffers<D>& k0, Buffers<D>& k1, Buffers<D>& v0,
                                            Buffers<D>& v1, uint32_t* flag) {
  const AttnArgs a = args_again();
  using T = Tiles<D, WAVES>;
  constexpr int BM = rows_of(WAVES);
  constexpr int QS = D / 16;  // matrix steps along head_dim
  constexpr int DB = D / 32;  // output blocks of 32 columns
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int c32 = lane & 31, half = lane >> 5;
  const Row r = g.r;
  const int rows = r.n * a.group;

  // the wave's query rows, one per lane column
  const int row = g.tile * BM + 32 * wave + c32;
  const bool live = row < rows;
  const int t = row / a.group, gh = row - t * a.group;
  Sight<PAGED> sight;
  sight.init(a, r, live ? t : r.n);
  u4 qf[QS];
  const uint16_t* q =
      a.q + (live ? (int64_t)(r.q0 + t) * a.q_token + (int64_t)(g.h * a.group + gh) * a.q_head : 0);
#pragma unroll
  for (int s = 0; s < QS; ++s) {
    const u4 x = *reinterpret_cast<const u4*>(q + 16 * s + 8 * half);
#pragma unroll
    for (int e = 0; e < 4; ++e) qf[s][e] = live ? x[e] : 0;
  }
  const bool active = g.tile * BM + 32 * wave < rows;  // (wave-uniform)
  // keys that every row of the tile sees, and the keys that any sees
  const int t0 = g.tile * BM / a.group;
  const int t1 = min((g.tile * BM + BM - 1) / a.group, r.n - 1);
  int common, most;
  if constexpr (PAGED) {
    common = a.mask ? r.pos : r.pos + t0 + 1;
    most = a.mask ? r.keys : r.pos + t1 + 1;
  } else {
    common = a.causal ? r.pos + t0 + 1 : r.keys;
    most = a.causal ? r.pos + t1 + 1 : r.keys;
  }
  common = min(common, r.keys);
  most = min(most, r.keys);
  const int u0 = g.u0, u1 = min(g.u1, (most + KB - 1) / KB);

  // Loads of a tile: wave w brings RW rows of it (16 or 8), from one page.  A
  // lane's place in them is a 32-bit offset, the same for every tile but one
  // that reaches past the row's last key, whose missing rows are read from the
  // last key's place.
  const uint16_t* kh = a.k + (int64_t)g.h * a.k_head;
  const uint16_t* vh = a.v + (int64_t)g.h * a.v_head;
  const int top = (r.keys - 1) & ~(T::RW - 1);
  auto tok_of = [&](int u) -> int64_t {  // pool or array token of the wave's first row
    const int kb = min(u * KB + T::RW * wave, top);
    if constexpr (PAGED) {
      return pool_token(a, g.b, kb);
    } else {
      return (int64_t)r.k0 + kb;
    }
  };
  typedef __attribute__((address_space(1))) const void* gp;
  typedef __attribute__((address_space(3))) void* lp;
  auto lane_off = [&](int i, int64_t token, int last) -> uint32_t {  // bytes
    const int in = T::RPL * i + lane / T::PC;  // row in the wave's
    return 2u * ((uint32_t)min(in, last) * (uint32_t)token + 8u * (uint32_t)((lane % T::PC) ^ T::swz(T::RW * wave + in)));
  };
  auto put = [&](const uint16_t* base, uint32_t off, int i, Buffers<D>& buf) {
    __builtin_amdgcn_global_load_lds((gp)(reinterpret_cast<const char*>(base) + off),
                                     (lp)&buf.t[(T::RW * wave + T::RPL * i) * D], 16, 0, 0);
  };
  auto load = [&](const uint16_t* base, int64_t token, int u, Buffers<D>& buf) {
    const int last = (u + 1) * KB <= r.keys ? T::RW - 1 : r.keys - 1 - min(u * KB + T::RW * wave, top);
#pragma unroll
    for (int i = 0; i < T::LOADS; ++i) put(base, lane_off(i, token, last), i, buf);
  };

  // A lane's places in a tile, in bytes.  K fragments: row lane % 32 (+ 32 x),
  // piece 2 s + half, so k_at ^ 32 s; transposing reads of V: row 4 half + i16
  // / 4 (+ 8 y + 16 k4) with i16 = lane % 16, columns 4 (i16 % 4) .. of the 16
  // of the lane's group (+ 32 db), so v_at[y] ^ 64 db.  The compiler is kept
  // from holding each of these in a register of its own.
  uint32_t k_at, v_at[2];
  {
    const int i16 = lane & 15, g2 = lane >> 4 & 1;
    k_at = 2 * D * c32 + 16 * (half ^ T::swz(c32));
#pragma unroll
    for (int y = 0; y < 2; ++y) {
      const int vrow = 8 * y + 4 * half + (i16 >> 2);
      v_at[y] = 2 * D * vrow + 16 * ((2 * g2 + (i16 >> 1 & 1)) ^ T::swz(vrow)) + 8 * (i16 & 1);
    }
  }

  // S^T of a tile
  f16v sc[2];
  auto scores = [&](const Buffers<D>& kt) {
    const char* base = reinterpret_cast<const char*>(kt.t);
    uint32_t at = k_at;
    asm volatile("" : "+v"(at));
#pragma unroll
    for (int s = 0; s < QS; ++s) {
#pragma unroll
      for (int x = 0; x < 2; ++x) {
        const u4 kf = *reinterpret_cast<const u4*>(base + (at ^ (32 * s)) + 2 * D * 32 * x);
        sc[x] = E::mfma32(kf, qf[s], s == 0 ? zero16() : sc[x]);
      }
    }
  };

  f16v o[DB];
#pragma unroll
  for (int i = 0; i < DB; ++i) o[i] = zero16();
  const float scale = a.scale;
  // m: the weights' reference, at most E::SLACK below the largest score; a tile
  // with scores above most_m needs another (far references: every tile)
  float m = NEG_INF, l = 0.f, most_m = NEG_INF;

  // the tile's scores into weights (P^T, 16 keys a piece); with `some` there
  // may be unseen keys among them, at -inf (whose product with a scale of 0 is
  // not)
  u4 pf[4];
  auto weigh = [&](auto some) {
    float mx = sc[0][0];
#pragma unroll
    for (int x = 0; x < 2; ++x)
#pragma unroll
      for (int i = 0; i < 16; ++i) mx = fmaxf(mx, sc[x][i]);
    mx = half_max(mx);
    mx = mx == NEG_INF ? NEG_INF : mx * scale;
    float by = scale, ref = m;
    if (__any(mx > most_m)) {
      const float mn = fmaxf(m, mx), w = mn == NEG_INF ? 1.f : exp2_(m - mn);
      m = ref = mn;
      most_m = far(mn) ? NEG_INF : mn + E::SLACK;
      l *= w;
#pragma unroll
      for (int i = 0; i < DB; ++i) o[i] *= w;
      if (__any(far(m))) {
#pragma unroll
        for (int x = 0; x < 2; ++x)
#pragma unroll
          for (int i = 0; i < 16; ++i) sc[x][i] = far_score(sc[x][i], scale, m == NEG_INF ? 0.f : m);
        by = 1.f, ref = 0.f;
      }
    }
    const float base = ref == NEG_INF ? 0.f : ref - E::LIFT;
#pragma unroll
    for (int k4 = 0; k4 < 4; ++k4) {
      const int x = k4 >> 1, e = 8 * (k4 & 1);
      float p[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        p[i] = exp2_(fmaf(sc[x][e + i], by, -base));
        if constexpr (decltype(some)::value) p[i] = sc[x][e + i] == NEG_INF ? 0.f : p[i];
        l += p[i];
      }
      pf[k4] = u4{E::pack(p[0], p[1]), E::pack(p[2], p[3]), E::pack(p[4], p[5]), E::pack(p[6], p[7])};
    }
  };

  // O^T += V^T P^T
  auto gather = [&](const Buffers<D>& vt) {
    const char* vb = reinterpret_cast<const char*>(vt.t);
    uint32_t at[2] = {v_at[0], v_at[1]};
    asm volatile("" : "+v"(at[0]), "+v"(at[1]));
#pragma unroll
    for (int k4 = 0; k4 < 4; ++k4)
#pragma unroll
      for (int db = 0; db < DB; ++db) {
        s4v v[2];
#pragma unroll
        for (int y = 0; y < 2; ++y)
          v[y] = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s4)(vb + (at[y] ^ (64 * db)) + 2 * D * 16 * k4));
        const u2 lo = __builtin_bit_cast(u2, v[0]), hi = __builtin_bit_cast(u2, v[1]);
        o[db] = E::mfma32(u4{lo[0], lo[1], hi[0], hi[1]}, pf[k4], o[db]);
      }
  };

  // A weight of 0 does not cancel a value that is infinite or NaN: in a tile
  // with unseen keys, find the keys that have one and clear it in LDS; the
  // whole workgroup, returns the keys.  Thread: WAVES to a key's row.
  auto odd_keys = [&](Buffers<D>& vt) -> uint64_t {
    if (threadIdx.x < 2) flag[threadIdx.x] = 0;
    __syncthreads();
    const int key = threadIdx.x / WAVES;
    u4* p = reinterpret_cast<u4*>(&vt.t[key * D + threadIdx.x % WAVES * (D / WAVES)]);
    uint32_t f = 0;
#pragma unroll
    for (int i = 0; i < D / WAVES / 8; ++i) {
      u4 w = p[i];
      uint32_t any = 0;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const uint32_t x = nonfinite<E>(w[j]);
        any |= x;
        w[j] &= ~((x - (x >> 15)) | x);
      }
      p[i] = w;
      f |= any;
    }
    if (f) atomicOr(&flag[key >> 5], 1u << (key & 31));
    __syncthreads();
    return (uint64_t)__builtin_amdgcn_readfirstlane(flag[1]) << 32 | __builtin_amdgcn_readfirstlane(flag[0]);
  };
  // ... and add them for the rows that see them
  auto add_odd = [&](uint64_t odd, int kb) {
    const AttnArgs a = args_again();
    const uint16_t* vh = a.v + (int64_t)g.h * a.v_head;
    const uint64_t mine = sight.window(a, r, kb);
    for (; odd; odd &= odd - 1) {
      const int key = __builtin_ctzll(odd), at = min(kb + key, r.keys - 1);
      int64_t tok;
      if constexpr (PAGED) {
        tok = pool_token(a, g.b, at);
      } else {
        tok = (int64_t)r.k0 + at;
      }
      const uint16_t* v = vh + tok * a.v_token;
      const uint32_t sees = mine >> key & 1 ? 0x8000u : 0u;
#pragma unroll
      for (int db = 0; db < DB; ++db)
#pragma unroll
        for (int i = 0; i < 16; ++i) {
          const uint16_t y = v[32 * db + 8 * (i / 4) + 4 * half + i % 4];
          o[db][i] += nonfinite<E>(y) & sees ? E::value(y) : 0.f;
        }
    }
  };

  // Order of a gather with scores behind it: a fragment is read AHEAD products
  // before its use.  (Left to itself the compiler reads many of them just before
  // it, into one set of registers, and the wait stands open: 16384-token prompt
  // 4185 -> 4160 us.)
  auto read_ahead = [&]() {
    constexpr int AHEAD = 3, READ = 0x100, MFMA = 0x008;
    __builtin_amdgcn_sched_group_barrier(READ, 2 * AHEAD, 0);
#pragma unroll
    for (int i = 0; i < 4 * DB - AHEAD; ++i) {
      __builtin_amdgcn_sched_group_barrier(MFMA, 1, 0);
      __builtin_amdgcn_sched_group_barrier(READ, 2, 0);
    }
#pragma unroll
    for (int i = 0; i < 2 * QS; ++i) {
      __builtin_amdgcn_sched_group_barrier(MFMA, 1, 0);
      __builtin_amdgcn_sched_group_barrier(READ, 1, 0);
    }
    __builtin_amdgcn_sched_group_barrier(MFMA, AHEAD, 0);
  };

  // Pipeline.  Step u: the weights of tile u, whose scores the step before
  // left (vector units), then its output sums and the scores of tile u + 1
  // (matrix cores); the two waves of a SIMD take turns at these.  K of tile
  // u + 1 and V of tile u were asked for one step ago; the barrier after the
  // wait also says that every wave is past step u - 1, so K of tile u + 2 may
  // go where tile u's was and V of tile u + 1 where tile u - 1's was.
  auto arrived = [&]() {
    __builtin_amdgcn_s_waitcnt(0x0F70);  // vmcnt 0
    lds_barrier();
  };
  // any step
  auto step = [&](int u, Buffers<D>& k_now, Buffers<D>& k_next, Buffers<D>& v_now, Buffers<D>& v_next) {
    const AttnArgs a = args_again();
    const uint16_t* kh = a.k + (int64_t)g.h * a.k_head;
    const uint16_t* vh = a.v + (int64_t)g.h * a.v_head;
    arrived();
    if (u + 2 < u1) load(kh + tok_of(u + 2) * a.k_token, a.k_token, u + 2, k_now);
    if (u + 1 < u1) load(vh + tok_of(u + 1) * a.v_token, a.v_token, u + 1, v_next);
    const int kb = u * KB;
    const bool masked = kb + KB > common;
    uint64_t odd = 0;
    if (masked) odd = odd_keys(v_now);
    if (active) {
      if (zero_scale(scale)) sc[0] -= sc[0], sc[1] -= sc[1];
      if (masked) {
        const AttnArgs a = args_again();
        const uint64_t seen = sight.window(a, r, kb) >> (4 * half);
#pragma unroll
        for (int x = 0; x < 2; ++x)
#pragma unroll
          for (int i = 0; i < 16; ++i) sc[x][i] = seen >> (32 * x + 8 * (i / 4) + i % 4) & 1 ? sc[x][i] : NEG_INF;
      }
      weigh(std::true_type{});
      gather(v_now);
      if (odd) add_odd(odd, kb);
      if (u + 1 < u1) scores(k_next);
    }
  };

  if (u0 < u1) {
    const int64_t tok0 = tok_of(u0);
    load(kh + tok0 * a.k_token, a.k_token, u0, k0);
    if (u0 + 1 < u1) load(kh + tok_of(u0 + 1) * a.k_token, a.k_token, u0 + 1, k1);
    load(vh + tok0 * a.v_token, a.v_token, u0, v0);
    arrived();
    if (active) scores(k0);
    // steps whose tile every row sees in full, two at a time (the waves without
    // rows compute along, on zeros).  Their loads are of whole tiles: in a page
    // the places behind the last key are there too, packed keys need all 64.
    // (The last ones bring tiles, and compute scores, that nothing uses.)
    int uf = min(common / KB, u1);
    if constexpr (!PAGED) uf = min(uf, r.keys / KB - 2);
    uf = u0 + ((uf - u0) & ~1);
    int u = u0;
    if (u < uf) {
      uint32_t ko[T::LOADS], vo[T::LOADS];
#pragma unroll
      for (int i = 0; i < T::LOADS; ++i) {
        ko[i] = lane_off(i, a.k_token, T::RW - 1);
        vo[i] = lane_off(i, a.v_token, T::RW - 1);
      }
      // (the tokens of the next loads are looked up a step ahead)
      int64_t tok1 = tok_of(u + 1), tok2 = tok_of(u + 2);
      auto fast = [&](Buffers<D>& k_now, Buffers<D>& k_next, Buffers<D>& v_now, Buffers<D>& v_next) {
        arrived();
        const uint16_t* kp = kh + tok2 * a.k_token;
        const uint16_t* vp = vh + tok1 * a.v_token;
#pragma unroll
        for (int i = 0; i < T::LOADS; ++i) {
          asm volatile("" : "+v"(ko[i]), "+v"(vo[i]));  // (kept as 32-bit offsets of a scalar base)
          put(kp, ko[i], i, k_now);
        }
#pragma unroll
        for (int i = 0; i < T::LOADS; ++i) put(vp, vo[i], i, v_next);
        tok1 = tok2;
        tok2 = tok_of(u + 3);
        ++u;
        weigh(std::false_type{});
        gather(v_now);
        scores(k_next);
        read_ahead();
      };
      while (u < uf) {
        fast(k0, k1, v0, v1);
        fast(k1, k0, v1, v0);
      }
    }
    for (; u < u1; u += 2) {
      step(u, k0, k1, v0, v1);
      if (u + 1 < u1) step(u + 1, k1, k0, v1, v0);
    }
    arrived();  // the buffers are free for the next segment
  }

  l = half_sum(l);
  if (!live) return;
  const AttnArgs e = args_again();
  const int t_ = row / e.group, g_ = row - t_ * e.group;
  if (g.slot < 0) {
      const float inv = l == 0.f ? 0.f : 1.f / l;
      uint16_t* out = e.o + (int64_t)(r.q0 + t_) * e.o_token + (int64_t)(g.h * e.group + g_) * e.o_head;
#pragma unroll
      for (int db = 0; db < DB; ++db)
#pragma unroll
        for (int i = 0; i < 4; ++i)
          *reinterpret_cast<u2*>(out + 32 * db + 8 * i + 4 * half) =
              u2{E::pack(o[db][4 * i] * inv, o[db][4 * i + 1] * inv),
                 E::pack(o[db][4 * i + 2] * inv, o[db][4 * i + 3] * inv)};
  } else {
    const Partials<BM, D> parts(e.ws, slots);
    const int pr = 32 * wave + c32;
#pragma unroll
    for (int db = 0; db < DB; ++db)
#pragma unroll
      for (int i = 0; i < 4; ++i)
        *parts.o_at(g.slot, pr, 8 * db + 2 * i + half) =
            f4{o[db][4 * i], o[db][4 * i + 1], o[db][4 * i + 2], o[db][4 * i + 3]};
    if (half == 0) {
      float* ml = parts.ml_at(g.slot, pr);
      ml[0] = m;
      ml[1] = l;
    }
  }
}

// Packed prompts: one item (tile of BM rows and key head) per workgroup, or one
// of `splits` parts of its keys.  The tiles of sequence b have the numbers from
// rows_before(b) / BM + b on, which is at least as many as it needs and can be
// looked up without a sum over the sequences.
template <int BM>
__device__ __forceinline__ int first_tile(const AttnArgs& a, int b) {
  return (int)((int64_t)a.cu[b] * a.group / BM) + b;
}

// tile number -> sequence and tile in it; false: no such tile
template <int BM>
__device__ __forceinline__ bool find_tile(const AttnArgs& a, int tile, Row& r, int& b, int& in) {
  b = find_row(a.rows, tile, [&](int i) { return first_tile<BM>(a, i); });
  r = row_of<false>(a, b);
  in = tile - first_tile<BM>(a, b);
  return in >= 0 && (int64_t)in * BM < (int64_t)r.n * a.group;
}

// where query row qr (t * group + g) of key head h has its output; NULL past the last
__device__ __forceinline__ uint16_t* output_row(const AttnArgs& a, const Row& r, int h, int qr) {
  const int t = qr / a.group, g = qr - t * a.group;
  return t < r.n ? a.o + (int64_t)(r.q0 + t) * a.o_token + (int64_t)(h * a.group + g) * a.o_head : nullptr;
}

// the part [u0, u1) of a tile's key tiles that split s takes
template <int BM>
__device__ __forceinline__ void split_range(const AttnArgs& a, const Row& r, int in, int splits, int s, int& u0,
                                            int& u1) {
  const int t1 = min((in * BM + BM - 1) / a.group, r.n - 1);
  int most = a.causal ? r.pos + t1 + 1 : r.keys;
  most = max(0, min(most, r.keys));
  const int units = (most + KB - 1) / KB;
  u0 = (int)((int64_t)units * s / splits);
  u1 = (int)((int64_t)units * (s + 1) / splits);
}

template <typename E, int D, int WAVES>
__global__ void __launch_bounds__(64 * WAVES, wide_waves(D, WAVES)) attn_prompt_kernel(AttnArgs a, int tiles, int splits) {
  constexpr int BM = rows_of(WAVES);
  __shared__ Buffers<D> k0, k1, v0, v1;
  __shared__ uint32_t flag[2];
  Segment g;
  // key head fastest: workgroups go to the XCDs round robin, so with 8 key
  // heads each XCD's cache serves one head's keys and values.  Late tiles,
  // which have the most keys under a causal mask, start first.
  const int id = blockIdx.x;
  g.h = id % a.heads_kv;
  const int s = id / a.heads_kv % splits;
  const int tile = tiles - 1 - id / a.heads_kv / splits;
  if (!find_tile<BM>(a, tile, g.r, g.b, g.tile)) return;
  split_range<BM>(a, g.r, g.tile, splits, s, g.u0, g.u1);
  g.slot = splits == 1 ? -1 : ((int64_t)tile * a.heads_kv + g.h) * splits + s;
  run_segment<E, D, false, WAVES>(g, (int64_t)tiles * a.heads_kv * splits, k0, k1, v0, v1, flag);
}

// One workgroup per 32 query rows of a tile and key head: joins their parts.
template <typename E, int D, int WAVES>
__global__ void __launch_bounds__(256) attn_prompt_join_kernel(AttnArgs a, int splits) {
  constexpr int BM = rows_of(WAVES);
  const int tile = blockIdx.x / (BM / 32), h = blockIdx.y;
  Row r;
  int b, in;
  if (!find_tile<BM>(a, tile, r, b, in)) return;
  const Partials<BM, D> parts(a.ws, (int64_t)(gridDim.x / (BM / 32)) * a.heads_kv * splits);
  join_rows<E>(parts, 32 * (blockIdx.x % (BM / 32)), splits, [&](int i) { return ((int64_t)tile * a.heads_kv + h) * splits + i; },
               [&](int row) { return output_row(a, r, h, in * BM + row); });
}

// Trees over the paged cache: the units of all items shared out evenly
// (Walk), so rows of very different lengths keep every workgroup busy.
template <typename E, int D, int WAVES>
__global__ void __launch_bounds__(64 * WAVES, wide_waves(D, WAVES)) attn_tree_kernel(AttnArgs a, int workgroups) {
  constexpr int BM = rows_of(WAVES);
  using U = Walk<BM, KB, true, 1>;
  __shared__ Buffers<D> k0, k1, v0, v1;
  __shared__ uint32_t flag[2];
  // (the rows are looked up again for every segment, of which there are few,
  // so that they occupy no registers during one)
  for (int64_t done = 0;;) {
    U walk;
    walk.init(a, workgroups);
    const int c = share_of(blockIdx.x, walk.shares());
    const int64_t u_begin = c * walk.per, u = u_begin + done;
    const int64_t u_end = u_begin + walk.per < walk.total ? u_begin + walk.per : walk.total;
    if (u >= u_end) break;
    const typename U::Piece p = walk.seek(a, u, u_end);
    Segment g{p.r, p.b, p.h, p.tile, p.k0, p.k1, 0};
    g.slot = g.u0 == 0 && g.u1 == p.of ? -1 : 2 * (int64_t)c + (done != 0);
    done += g.u1 - g.u0;
    run_segment<E, D, true, WAVES>(g, 2 * (int64_t)workgroups, k0, k1, v0, v1, flag);
  }
}

// One workgroup per 32 query rows of a tile and key head: joins the parts of
// an item that lay in several workgroups.
template <typename E, int D, int WAVES>
__global__ void __launch_bounds__(256) attn_tree_join_kernel(AttnArgs a, int workgroups) {
  constexpr int BM = rows_of(WAVES);
  using U = Walk<BM, KB, true, 1>;
  U walk;
  walk.init(a, workgroups);
  const int tile = blockIdx.x / (BM / 32), h = blockIdx.y;
  auto first_at = [&](int q0, int b) { return (int)((int64_t)q0 * a.group / BM) + b; };
  const int b = walk.find(a, tile, [&](const Row& r, int i) { return first_at(r.q0, i); },
                          [&](int i) { return first_at(a.cu[i], i); });
  Row r;
  int64_t first;
  walk.seek_row(a, b, r, first);
  const int in = tile - first_at(r.q0, b);
  if (in < 0 || in >= U::tiles(a, r)) return;
  const typename U::Parts p = walk.parts(first + (int64_t)(h * U::tiles(a, r) + in) * U::units(r), U::units(r));
  if (p.n == 1) return;
  join_rows<E>(Partials<BM, D>(a.ws, 2 * (int64_t)workgroups), 32 * (blockIdx.x % (BM / 32)), p.n,
               [&](int i) { return p.slot(i); }, [&](int row) { return output_row(a, r, h, in * BM + row); });
}

template <typename E, int D, int WAVES>
hipError_t prompt(const AttnArgs& a, hipStream_t s) {
  constexpr int BM = rows_of(WAVES);
  const int tiles = wide_tiles(a.tokens, a.rows, a.group, WAVES);
  const int splits = prompt_splits(a.tokens, a.tokens_k, a.rows, a.heads_kv, a.group, D, WAVES);
  const int64_t grid = (int64_t)tiles * a.heads_kv * splits;
  hipLaunchKernelGGL((attn_prompt_kernel<E, D, WAVES>), dim3((unsigned)grid), dim3(64 * WAVES), 0, s, a, tiles, splits);
  if (splits > 1)
    hipLaunchKernelGGL((attn_prompt_join_kernel<E, D, WAVES>), dim3((unsigned)tiles * (BM / 32), (unsigned)a.heads_kv),
                       dim3(256), 0, s, a, splits);
  return hipGetLastError();
}

template <typename E, int D, int WAVES>
hipError_t tree(const AttnArgs& a, hipStream_t s) {
  constexpr int BM = rows_of(WAVES);
  const int workgroups = wide_workgroups(D, WAVES);
  hipLaunchKernelGGL((attn_tree_kernel<E, D, WAVES>), dim3(workgroups), dim3(64 * WAVES), 0, s, a, workgroups);
  hipLaunchKernelGGL((attn_tree_join_kernel<E, D, WAVES>),
                     dim3((unsigned)wide_tiles(a.tokens, a.rows, a.group, WAVES) * (BM / 32), (unsigned)a.heads_kv),
                     dim3(256), 0, s, a, workgroups);
  return hipGetLastError();
}

template <typename E, int D>
hipError_t launch(const AttnArgs& a, hipStream_t s) {
  if (a.tables) return tree_waves(a.tokens, a.rows, a.group) == 8 ? tree<E, D, 8>(a, s) : tree<E, D, 4>(a, s);
  return prompt<E, D, PROMPT_WAVES>(a, s);
}

}  // namespace

hipError_t launch_attn_wide(const AttnArgs& a, hipStream_t s) {
  if (a.head_dim == 128) return a.bf16 ? launch<BF16, 128>(a, s) : launch<F16, 128>(a, s);
  return a.bf16 ? launch<BF16, 64>(a, s) : launch<F16, 64>(a, s);
}

}  // namespace qg
