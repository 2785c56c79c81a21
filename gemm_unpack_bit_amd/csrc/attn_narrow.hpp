// Attention for few query rows per key head: decode (one token per row) and
// small drafted trees, over paged or packed keys.
//
// Mathematics.  For one key head the query rows are r = t * group + g (token
// t, head g of the group), so grouped heads share one read of the keys and
// values.  Over the keys in steps of 32 a wave keeps, per row, the running
// maximum m, the sum l = sum 2^(x - m) and the output sums O = sum 2^(x - m) v,
// x = score * scale * log2(e); a step with a new maximum scales l and O by
// 2^(m_old - m_new).
//
// Bound: memory.  Each key and value is read once, straight from global
// memory into registers, with no LDS on the way:
// - S^T = K Q^T on the matrix cores (16 x 16 x 32): a lane's A operand is 8
//   consecutive elements of one key, one 16-byte load.
// - O^T = V^T P^T: the matrix product may take its 32 keys in any order if
//   both operands agree, so a lane keeps the scores where S^T left them (the
//   keys 4 q + i and 16 + 4 q + i of lane quarter q) as B operand, and for A
//   needs 8 keys of one output column.  It loads D / 16 columns of its 8 keys
//   (16 lanes read a key's whole row) and pairs the keys of a column by one
//   byte permute per two elements.  The output columns are then
//   D / 16 * m + j for matrix row m of product j: again only an order.
// - row statistics are per lane (row = lane % 16): the maximum crosses the
//   four lane quarters by two swaps, the sum only once at the end.
// The waves of a workgroup take the steps of its key range in turn, each with
// its own m, l, O, joined in LDS at the end.  Few rows leave few tiles, so the
// key axis is split over workgroups (Walk).
//
// Measured (fp16, head_dim 128, pages of 16): one token of 64 heads over 8 key
// heads for 32 rows of 18000 cached tokens, 399 us, 5.9 TB/s (a streaming read
// of memory reaches 7.1); one row of 777 tokens, 32 heads over 8, 7.9 us, most
// of it a launch and three trips to memory one behind the other.
//
// A cache of 8 bits: the same with codes in place of values on their way, which
// become values of the element type (e4m3.hpp) when they are used; a tile of 16
// keys is one block, whose exponents travel with its codes.
#pragma once

#include <type_traits>

#include "attn_common.hpp"
#include "e4m3.hpp"

namespace qg {
namespace {

constexpr int KB = 128;      // keys of a unit: 32 per wave
constexpr int WAVES = 4;

// Partial results in the workspace: [slots][BM] (max, sum); per slot BM * D
// sums in 16-byte pieces, so that a wave's store or load of a piece per lane is
// 1 KB; two words per share for the tickets.
//
// The workgroups that write and read a part sit on different XCDs, whose caches
// do not see each other.  Fences would write back and drop whole caches (a
// decode batch of 144k keys took 177 us instead of 108); instead every access
// to a part goes past them (device scope, like the atomics on the tickets).
// Joining here rather than in a second kernel saves that kernel's launch and
// its look at all rows (8 us of 116 on the same batch).
constexpr int CPOL_DEVICE = 16;
template <int BM, int D>
struct Parts {
  rsrc_t r;
  uint32_t sums;  // byte offset of the sums
  unsigned long long* tickets;
  __device__ __forceinline__ Parts(float* ws, int64_t slots)
      : r(make_rsrc(ws, (uint32_t)(slots * BM * (D + 2) * 4))),
        sums((uint32_t)(slots * BM * 8)),
        tickets(reinterpret_cast<unsigned long long*>(ws + slots * BM * (D + 2))) {}
  __device__ __forceinline__ void put_ml(int64_t slot, int row, float m, float l) const {
    __builtin_amdgcn_raw_buffer_store_b64(__builtin_bit_cast(u2, f2v{m, l}), r, (uint32_t)((slot * BM + row) * 8), 0,
                                          CPOL_DEVICE);
  }
  __device__ __forceinline__ f2v ml(int64_t slot, int row) const {
    return __builtin_bit_cast(
        f2v, __builtin_amdgcn_raw_buffer_load_b64(r, (uint32_t)((slot * BM + row) * 8), 0, CPOL_DEVICE));
  }
  // piece x of thread t (of 16) of a row: four columns
  __device__ __forceinline__ uint32_t at(int64_t slot, int row, int x, int t) const {
    return sums + (uint32_t)(slot * (BM * D / 4) + ((row >> 4) * (D / 64) + x) * 256 + (row & 15) * 16 + t) * 16;
  }
  __device__ __forceinline__ void put(int64_t slot, int row, int x, int t, f4 v) const {
    __builtin_amdgcn_raw_buffer_store_b128(__builtin_bit_cast(u4, v), r, at(slot, row, x, t), 0, CPOL_DEVICE);
  }
  __device__ __forceinline__ f4 get(int64_t slot, int row, int x, int t) const {
    return __builtin_bit_cast(f4, bload16<CPOL_DEVICE>(r, at(slot, row, x, t)));
  }
};

// Whether this workgroup's part of an item is the last of `parts` to be
// written; the one for which it is joins them all, in key order, so the result
// does not depend on which one that is, and no workgroup waits for another.
// Called by the whole workgroup after its part's stores.
//
// The first word of a ticket is CLEAN plus the number of parts written so far,
// and CLEAN again after the last.  The workspace comes without initial contents:
// where the word is nothing of the kind (a workspace's first call), all parts of
// the item see that, and count in the second word instead, under the call's
// nonce (48 bits, another one for every call); what does not carry the nonce
// there counts as 0.  (A stray value is taken for a count once in 2^48.)
constexpr unsigned long long CLEAN = 0x9C3B5E2D71A60000ull;
__device__ __forceinline__ bool last_part(unsigned long long* ticket, uint64_t nonce, int parts, uint32_t* shared) {
  __builtin_amdgcn_s_waitcnt(0x0F70);  // vmcnt 0: this wave's stores have reached the device's memory
  __syncthreads();                     // ... and every wave's
  if (threadIdx.x == 0) {
    bool last;
    unsigned long long old = __hip_atomic_fetch_add(ticket, 1ull, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    if (old - CLEAN < 0xFFFF) {
      last = (int)(old - CLEAN) == parts - 1;
    } else {
      unsigned long long now;
      old = __hip_atomic_load(ticket + 1, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
      do {
        const int n = old >> 16 == nonce ? (int)(old & 0xFFFF) + 1 : 1;
        last = n == parts;
        now = nonce << 16 | (unsigned)n;
      } while (!__hip_atomic_compare_exchange_strong(ticket + 1, &old, now, __ATOMIC_RELAXED, __ATOMIC_RELAXED,
                                                     __HIP_MEMORY_SCOPE_AGENT));
      if (last) __hip_atomic_store(ticket + 1, 0ull, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    }
    if (last) __hip_atomic_store(ticket, CLEAN, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    *shared = last;
  }
  __syncthreads();
  return __builtin_amdgcn_readfirstlane(*shared) != 0;
}

// RT: 16-row tiles of query rows held by a wave (BM = 16 RT rows)
// Q8: paged keys of a cache of 8 bits
template <typename E, int D, int RT, bool PAGED, bool Q8>
__global__ void __launch_bounds__(64 * WAVES, 2) attn_narrow_kernel(AttnArgs a, int workgroups) {
  static_assert(PAGED || !Q8, "packed keys have 16 bits");
  constexpr int BM = 16 * RT;
  constexpr int KS = D / 32;  // matrix steps along head_dim
  constexpr int DL = D / 16;  // output columns of a lane
  constexpr int DW = DL / 2;  // ... in 32-bit words
  constexpr int PITCH = D + 4;
  typedef uint32_t vw __attribute__((ext_vector_type(DW)));
  using U = Walk<BM, KB, PAGED, 16>;
  __shared__ __attribute__((aligned(16))) float o_s[WAVES][BM][PITCH];
  __shared__ float m_s[WAVES][BM], l_s[WAVES][BM];
  __shared__ uint32_t last_s;

  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int n16 = lane & 15, quarter = lane >> 4;
  U walk;
  walk.init(a, workgroups);
  const int c = share_of(blockIdx.x, walk.shares());
  int64_t u = c * walk.per;
  const int64_t u_end = u + walk.per < walk.total ? u + walk.per : walk.total;
  const int64_t u_begin = u;
  const Parts<BM, D> parts(a.ws, 2 * (int64_t)workgroups);

  while (u < u_end) {
    const typename U::Piece piece = walk.seek(a, u, u_end);
    const Row r = piece.r;
    const int b = piece.b, h = piece.h, tile = piece.tile, ku = piece.k0, ku_end = piece.k1;
    const int rows = r.n * a.group;

    // the wave's query rows: lane column n16 of each 16-row tile
    u4 qf[RT][KS];
    Sight<PAGED> sight[RT];
#pragma unroll
    for (int i = 0; i < RT; ++i) {
      const int row = tile * BM + 16 * i + n16;
      const int t = row / a.group, g = row - t * a.group;
      const bool live = row < rows;
      sight[i].init(a, r, live ? t : r.n);
      const uint16_t* q = a.q + (live ? (int64_t)(r.q0 + t) * a.q_token + (int64_t)(h * a.group + g) * a.q_head : 0);
#pragma unroll
      for (int s = 0; s < KS; ++s) {
        // (a lane's 16 codes of a key serve two products)
        const u4 x = *reinterpret_cast<const u4*>(q + (Q8 ? 64 * (s / 2) + 16 * quarter + 8 * (s & 1) : 32 * s + 8 * quarter));
#pragma unroll
        for (int e = 0; e < 4; ++e) qf[i][s][e] = live ? x[e] : 0;
      }
    }
    // keys that every row of the tile sees
    const int first_t = tile * BM / a.group;
    int common;
    if constexpr (PAGED) common = a.mask ? r.pos : r.pos + first_t + 1;
    else common = a.causal ? r.pos + first_t + 1 : r.keys;
    common = common < r.keys ? common : r.keys;

    f4 o[RT][DL];
    float m[RT], l[RT], most[RT];  // a step with scores above most needs another m (far ones: every step)
#pragma unroll
    for (int i = 0; i < RT; ++i) {
      m[i] = most[i] = NEG_INF;
      l[i] = 0.f;
#pragma unroll
      for (int j = 0; j < DL; ++j) o[i][j] = f4{0.f, 0.f, 0.f, 0.f};
    }

    // Loads of a step: two tiles of 16 keys, each 16 rows of one page, by a
    // scalar base and a lane's 32-bit offset.  A tile past the row's last key
    // falls back on the last tile that has any, and a key past the last is read
    // from the last one's place.
    constexpr int W = Q8 ? 1 : 2;  // bytes of a key's element
    const char* kh = reinterpret_cast<const char*>(a.k) + (int64_t)h * a.k_head * W;
    const char* vh = reinterpret_cast<const char*>(a.v) + (int64_t)h * a.v_head * W;
    const uint32_t k_row = (uint32_t)W * (uint32_t)a.k_token, v_row = (uint32_t)W * (uint32_t)a.v_token;  // bytes
    const int top = (r.keys - 1) & ~15;
    auto token_at = [&](int kb) -> int64_t {
      kb = kb < top ? kb : top;
      if constexpr (PAGED) return pool_token(a, b, kb);
      else return (int64_t)r.k0 + kb;
    };
    u4 kf[2][Q8 ? KS / 2 : KS];
    vw vf[8];
    // codes of the next step's values, and the exponents of both of its tiles
    typedef uint32_t cw __attribute__((ext_vector_type(Q8 ? (DW / 2 > 1 ? 2 : 1) : 1)));
    cw vc[Q8 ? 8 : 1];
    uint32_t ke[2], ve[2];
    // (a lane's offsets in a tile with all its keys)
    const uint32_t k_off = (uint32_t)n16 * k_row + 16u * quarter, v_off = 4u * quarter * v_row + (uint32_t)W * DL * n16;
    auto last_of = [&](int k0) { return r.keys - 1 - (k0 < top ? k0 : top); };
    auto load_k = [&](int kb, const int64_t (&tok)[2]) {
#pragma unroll
      for (int x = 0; x < 2; ++x) {
        const int k0 = kb + 16 * x;
        const char* p = kh + tok[x] * a.k_token * W;
        uint32_t off = k_off;
        if (k0 + 16 > r.keys) off = (uint32_t)min(n16, last_of(k0)) * k_row + 16u * quarter;
#pragma unroll
        for (int s = 0; s < (Q8 ? KS / 2 : KS); ++s) kf[x][s] = *reinterpret_cast<const u4*>(p + off + 64 * s);
        if constexpr (Q8) ke[x] = a.k_exps[(tok[x] / KV_BLOCK) * a.heads_kv + h];
      }
    };
    auto load_v = [&](int kb, const int64_t (&tok)[2]) {
#pragma unroll
      for (int x = 0; x < 2; ++x) {
        const int k0 = kb + 16 * x;
        const char* p = vh + tok[x] * a.v_token * W;
        uint32_t off[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) off[i] = v_off + i * v_row;
        if (k0 + 16 > r.keys)
#pragma unroll
          for (int i = 0; i < 4; ++i) off[i] = (uint32_t)min(4 * quarter + i, last_of(k0)) * v_row + (uint32_t)W * DL * n16;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          if constexpr (Q8) vc[4 * x + i] = __builtin_nontemporal_load(reinterpret_cast<const cw*>(p + off[i]));
          else vf[4 * x + i] = __builtin_nontemporal_load(reinterpret_cast<const vw*>(p + off[i]));
        }
        if constexpr (Q8) ve[x] = a.v_exps[(tok[x] / KV_BLOCK) * a.heads_kv + h];
      }
    };
    // K fragment of product s of a tile; the values of the step's keys
    auto k_frag = [&](int x, int s) -> u4 {
      if constexpr (Q8) return decode8<E>(kf[x][s / 2][2 * (s & 1)], kf[x][s / 2][2 * (s & 1) + 1], exp_scale(ke[x]));
      else return kf[x][s];
    };
    auto values = [&]() {
      if constexpr (Q8) {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const float by = exp_scale(ve[i / 4]);
#pragma unroll
          for (int w = 0; w < DW; ++w) vf[i][w] = w & 1 ? decode2<E, true>(vc[i][w / 2], by) : decode2<E, false>(vc[i][w / 2], by);
        }
      }
    };

    // Pipeline: the next step's keys are asked for as soon as this one's are
    // used up, and its values likewise, into the same registers: at any time
    // one or the other is on its way.  (The scheduling barriers keep the loads
    // where they stand.)
    const int k_end = ku_end * KB < r.keys ? ku_end * KB : r.keys;
    int kb = ku * KB + 32 * wave;
    // The values taken out of masked steps, added up in the wave's part of o_s
    // (a key at a time for the rows that see it, a column per lane; no
    // rescaling: they are infinite or NaN)
    bool odd_any = false;
    auto add_odd = [&](uint64_t odd, int kb) {
      const AttnArgs e = args_again();
      float* sums = &o_s[wave][0][0];
      if (!odd_any)
        for (int x = lane; x < BM * PITCH; x += 64) sums[x] = 0.f;
      odd_any = true;
      for (; odd; odd &= odd - 1) {
        const int key = __builtin_ctzll(odd), at = min(kb + key, r.keys - 1);
        const int64_t tok = token_at(at & ~15) + (at & 15), v0 = (int64_t)h * e.v_head + tok * e.v_token;
        auto value = [&](int d) -> uint16_t {
          if constexpr (Q8)
            return (uint16_t)decode2<E, false>(reinterpret_cast<const uint8_t*>(e.v)[v0 + d],
                                               exp_scale(e.v_exps[tok / KV_BLOCK * e.heads_kv + h]));
          else return e.v[v0 + d];
        };
#pragma unroll
        for (int i = 0; i < RT; ++i) {
          uint32_t see = (uint32_t)__ballot(sight[i].window(e, r, kb) >> key & 1) & 0xFFFF;
          for (; see; see &= see - 1)
#pragma unroll
            for (int d0 = 0; d0 < D; d0 += 64) {
              const uint16_t y = value(d0 + lane);
              sums[(16 * i + __builtin_ctz(see)) * PITCH + d0 + lane] += nonfinite<E>(y) & 0x8000u ? E::value(y) : 0.f;
            }
        }
      }
    };
    int64_t tok1[2];  // the next step's
    auto step = [&](auto more) {
      f4 sc[RT][2];
#pragma unroll
      for (int i = 0; i < RT; ++i)
#pragma unroll
        for (int x = 0; x < 2; ++x) {
          sc[i][x] = f4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
          for (int s = 0; s < KS; ++s) sc[i][x] = E::mfma16(k_frag(x, s), qf[i][s], sc[i][x]);
        }
      __builtin_amdgcn_sched_barrier(0);
      if constexpr (decltype(more)::value) load_k(kb + 32 * WAVES, tok1);
      __builtin_amdgcn_sched_barrier(0);

      if (zero_scale(a.scale))
#pragma unroll
        for (int i = 0; i < RT; ++i) sc[i][0] -= sc[i][0], sc[i][1] -= sc[i][1];
      values();
      if constexpr (Q8 && decltype(more)::value) {
        __builtin_amdgcn_sched_barrier(0);
        load_v(kb + 32 * WAVES, tok1);
        __builtin_amdgcn_sched_barrier(0);
      }
      const bool masked = kb + 32 > common;
      uint64_t odd = 0;  // keys of the step with a value that is not finite (masked steps)
      if (masked) {
#pragma unroll
        for (int i = 0; i < RT; ++i) {
          const uint64_t seen = sight[i].window(a, r, kb) >> (4 * quarter);
#pragma unroll
          for (int x = 0; x < 2; ++x)
#pragma unroll
            for (int e = 0; e < 4; ++e) sc[i][x][e] = seen >> (16 * x + e) & 1 ? sc[i][x][e] : NEG_INF;
        }
        // a weight of 0 does not cancel a value that is infinite or NaN:
        // take those out and add them for the rows that see them
        uint32_t bad = 0;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          uint32_t f = 0;
#pragma unroll
          for (int w = 0; w < DW; ++w) {
            const uint32_t x = nonfinite<E>(vf[i][w]);
            f |= x;
            // halves to clear: 0x8000 of a half becomes 0xFFFF
            vf[i][w] &= ~((x - (x >> 15)) | x);
          }
          bad |= f ? 1u << i : 0u;
        }
        if (__any(bad))
#pragma unroll
          for (int i = 0; i < 8; ++i)
#pragma unroll
            for (int qd = 0; qd < 4; ++qd)
              if (__ballot(bad >> i & 1) >> (16 * qd) & 0xFFFF) odd |= 1ull << ((i < 4 ? i : 12 + i) + 4 * qd);
      }

#pragma unroll
      for (int i = 0; i < RT; ++i) {
        f4 s0 = sc[i][0], s1 = sc[i][1];
        float mx = fmaxf(fmaxf(fmaxf(s0[0], s0[1]), fmaxf(s0[2], s0[3])), fmaxf(fmaxf(s1[0], s1[1]), fmaxf(s1[2], s1[3])));
        mx = quarter_max(mx);
        mx = mx == NEG_INF ? NEG_INF : mx * a.scale;
        float by = a.scale, ref = m[i];
        if (__any(mx > most[i])) {
          const float mn = fmaxf(m[i], mx), w = mn == NEG_INF ? 1.f : exp2_(m[i] - mn);
          m[i] = ref = mn;
          most[i] = far(mn) ? NEG_INF : mn + E::SLACK;
          l[i] *= w;
#pragma unroll
          for (int j = 0; j < DL; ++j) o[i][j] *= w;
          if (__any(far(mn))) {
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              s0[e] = far_score(s0[e], a.scale, mn == NEG_INF ? 0.f : mn);
              s1[e] = far_score(s1[e], a.scale, mn == NEG_INF ? 0.f : mn);
            }
            by = 1.f, ref = 0.f;
          }
        }
        const float base = ref == NEG_INF ? 0.f : ref - E::LIFT;
        float p[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          const float x = e < 4 ? s0[e & 3] : s1[e & 3];
          p[e] = x == NEG_INF ? 0.f : exp2_(fmaf(x, by, -base));
          l[i] += p[e];
        }
        const u4 pf = u4{E::pack(p[0], p[1]), E::pack(p[2], p[3]), E::pack(p[4], p[5]), E::pack(p[6], p[7])};
#pragma unroll
        for (int j = 0; j < DL; ++j) {
          u4 va;
#pragma unroll
          for (int w = 0; w < 4; ++w)
            va[w] = __builtin_amdgcn_perm(vf[2 * w + 1][j / 2], vf[2 * w][j / 2], j & 1 ? 0x07060302u : 0x05040100u);
          o[i][j] = E::mfma16(va, pf, o[i][j]);
        }
      }
      if (odd) add_odd(odd, kb);
      __builtin_amdgcn_sched_barrier(0);
      if constexpr (!Q8 && decltype(more)::value) load_v(kb + 32 * WAVES, tok1);
      __builtin_amdgcn_sched_barrier(0);
    };
    if (kb < k_end) {
      const int64_t tok0[2] = {token_at(kb), token_at(kb + 16)};
      load_k(kb, tok0);
      load_v(kb, tok0);
#pragma unroll
      for (int x = 0; x < 2; ++x) tok1[x] = token_at(kb + 32 * WAVES + 16 * x);
      for (; kb + 32 * WAVES < k_end; kb += 32 * WAVES) {
        // (looked up a step ahead of the loads)
        const int64_t tok2[2] = {token_at(kb + 64 * WAVES), token_at(kb + 64 * WAVES + 16)};
        step(std::true_type{});
        tok1[0] = tok2[0], tok1[1] = tok2[1];
      }
      step(std::false_type{});
    }

    // join the waves
#pragma unroll
    for (int i = 0; i < RT; ++i) {
      const int row = 16 * i + n16;
#pragma unroll
      for (int e = 0; e < 4; ++e)
#pragma unroll
        for (int j = 0; j < DL; j += 4) {
          f4* at = reinterpret_cast<f4*>(&o_s[wave][row][DL * (4 * quarter + e) + j]);
          f4 x = f4{o[i][j][e], o[i][j + 1][e], o[i][j + 2][e], o[i][j + 3][e]};
          if (odd_any) x += *at;
          *at = x;
        }
      const float sum = quarter_sum(l[i]);
      if (quarter == 0) m_s[wave][row] = m[i], l_s[wave][row] = sum;
    }
    __syncthreads();
    const bool whole = ku == 0 && ku_end == piece.of;
    const int64_t slot = 2 * (int64_t)c + (u != u_begin);
    constexpr int TPR = 64 * WAVES / 16;  // 16 threads per row, DL columns each
    static_assert(TPR == 16, "a row's columns are DL per thread");
#pragma unroll
    for (int i = 0; i < RT; ++i) {
      const int row = 16 * i + (threadIdx.x >> 4), col = DL * (threadIdx.x & 15);
      float M = NEG_INF;
#pragma unroll
      for (int w = 0; w < WAVES; ++w) M = fmaxf(M, m_s[w][row]);
      const float base = M == NEG_INF ? 0.f : M;
      float sum = 0.f, acc[DL] = {};
#pragma unroll
      for (int w = 0; w < WAVES; ++w) {
        const float f = exp2_(m_s[w][row] - base);
        sum += f * l_s[w][row];
#pragma unroll
        for (int j = 0; j < DL; ++j) acc[j] += f * o_s[w][row][col + j];
      }
      const int qr = tile * BM + row;
      if (whole) {
        if (qr < rows) {
          const int t = qr / a.group, g = qr - t * a.group;
          const float inv = sum == 0.f ? 0.f : 1.f / sum;
          vw y;
#pragma unroll
          for (int j = 0; j < DW; ++j) y[j] = E::pack(acc[2 * j] * inv, acc[2 * j + 1] * inv);
          *reinterpret_cast<vw*>(a.o + (int64_t)(r.q0 + t) * a.o_token + (int64_t)(h * a.group + g) * a.o_head + col) = y;
        }
      } else {
        if (qr < rows) {
#pragma unroll
          for (int j = 0; j < DL; j += 4)
            parts.put(slot, row, j / 4, threadIdx.x & 15, f4{acc[j], acc[j + 1], acc[j + 2], acc[j + 3]});
          if ((threadIdx.x & 15) == 0) parts.put_ml(slot, row, M, sum);
        }
      }
    }
    if (!whole) {
      // (at most one item goes on from a share into the next: the share's number
      // is its ticket's)
      const typename U::Parts p = walk.parts(u - ku, piece.of);
      if (last_part(parts.tickets + 2 * p.c0, a.nonce, p.n, &last_s)) {
        // 16 threads hold a row's columns; with few rows, several such rows of
        // threads take every PL-th part of one and are added up in LDS
        const int live = min(BM, rows - tile * BM);
        const int lg = live <= 1 ? 0 : live <= 2 ? 1 : live <= 4 ? 2 : live <= 8 ? 3 : 4;  // log2 of rows at a time
        const int RP = 1 << lg, PL = 16 >> lg;
        const int rl = threadIdx.x >> 4, pl = rl >> lg, col = DL * (threadIdx.x & 15);
        typedef float fl __attribute__((ext_vector_type(DL)));
        constexpr int AT_ONCE = 4;  // parts on their way
        for (int row0 = 0; row0 < live; row0 += RP) {
          const int row = row0 + (rl & (RP - 1));
          float mj = NEG_INF, lj = 0.f;
          fl acc;
#pragma unroll
          for (int j = 0; j < DL; ++j) acc[j] = 0.f;
          if (row < live)
            for (int i = pl; i < p.n; i += AT_ONCE * PL) {
              float mi[AT_ONCE], li[AT_ONCE];
              fl oi[AT_ONCE];
#pragma unroll
              for (int x = 0; x < AT_ONCE; ++x) {
                const int64_t at = p.slot(i + x * PL < p.n ? i + x * PL : i);
                const f2v ml = parts.ml(at, row);
                mi[x] = i + x * PL < p.n ? ml[0] : NEG_INF;
                li[x] = i + x * PL < p.n ? ml[1] : 0.f;
#pragma unroll
                for (int j = 0; j < DL; j += 4) {
                  const f4 y = parts.get(at, row, j / 4, threadIdx.x & 15);
                  oi[x][j] = y[0], oi[x][j + 1] = y[1], oi[x][j + 2] = y[2], oi[x][j + 3] = y[3];
                }
              }
              float mn = mj;
#pragma unroll
              for (int x = 0; x < AT_ONCE; ++x) mn = fmaxf(mn, mi[x]);
              const float base = mn == NEG_INF ? 0.f : mn, w = exp2_(mj - base);
              lj *= w;
              acc *= w;
#pragma unroll
              for (int x = 0; x < AT_ONCE; ++x) {
                const float wx = exp2_(mi[x] - base);
                lj += wx * li[x];
#pragma unroll
                for (int j = 0; j < DL; ++j) acc[j] += i + x * PL < p.n ? wx * oi[x][j] : 0.f;
              }
              mj = mn;
            }
          float* sums = &o_s[0][0][0];
          float* ms = &m_s[0][0];  // 16 of each: WAVES * BM are at least 64
          float* ls = &l_s[0][0];
          *reinterpret_cast<fl*>(sums + rl * D + col) = acc;
          if (col == 0) ms[rl] = mj, ls[rl] = lj;
          __syncthreads();
          if (pl == 0 && row < live) {
            float M = NEG_INF;
            for (int x = 0; x < PL; ++x) M = fmaxf(M, ms[rl + x * RP]);
            const float base = M == NEG_INF ? 0.f : M;
            float sum = 0.f;
#pragma unroll
            for (int j = 0; j < DL; ++j) acc[j] = 0.f;
            for (int x = 0; x < PL; ++x) {
              const float w = exp2_(ms[rl + x * RP] - base);
              sum += w * ls[rl + x * RP];
              acc += w * *reinterpret_cast<const fl*>(sums + (rl + x * RP) * D + col);
            }
            const int qr = tile * BM + row, t = qr / a.group, g = qr - t * a.group;
            const float inv = sum == 0.f ? 0.f : 1.f / sum;
            vw y;
#pragma unroll
            for (int j = 0; j < DW; ++j) y[j] = E::pack(acc[2 * j] * inv, acc[2 * j + 1] * inv);
            *reinterpret_cast<vw*>(a.o + (int64_t)(r.q0 + t) * a.o_token + (int64_t)(h * a.group + g) * a.o_head + col) = y;
          }
          __syncthreads();
        }
      }
    }
    __syncthreads();  // the buffers are free for the next segment
    u += ku_end - ku;
  }
}

template <typename E, int D, int RT, bool PAGED, bool Q8>
hipError_t launch(const AttnArgs& a, hipStream_t s) {
  const int workgroups = narrow_workgroups(a.rows, a.heads_kv);
  hipLaunchKernelGGL((attn_narrow_kernel<E, D, RT, PAGED, Q8>), dim3(workgroups), dim3(64 * WAVES), 0, s, a, workgroups);
  return hipGetLastError();
}

template <int RT, bool PAGED, bool Q8>
hipError_t launch_d(const AttnArgs& a, hipStream_t s) {
  if (a.head_dim == 128) return a.bf16 ? launch<BF16, 128, RT, PAGED, Q8>(a, s) : launch<F16, 128, RT, PAGED, Q8>(a, s);
  return a.bf16 ? launch<BF16, 64, RT, PAGED, Q8>(a, s) : launch<F16, 64, RT, PAGED, Q8>(a, s);
}

}  // namespace
}  // namespace qg
