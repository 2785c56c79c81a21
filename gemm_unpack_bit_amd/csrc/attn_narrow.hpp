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
// A cache of 8 bits: the same with codes in place of values on their way, by LDS
// (Codes), which become values of the element type (e4m3.hpp) when they are used;
// a tile of 16 keys is one block, with one exponent for its keys and one for its
// values.  Measured: 32 rows of 4500 keys on average, 64 heads over 8, 72 us, of
// 18000 239 us (4.3 and 5.1 TB/s; 16-bit keys 115 and 410 us, 5.3 and 5.8).  What
// bounds it is the codes' way from memory, though not its rate: before the loads
// were marked as read once only, they alone, without any products, took 75 and 256
// of 79 and 262 us, whether one step or two were on their way, in pages of 16 as
// in pages of 256.
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

// Codes of two steps on their way: a part of LDS for each wave, per step two tiles
// of 16 keys and of their values.  They go from memory straight into LDS, so that
// neighbouring lanes ask for neighbouring pieces of a key, 128 bytes at once, and
// marked as read once only.  (Unmarked 79 and 262 us in place of 72 and 239.  Loads
// into the registers where the matrix products want them, 16 bytes of each of 16
// keys, took 75 and 247 us, marked or not.)
//
// A row of a tile is one key's codes (or values').  The 16-byte pieces of a key are
// stored in an order of its own, and the rows of values in another order, so that
// the lanes' reads spread over the banks.
template <int D>
struct __attribute__((aligned(16))) Codes {
  static constexpr int PC = D / 16;       // pieces of a row
  static constexpr int RPL = 64 / PC;     // rows of a wave-wide load
  static constexpr int LOADS = 16 / RPL;  // loads of a tile
  struct Stage {
    uint8_t k[2][16 * D], v[2][16 * D];
  } stage[2];
  static __device__ __forceinline__ int piece_order(int key) { return D == 128 ? key >> 1 & 7 : key >> 2 & 3; }
  static __device__ __forceinline__ int row_order(int key) { return key ^ (key >> 2); }  // (its own inverse)
  typedef __attribute__((address_space(3))) uint8_t* lds;
  typedef __attribute__((address_space(1))) const char* global;

  // Asks for a tile: keys past `last` (of 16) from the last one's place.
  template <bool V>
  static __device__ __forceinline__ void load(uint8_t* tile, global from, uint32_t row_bytes, int last) {
    const int lane = threadIdx.x & 63;
#pragma unroll
    for (int i = 0; i < LOADS; ++i) {
      const int row = RPL * i + lane / PC, key = V ? row_order(row) : row;
      const int piece = V ? lane % PC : (lane % PC) ^ piece_order(row);
      __builtin_amdgcn_global_load_lds(
          (__attribute__((address_space(1))) const void*)(from + (uint32_t)min(key, last) * row_bytes + 16 * piece),
          (__attribute__((address_space(3))) void*)(tile + 1024 * i), 16, 0, CPOL_NT);
    }
  }
  // Both read once their tiles have arrived: AFTER loads, at least, have been asked
  // for behind these, and arrive behind them.  (The wait is in the block with the
  // reads; by itself the compiler waits for every load on its way.)
  //
  // K: a lane's pieces of key n16 of both tiles: piece `quarter`, and of 8 pieces
  // the one 4 behind it.
  template <int AFTER>
  static __device__ __forceinline__ void read_k(const Stage& s, int n16, int quarter, u4 (&c)[2][PC / 4]) {
    const uint32_t at = (uint32_t)(uintptr_t)(lds)(uint8_t*)s.k + n16 * D + 16 * (quarter ^ piece_order(n16));
    if constexpr (D == 128)
      asm volatile(
          "s_waitcnt vmcnt(%6)\n\tds_read_b128 %0, %4\n\tds_read_b128 %1, %5\n\tds_read_b128 %2, %4 offset:2048\n\t"
          "ds_read_b128 %3, %5 offset:2048\n\ts_waitcnt lgkmcnt(0)"
          : "=&v"(c[0][0]), "=&v"(c[0][1]), "=&v"(c[1][0]), "=&v"(c[1][1])
          : "v"(at), "v"(at ^ 64), "n"(AFTER)
          : "memory");
    else
      asm volatile("s_waitcnt vmcnt(%3)\n\tds_read_b128 %0, %2\n\tds_read_b128 %1, %2 offset:1024\n\ts_waitcnt lgkmcnt(0)"
                   : "=&v"(c[0][0]), "=&v"(c[1][0])
                   : "v"(at), "n"(AFTER)
                   : "memory");
  }
  // V: the lane's D / 16 columns of the keys 4 quarter + i of both tiles
  template <int AFTER, typename W>
  static __device__ __forceinline__ void read_v(const Stage& s, int n16, int quarter, W (&c)[8]) {
    const uint32_t base = (uint32_t)(uintptr_t)(lds)(uint8_t*)s.v + D / 16 * n16;
    uint32_t at[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) at[i] = base + row_order(4 * quarter + i) * D;
    if constexpr (D == 128)
      asm volatile(
          "s_waitcnt vmcnt(%12)\n\tds_read_b64 %0, %8\n\tds_read_b64 %1, %9\n\tds_read_b64 %2, %10\n\tds_read_b64 %3, %11\n\t"
          "ds_read_b64 %4, %8 offset:2048\n\tds_read_b64 %5, %9 offset:2048\n\tds_read_b64 %6, %10 offset:2048\n\t"
          "ds_read_b64 %7, %11 offset:2048\n\ts_waitcnt lgkmcnt(0)"
          : "=&v"(c[0]), "=&v"(c[1]), "=&v"(c[2]), "=&v"(c[3]), "=&v"(c[4]), "=&v"(c[5]), "=&v"(c[6]), "=&v"(c[7])
          : "v"(at[0]), "v"(at[1]), "v"(at[2]), "v"(at[3]), "n"(AFTER)
          : "memory");
    else {
      uint32_t w[8];
      asm volatile(
          "s_waitcnt vmcnt(%12)\n\tds_read_b32 %0, %8\n\tds_read_b32 %1, %9\n\tds_read_b32 %2, %10\n\tds_read_b32 %3, %11\n\t"
          "ds_read_b32 %4, %8 offset:1024\n\tds_read_b32 %5, %9 offset:1024\n\tds_read_b32 %6, %10 offset:1024\n\t"
          "ds_read_b32 %7, %11 offset:1024\n\ts_waitcnt lgkmcnt(0)"
          : "=&v"(w[0]), "=&v"(w[1]), "=&v"(w[2]), "=&v"(w[3]), "=&v"(w[4]), "=&v"(w[5]), "=&v"(w[6]), "=&v"(w[7])
          : "v"(at[0]), "v"(at[1]), "v"(at[2]), "v"(at[3]), "n"(AFTER)
          : "memory");
#pragma unroll
      for (int i = 0; i < 8; ++i) c[i][0] = w[i];
    }
  }
};

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
  // (the codes' places are those of the sums that are joined behind the last step)
  constexpr size_t SUMS = sizeof(float) * WAVES * BM * PITCH, CODES = Q8 ? sizeof(Codes<D>) * WAVES : 0;
  __shared__ __attribute__((aligned(16))) uint8_t places[SUMS > CODES ? SUMS : CODES];
  auto& o_s = *reinterpret_cast<float(*)[WAVES][BM][PITCH]>(places);
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

    // Loads of a step: tiles of 16 keys, each 16 rows of one page, by a
    // scalar base and a lane's 32-bit offset.  A tile past the row's last key
    // falls back on the last tile that has any, and a key past the last is read
    // from the last one's place.
    constexpr int W = Q8 ? 1 : 2;  // bytes of a key's element
    typedef __attribute__((address_space(1))) const char* global;
    global kh = (global)(reinterpret_cast<const char*>(a.k) + (int64_t)h * a.k_head * W);
    global vh = (global)(reinterpret_cast<const char*>(a.v) + (int64_t)h * a.v_head * W);
    uint32_t k_row = (uint32_t)W * (uint32_t)a.k_token, v_row = (uint32_t)W * (uint32_t)a.v_token;  // bytes
    int shift = a.page_shift;
    // (kept in registers: read again from the arguments, a step would wait for them)
    if constexpr (Q8) asm volatile("" : "+s"(kh), "+s"(vh), "+s"(k_row), "+s"(v_row), "+s"(shift));
    const int top = (r.keys - 1) & ~15;
    auto token_at = [&](int kb) -> int64_t {
      kb = kb < top ? kb : top;
      if constexpr (PAGED) return pool_token(a, b, kb);
      else return (int64_t)r.k0 + kb;
    };
    u4 kf[2][Q8 ? KS / 2 : KS];
    vw vf[Q8 ? 1 : 8];
    // a step's codes of values, and both exponents of the tiles of the steps on
    // their way
    typedef uint32_t cw __attribute__((ext_vector_type(DW > 2 ? 2 : 1)));
    cw vc[Q8 ? 8 : 1];
    uint32_t ex[2][2];
    Codes<D>* codes = reinterpret_cast<Codes<D>*>(places) + wave;
    // (a lane's offsets in a tile with all its keys)
    const uint32_t k_off = (uint32_t)n16 * k_row + 16u * quarter, v_off = 4u * quarter * v_row + (uint32_t)W * DL * n16;
    // Codes: the tiles of the wave's next 32 steps are looked up at once, one per
    // lane, pages and exponents, so that a step needs a few lane reads.  (With
    // lookups in every step, 80 us in place of 75 on the same 32 rows of 4500 keys.)
    uint32_t pages_l = 0, exps_l = 0;
    int from = 0;  // the first of these steps
    auto look_up = [&](int kb) {
      from = kb;
      const AttnArgs e = args_again();
      const int at = min(kb + (lane >> 1) * KB + 16 * (lane & 1), top);
      const int page = e.tables[(int64_t)b * e.max_pages + (at >> e.page_shift)];
      pages_l = (unsigned)page < (unsigned)e.pages ? page : 0;
      const int64_t block = (((int64_t)pages_l << e.page_shift) + (at & ((1 << e.page_shift) - 1))) / KV_BLOCK * e.heads_kv + h;
      exps_l = e.k_exps[block] | (uint32_t)e.v_exps[block] << 8;
    };
    struct Tiles {
      int64_t tok[2];
      uint32_t ex[2];
    };
    auto tiles_at = [&](int kb) {
      if (kb - from >= 32 * KB) look_up(kb);
      Tiles t;
#pragma unroll
      for (int x = 0; x < 2; ++x) {
        const int l = 2 * ((kb - from) / KB) + x;
        t.tok[x] = ((int64_t)__builtin_amdgcn_readlane(pages_l, l) << shift) + (min(kb + 16 * x, top) & ((1 << shift) - 1));
        t.ex[x] = __builtin_amdgcn_readlane(exps_l, l);
      }
      return t;
    };
    auto last_of = [&](int k0) { return r.keys - 1 - (k0 < top ? k0 : top); };
    auto load_k = [&](int st, int kb, const int64_t (&tok)[2]) {
#pragma unroll
      for (int x = 0; x < 2; ++x) {
        const int k0 = kb + 16 * x;
        if constexpr (Q8) {
          Codes<D>::template load<false>(codes->stage[st].k[x], kh + tok[x] * k_row, k_row, k0 + 16 > r.keys ? last_of(k0) : 15);
        } else {
          global p = kh + tok[x] * a.k_token * W;
          uint32_t off = k_off;
          if (k0 + 16 > r.keys) off = (uint32_t)min(n16, last_of(k0)) * k_row + 16u * quarter;
#pragma unroll
          for (int s = 0; s < KS; ++s) kf[x][s] = *(__attribute__((address_space(1))) const u4*)(p + off + 64 * s);
        }
      }
    };
    auto load_v = [&](int st, int kb, const int64_t (&tok)[2]) {
#pragma unroll
      for (int x = 0; x < 2; ++x) {
        const int k0 = kb + 16 * x;
        if constexpr (Q8) {
          Codes<D>::template load<true>(codes->stage[st].v[x], vh + tok[x] * v_row, v_row, k0 + 16 > r.keys ? last_of(k0) : 15);
        } else {
          global p = vh + tok[x] * a.v_token * W;
          uint32_t off[4];
#pragma unroll
          for (int i = 0; i < 4; ++i) off[i] = v_off + i * v_row;
          if (k0 + 16 > r.keys)
#pragma unroll
            for (int i = 0; i < 4; ++i) off[i] = (uint32_t)min(4 * quarter + i, last_of(k0)) * v_row + (uint32_t)W * DL * n16;
#pragma unroll
          for (int i = 0; i < 4; ++i)
            vf[4 * x + i] = __builtin_nontemporal_load((__attribute__((address_space(1))) const vw*)(p + off[i]));
        }
      }
    };
    // K fragments of the products s and s + 1 (s even) of a tile: a lane's 16 codes
    // serve both
    auto k_frags = [&](int st, int x, int s, u4& k0, u4& k1) {
      if constexpr (Q8) {
        const u4 c = kf[x][s / 2];
        const float by = exp_scale(ex[st][x] & 0xFF);
        k0 = decode8<E>(c[0], c[1], by);
        k1 = decode8<E>(c[2], c[3], by);
      } else {
        k0 = kf[x][s];
        k1 = kf[x][s + 1];
      }
    };
    // V fragments of the products j and j + 1 (j even): a column's 8 keys.  Of
    // codes, a permute gathers two keys' of both columns.
    auto v_frags = [&](int st, int j, u4& va, u4& vb) {
#pragma unroll
      for (int w = 0; w < 4; ++w) {
        if constexpr (Q8) {
          const uint32_t c = __builtin_amdgcn_perm(vc[2 * w + 1][j / 4], vc[2 * w][j / 4], j & 2 ? 0x07030602u : 0x05010400u);
          const float by = exp_scale(ex[st][w / 2] >> 8);
          va[w] = decode2<E, false>(c, by);
          vb[w] = decode2<E, true>(c, by);
        } else {
          va[w] = __builtin_amdgcn_perm(vf[2 * w + 1][j / 2], vf[2 * w][j / 2], 0x05040100u);
          vb[w] = __builtin_amdgcn_perm(vf[2 * w + 1][j / 2], vf[2 * w][j / 2], 0x07060302u);
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
    // rescaling: they are infinite or NaN).  Codes are in the way there: their
    // values go into the lane's sums.
    bool odd_any = false;
    auto add_odd = [&](uint64_t odd, int kb) {
      const AttnArgs e = args_again();
      float* sums = &o_s[wave][0][0];
      if constexpr (!Q8) {
        if (!odd_any)
          for (int x = lane; x < BM * PITCH; x += 64) sums[x] = 0.f;
        odd_any = true;
      }
      for (; odd; odd &= odd - 1) {
        const int key = __builtin_ctzll(odd), at = min(kb + key, r.keys - 1);
        const int64_t tok = token_at(at & ~15) + (at & 15), v0 = (int64_t)h * e.v_head + tok * e.v_token;
        if constexpr (Q8) {
          const uint8_t* c = reinterpret_cast<const uint8_t*>(e.v) + v0 + DL * 4 * quarter;
          const float by = exp_scale(e.v_exps[tok / KV_BLOCK * e.heads_kv + h]);
#pragma unroll
          for (int i = 0; i < RT; ++i) {
            const uint32_t sees = sight[i].window(e, r, kb) >> key & 1 ? 0x8000u : 0u;
#pragma unroll
            for (int j = 0; j < DL; ++j)
#pragma unroll
              for (int d = 0; d < 4; ++d) {
                const uint16_t y = (uint16_t)decode2<E, false>(c[DL * d + j], by);
                o[i][j][d] += nonfinite<E>(y) & sees ? E::value(y) : 0.f;
              }
          }
        } else {
#pragma unroll
          for (int i = 0; i < RT; ++i) {
            uint32_t see = (uint32_t)__ballot(sight[i].window(e, r, kb) >> key & 1) & 0xFFFF;
            for (; see; see &= see - 1)
#pragma unroll
              for (int d0 = 0; d0 < D; d0 += 64) {
                const uint16_t y = e.v[v0 + d0 + lane];
                sums[(16 * i + __builtin_ctz(see)) * PITCH + d0 + lane] += nonfinite<E>(y) & 0x8000u ? E::value(y) : 0.f;
              }
          }
        }
      }
    };
    int64_t tok1[2];  // the next step's
    // Takes values that are infinite or NaN out of the step's, and returns the
    // keys that have one: a weight of 0 does not cancel them.
    auto clean = [&](int st) -> uint64_t {
      uint32_t bad = 0;
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        uint32_t f = 0;
        if constexpr (Q8) {
#pragma unroll
          for (int w = 0; w < (DW > 2 ? 2 : 1); ++w) {
            const float by = exp_scale(ex[st][i / 4] >> 8);
            const uint32_t c = vc[i][w];
            const uint32_t x = nonfinite<E>(decode2<E, false>(c, by)), y = nonfinite<E>(decode2<E, true>(c, by));
            f |= x | y;
            // codes to clear: bits 15 and 31 of x and y, a byte each
            const uint32_t z = (x >> 15 & 1) | (x >> 23 & 0x100) | (y << 1 & 0x10000) | (y >> 7 & 0x1000000);
            vc[i][w] &= ~(z * 0xFF);
          }
        } else {
#pragma unroll
          for (int w = 0; w < DW; ++w) {
            const uint32_t x = nonfinite<E>(vf[i][w]);
            f |= x;
            // halves to clear: 0x8000 of a half becomes 0xFFFF
            vf[i][w] &= ~((x - (x >> 15)) | x);
          }
        }
        bad |= f ? 1u << i : 0u;
      }
      uint64_t odd = 0;
      if (__any(bad))
#pragma unroll
        for (int i = 0; i < 8; ++i)
#pragma unroll
          for (int qd = 0; qd < 4; ++qd)
            if (__ballot(bad >> i & 1) >> (16 * qd) & 0xFFFF) odd |= 1ull << ((i < 4 ? i : 12 + i) + 4 * qd);
      return odd;
    };
    // Stage st holds the step's keys and values, and takes those of the step `next`
    // keys on, where `more` says that there are any (at tok1).  after: loads asked
    // for behind the step's keys, and behind its values (codes).
    auto step = [&](int st, int next, bool more, auto after) {
      f4 sc[RT][2];
      if constexpr (Q8) {
        Codes<D>::template read_k<decltype(after)::value>(codes->stage[st], n16, quarter, kf);
        __builtin_amdgcn_sched_barrier(0);
        if (more) load_k(st, kb + next, tok1);
        __builtin_amdgcn_sched_barrier(0);
      }
#pragma unroll
      for (int x = 0; x < 2; ++x)
#pragma unroll
        for (int s = 0; s < KS; s += 2) {
          u4 k0, k1;
          k_frags(st, x, s, k0, k1);
#pragma unroll
          for (int i = 0; i < RT; ++i) {
            sc[i][x] = E::mfma16(k0, qf[i][s], s ? sc[i][x] : f4{0.f, 0.f, 0.f, 0.f});
            sc[i][x] = E::mfma16(k1, qf[i][s + 1], sc[i][x]);
          }
        }
      if constexpr (!Q8) {
        __builtin_amdgcn_sched_barrier(0);
        if (more) load_k(st, kb + next, tok1);
        __builtin_amdgcn_sched_barrier(0);
      }

      if (zero_scale(a.scale))
#pragma unroll
        for (int i = 0; i < RT; ++i) sc[i][0] -= sc[i][0], sc[i][1] -= sc[i][1];
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
        if constexpr (!Q8) odd = clean(st);
      }

      u4 pf[RT];
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
        pf[i] = u4{E::pack(p[0], p[1]), E::pack(p[2], p[3]), E::pack(p[4], p[5]), E::pack(p[6], p[7])};
      }
      if constexpr (Q8) {
        Codes<D>::template read_v<decltype(after)::value>(codes->stage[st], n16, quarter, vc);
        __builtin_amdgcn_sched_barrier(0);
        if (more) load_v(st, kb + next, tok1);
        __builtin_amdgcn_sched_barrier(0);
        if (masked) odd = clean(st);
      }
#pragma unroll
      for (int j = 0; j < DL; j += 2) {
        u4 va, vb;
        v_frags(st, j, va, vb);
#pragma unroll
        for (int i = 0; i < RT; ++i) {
          o[i][j] = E::mfma16(va, pf[i], o[i][j]);
          o[i][j + 1] = E::mfma16(vb, pf[i], o[i][j + 1]);
        }
      }
      if (odd) add_odd(odd, kb);
      if constexpr (!Q8) {
        __builtin_amdgcn_sched_barrier(0);
        if (more) load_v(st, kb + next, tok1);
        __builtin_amdgcn_sched_barrier(0);
      }
    };
    constexpr std::integral_constant<int, 0> none{};
    if constexpr (Q8) {
      if (kb < k_end) {
        look_up(kb);
        auto fill = [&](int st) {
          const Tiles t = tiles_at(kb + KB * st);
          __builtin_amdgcn_sched_barrier(0);
          load_k(st, kb + KB * st, t.tok);
          __builtin_amdgcn_sched_barrier(0);
          load_v(st, kb + KB * st, t.tok);
          __builtin_amdgcn_sched_barrier(0);
          ex[st][0] = t.ex[0], ex[st][1] = t.ex[1];
        };
        auto turn = [&](int st, bool more, auto after) {
          Tiles t = {};
          if (more) t = tiles_at(kb + 2 * KB);
          tok1[0] = t.tok[0], tok1[1] = t.tok[1];
          step(st, 2 * KB, more, after);
          ex[st][0] = t.ex[0], ex[st][1] = t.ex[1];
          kb += KB;
        };
        fill(0);
        if (kb + KB < k_end) fill(1);
        // Behind a step's keys: its values, and the next step's keys and values;
        // behind its values: these, and the keys of the step after that.
        constexpr std::integral_constant<int, 3 * 2 * Codes<D>::LOADS> three{};
        while (kb + 3 * KB < k_end) {
          turn(0, true, three);
          turn(1, true, three);
        }
        // (the last ones wait for all)
        for (;;) {
          turn(0, kb + 2 * KB < k_end, none);
          if (kb >= k_end) break;
          turn(1, kb + 2 * KB < k_end, none);
          if (kb >= k_end) break;
        }
      }
      __syncthreads();  // the codes' places are free
    } else if (kb < k_end) {
      const int64_t tok0[2] = {token_at(kb), token_at(kb + 16)};
      load_k(0, kb, tok0);
      load_v(0, kb, tok0);
#pragma unroll
      for (int x = 0; x < 2; ++x) tok1[x] = token_at(kb + KB + 16 * x);
      for (; kb + KB < k_end; kb += KB) {
        // (looked up a step ahead of the loads)
        const int64_t tok2[2] = {token_at(kb + 2 * KB), token_at(kb + 2 * KB + 16)};
        step(0, KB, true, none);
        tok1[0] = tok2[0], tok1[1] = tok2[1];
      }
      step(0, KB, false, none);
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
