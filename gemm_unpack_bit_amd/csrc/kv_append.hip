// New tokens into the paged cache with their position rotation, and values of
// the cache back into packed arrays.
//
// Mathematics.  Pair i of a head (elements i and i + rot / 2, or 2 i and
// 2 i + 1) turns by the angle t = position * freqs[i]:
//     (a, b) -> (a cos t - b sin t, a sin t + b cos t)
// in fp32, rounded once: to 16 bits, or to e4m3 under the block's exponent.
// The angle's whole turns are taken off in 64 bits (in 32, a position of
// 131072 would leave 2^-7 of a radian), its sine and cosine are of 32 bits.
//
// Cache of 8 bits: a block of 16 tokens and head has one power of two, the
// least that holds the largest of its tokens without saturation.  A new token
// may ask for more than the block has: then the codes that are there are
// written anew under the larger one (exact but for codes that become
// subnormal).  Infinities and NaN become NaN codes and do not count.
//
// Bound: memory; a decode step's few tokens: launch and four trips to memory
// (row, position, page, exponent).  A lane has 16 elements: two pieces of 8,
// whose pairs turn by the same eight angles in every head, so a wave works out
// the sines of its token once for all heads that it takes.
//
// Measured: 48 tokens of 32 heads over 8 into 16 bits 4.2 us, into 8 bits 5;
// 8192 tokens of 64 heads over 8 into 16 bits 65 us (335 MB, 5.2 TB/s), into 8
// bits 63; 10000 tokens read back out of 8 bits 14 to 15 us, out of 16 bits 13 to 14.
#include "e4m3.hpp"

namespace qg {
namespace {

constexpr int WAVES = 4;

// a lane's 16 elements of a head: pieces of 8 at `first` and `second`
template <int D>
struct Unit {
  int first, second;
  bool turns;
  __device__ __forceinline__ Unit(const KvAppendArgs& a, int u) {
    turns = 16 * u < a.rot;
    const bool halves = turns && !a.interleaved;
    first = halves ? 8 * u : 16 * u;
    second = halves ? a.rot / 2 + 8 * u : 16 * u + 8;
  }
};

struct Angles {
  float c[8], s[8];
  __device__ __forceinline__ void set(const KvAppendArgs& a, int u, int at) {
    const f4* f = reinterpret_cast<const f4*>(a.freqs + 8 * u);
    const f4 f0 = f[0], f1 = f[1];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const double turns = (double)at * ((double)(i < 4 ? f0[i & 3] : f1[i & 3]) * 0.15915494309189535);
      sincospif(2.f * (float)(turns - __builtin_rint(turns)), &s[i], &c[i]);
    }
  }
  // x: the lane's elements, pieces one behind the other
  __device__ __forceinline__ void turn(float (&x)[16], bool interleaved) const {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float a = interleaved ? x[2 * i] : x[i], b = interleaved ? x[2 * i + 1] : x[8 + i];
      const float p = a * c[i] - b * s[i], q = a * s[i] + b * c[i];
      if (interleaved) x[2 * i] = p, x[2 * i + 1] = q;
      else x[i] = p, x[8 + i] = q;
    }
  }
};

template <typename E>
__device__ __forceinline__ void unpack16(const u4& lo, const u4& hi, float (&x)[16]) {
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    x[i] = E::value((uint16_t)(lo[i / 2] >> (16 * (i & 1))));
    x[8 + i] = E::value((uint16_t)(hi[i / 2] >> (16 * (i & 1))));
  }
}
template <typename E>
__device__ __forceinline__ u4 pack8(const float* x) {
  return u4{E::pack(x[0], x[1]), E::pack(x[2], x[3]), E::pack(x[4], x[5]), E::pack(x[6], x[7])};
}

// the row of token t, or -1: its number b, the token's place in the row
struct Place {
  int b, i;
};
__device__ __forceinline__ Place place_of(const int32_t* cu, int rows, int t) {
  const int b = find_row(rows, t, [&](int r) { return cu[r]; });
  const int i = t - cu[b];
  return {i < 0 || t >= cu[b + 1] ? -1 : b, i};
}
// the pool token (page * page_size + place) of position p of row b; -1: none
__device__ __forceinline__ int64_t pool_place(const KvArgs& c, int b, int64_t p) {
  const int64_t slot = p >> c.page_shift;
  if (p < 0 || slot >= c.max_pages) return -1;
  const int page = c.tables[(int64_t)b * c.max_pages + slot];
  if ((unsigned)page >= (unsigned)c.pages) return -1;
  return ((int64_t)page << c.page_shift) + (p & ((1 << c.page_shift) - 1));
}

// Heads of one token by one wave: `n` heads from `h0` on of the queries, then
// keys, then values (a cache of 8 bits: of the queries).  2 H of them are on
// their way at any time, the first ones while their place is found.
template <typename E, int D, bool TURN>
__device__ __forceinline__ void token_heads(const KvAppendArgs& a, int t, int h0, int n) {
  constexpr int U = D / 16, H = 64 / U;  // units of a head, heads at a time
  const int lane = threadIdx.x & 63, u = lane % U;
  const Unit<D> unit(a, u);
  u4 next[2][2];
  auto load = [&](int i) {
#pragma unroll
    for (int x = 0; x < 2; ++x) {
      if (i + H * x >= n) continue;
      const int h = h0 + i + H * x, hk = h - a.heads, hv = hk - a.c.heads_kv;
      const uint16_t* from = hk < 0   ? a.q + (int64_t)t * a.q_token + h * a.q_head
                             : hv < 0 ? a.k + (int64_t)t * a.k_token + hk * a.k_head
                                      : a.v + (int64_t)t * a.v_token + hv * a.v_head;
      next[x][0] = *reinterpret_cast<const u4*>(from + unit.first);
      next[x][1] = *reinterpret_cast<const u4*>(from + unit.second);
    }
  };
  load(lane / U);
  const Place w = place_of(a.cu, a.c.rows, t);
  if (w.b < 0) return;
  const int p0 = a.pos[w.b];
  if (p0 < 0) return;
  const int64_t p = (int64_t)p0 + w.i;
  const int64_t at = h0 + n > a.heads ? pool_place(a.c, w.b, p) : -1;
  const int64_t row = (int64_t)a.c.heads_kv * D;
  Angles ang;
  if (TURN && unit.turns) ang.set(a, u, a.at ? a.at[t] : (int)p);
  for (int i = lane / U; i < n; i += 2 * H) {
    u4 now[2][2];
#pragma unroll
    for (int x = 0; x < 2; ++x) now[x][0] = next[x][0], now[x][1] = next[x][1];
    load(i + 2 * H);
#pragma unroll
    for (int x = 0; x < 2; ++x) {
      if (i + H * x >= n) continue;
      const int h = h0 + i + H * x, hk = h - a.heads, hv = hk - a.c.heads_kv;
      uint16_t* to;
      if (hk < 0) {
        to = a.o + (int64_t)t * a.o_token + h * a.o_head;
      } else {
        if (at < 0) continue;
        const int64_t in_layer = ((int64_t)a.layer * a.c.pages << a.c.page_shift) + at;
        to = (hv < 0 ? a.c.k : a.c.v) + in_layer * row + (hv < 0 ? hk : hv) * D;
      }
      u4 lo = now[x][0], hi = now[x][1];
      if (TURN && unit.turns && hv < 0) {
        float v[16];
        unpack16<E>(lo, hi, v);
        if (a.interleaved) ang.turn(v, true);
        else ang.turn(v, false);
        lo = pack8<E>(v);
        hi = pack8<E>(v + 8);
      }
      *reinterpret_cast<u4*>(to + unit.first) = lo;
      *reinterpret_cast<u4*>(to + unit.second) = hi;
    }
  }
}

// One block of 16 tokens of the 8-bit cache: heads [h0, h1) of keys (which 0)
// or values (1), by one wave.  A lane has one unit of every token t % TP, TP
// tokens at a time.
template <typename E, int D, bool TURN>
__device__ __forceinline__ void block_heads(const KvAppendArgs& a, int b, int p0, int n, int64_t first, int which, int h0,
                                            int h1) {
  constexpr int U = D / 16, TP = 64 / U, PASSES = KV_BLOCK / TP;
  const int lane = threadIdx.x & 63, u = lane % U;
  const Unit<D> unit(a, u);
  const bool turn = TURN && which == 0 && unit.turns;
  const uint16_t* src = which ? a.v : a.k;
  const int64_t token = which ? a.v_token : a.k_token, head = which ? a.v_head : a.k_head;
  const int64_t end = (int64_t)p0 + n;
  const int i0 = p0 > first ? (int)(p0 - first) : 0, i1 = end - first < KV_BLOCK ? (int)(end - first) : KV_BLOCK;  // new ones
  const int64_t t0 = a.cu[b] + (first - p0);  // the token at the block's first place
  // (a head's pieces are on their way while the one before it is written)
  u4 next[PASSES][2];
  auto load = [&](int h) {
#pragma unroll
    for (int x = 0; x < PASSES; ++x) {
      const int i = TP * x + lane / U;
      if (i < i0 || i >= i1) continue;
      const uint16_t* from = src + (t0 + i) * token + h * head;
      next[x][0] = *reinterpret_cast<const u4*>(from + unit.first);
      next[x][1] = *reinterpret_cast<const u4*>(from + unit.second);
    }
  };
  load(h0);
  const int64_t place = pool_place(a.c, b, first);  // (a block lies in one page)
  if (place < 0) return;
  const int64_t in_layer = ((int64_t)a.layer * a.c.pages << a.c.page_shift) + place;
  uint8_t* codes = reinterpret_cast<uint8_t*>(which ? a.c.v : a.c.k) + in_layer * a.c.heads_kv * D;
  uint8_t* exps = (which ? a.c.v_exps : a.c.k_exps) + in_layer / KV_BLOCK * a.c.heads_kv;
  Angles ang[PASSES];
  if (turn)
#pragma unroll
    for (int x = 0; x < PASSES; ++x) {
      const int i = TP * x + lane / U;
      if (i >= i0 && i < i1) ang[x].set(a, u, a.at ? a.at[t0 + i] : (int)(first + i));
    }
  for (int h = h0; h < h1; ++h) {
    float v[PASSES][16];
    float most = 0.f;
    const int had = i0 ? exps[h] : 0;
    u4 raw[PASSES][2];
#pragma unroll
    for (int x = 0; x < PASSES; ++x) raw[x][0] = next[x][0], raw[x][1] = next[x][1];
    if (h + 1 < h1) load(h + 1);
#pragma unroll
    for (int x = 0; x < PASSES; ++x) {
      const int i = TP * x + lane / U;
      if (i < i0 || i >= i1) continue;
      unpack16<E>(raw[x][0], raw[x][1], v[x]);
      if (turn) {
        if (a.interleaved) ang[x].turn(v[x], true);
        else ang[x].turn(v[x], false);
      }
#pragma unroll
      for (int e = 0; e < 16; ++e) {
        const bool odd = (__float_as_uint(v[x][e]) & 0x7F800000u) == 0x7F800000u;
        v[x][e] = odd ? __builtin_nanf("") : v[x][e];
        most = fmaxf(most, fabsf(v[x][e]));  // (passes over NaN)
      }
    }
    most = fmaxf(most, dpp<DPP_QP_XOR1>(most));
    most = fmaxf(most, dpp<DPP_QP_XOR2>(most));
    most = fmaxf(most, dpp<DPP_ROR4>(most));
    most = fmaxf(most, dpp<DPP_ROR8>(most));
    const int need = exp_byte(quarter_max(most));
    // (what the block has may be any exponent, below the least that is given here
    // and above the largest too)
    const int old = (int)exp_of(had), now = i0 && old > need ? old : need;
    const float by = exp_inverse(now);
#pragma unroll
    for (int x = 0; x < PASSES; ++x) {
      const int i = TP * x + lane / U;
      uint8_t* to = codes + ((int64_t)i * a.c.heads_kv + h) * D;
      if (i < i0) {
        if (now == old) continue;
        u4* at = reinterpret_cast<u4*>(to + 16 * u);
        u4 w = *at;
#pragma unroll
        for (int e = 0; e < 4; ++e) w[e] = rescale4(w[e], exp_ratio(old, now));
        *at = w;
      } else if (i < i1) {
        u4 w;
#pragma unroll
        for (int e = 0; e < 4; ++e)
          w[e] = encode4(v[x][4 * e] * by, v[x][4 * e + 1] * by, v[x][4 * e + 2] * by, v[x][4 * e + 3] * by);
        *reinterpret_cast<u2*>(to + unit.first) = u2{w[0], w[1]};
        *reinterpret_cast<u2*>(to + unit.second) = u2{w[2], w[3]};
      }
    }
    if (lane == 0) exps[h] = (uint8_t)now;
  }
}

// Work of a wave: first (8 bits) the blocks, whose waves have more to do, then
// the tokens' heads, `slice` of them at a time.  Row b's blocks have the numbers
// from cu[b] / 16 + 2 b on, which is at least as many as it touches and needs no
// sum over the rows.
template <typename E, int D, bool TURN, bool Q8>
__global__ void __launch_bounds__(64 * WAVES) kv_append_kernel(KvAppendArgs a, int slices, int slice, int group) {
  int64_t wave = (int64_t)blockIdx.x * WAVES + __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  if constexpr (Q8) {
    const int parts = 2 * ((a.c.heads_kv + group - 1) / group);
    const int64_t blocks = (int64_t)a.tokens / KV_BLOCK + 2 * (int64_t)a.c.rows;
    if (wave < blocks * parts) {
      const int slot = (int)(wave / parts), part = (int)(wave % parts), which = part & 1, h0 = part / 2 * group;
      const int b = find_row(a.c.rows, slot, [&](int r) { return clamp_cu(a.cu[r], a.tokens) / KV_BLOCK + 2 * r; });
      const int c0 = clamp_cu(a.cu[b], a.tokens), n = clamp_cu(a.cu[b + 1], a.tokens) - c0, p0 = a.pos[b];
      if (n <= 0 || p0 < 0 || a.cu[b] != c0) return;
      const int64_t first = ((int64_t)(p0 / KV_BLOCK) + slot - (c0 / KV_BLOCK + 2 * b)) * KV_BLOCK;
      if (first < p0 - KV_BLOCK + 1 || first >= (int64_t)p0 + n) return;
      block_heads<E, D, TURN>(a, b, p0, n, first, which, h0, min(h0 + group, a.c.heads_kv));
      return;
    }
    wave -= blocks * parts;
  }
  if (wave >= (int64_t)a.tokens * slices) return;  // (8 bits without queries: no slices)
  const int t = (int)(wave / slices), h0 = (int)(wave % slices) * slice;
  const int all = Q8 ? a.heads : a.heads + 2 * a.c.heads_kv;
  token_heads<E, D, TURN>(a, t, h0, min(slice, all - h0));
}

// One wave per token: units of its keys, then of its values.
template <typename E, int D, bool Q8>
__global__ void __launch_bounds__(64 * WAVES) kv_read_kernel(KvReadArgs a) {
  constexpr int U = D / 16;
  const int lane = threadIdx.x & 63;
  const int t = __builtin_amdgcn_readfirstlane(blockIdx.x * WAVES + (threadIdx.x >> 6));
  if (t >= a.tokens) return;
  const Place w = place_of(a.cu, a.c.rows, t);
  if (w.b < 0) return;
  const int p0 = a.start[w.b];
  if (p0 < 0) return;
  const int64_t at = pool_place(a.c, w.b, (int64_t)p0 + w.i);
  if (at < 0) return;
  const int64_t in_layer = ((int64_t)a.layer * a.c.pages << a.c.page_shift) + at;
  const int64_t row = (int64_t)a.c.heads_kv * D;
#pragma unroll 2
  for (int i = lane; i < 2 * a.c.heads_kv * U; i += 64) {
    const bool value = i >= a.c.heads_kv * U;
    const int h = i / U - (value ? a.c.heads_kv : 0), d = 16 * (i % U);
    const uint16_t* pool = value ? a.c.v : a.c.k;
    uint16_t* to = value ? a.v + (int64_t)t * a.v_token + h * a.v_head + d : a.k + (int64_t)t * a.k_token + h * a.k_head + d;
    u4 lo, hi;
    if constexpr (Q8) {
      const u4 c = *reinterpret_cast<const u4*>(reinterpret_cast<const uint8_t*>(pool) + in_layer * row + h * D + d);
      const float s = exp_scale((value ? a.c.v_exps : a.c.k_exps)[in_layer / KV_BLOCK * a.c.heads_kv + h]);
      lo = decode8<E>(c[0], c[1], s);
      hi = decode8<E>(c[2], c[3], s);
    } else {
      const u4* from = reinterpret_cast<const u4*>(pool + in_layer * row + h * D + d);
      lo = from[0], hi = from[1];
    }
    u4* out = reinterpret_cast<u4*>(to);
    out[0] = lo;
    out[1] = hi;
  }
}

template <typename E, int D, bool TURN, bool Q8>
hipError_t append(const KvAppendArgs& a, hipStream_t s) {
  constexpr int H = 64 / (D / 16);
  const int all = Q8 ? a.heads : a.heads + 2 * a.c.heads_kv, kv = a.c.heads_kv;
  // heads of a token that one wave takes with the same sines: 2 H, or twice as
  // many where enough waves are left (64 + 16 heads of 128, 16 bits: 256 tokens
  // 5.4 us with 2 H, 5.9 with 4 H, 6.5 with 8 H, 1024 tokens 11.8, 10.5, 10.7,
  // 8192 tokens 69, 65, 67)
  int slice = 4 * H;
  if ((int64_t)a.tokens * ((all + slice - 1) / slice) < 1536) slice = 2 * H;
  const int slices = (all + slice - 1) / slice;
  const int64_t blocks = Q8 ? (int64_t)a.tokens / KV_BLOCK + 2 * (int64_t)a.c.rows : 0;
  // ... and heads of a block (64 heads over 8 of 128: 512 tokens 8.6 us with 1
  // head, 11.4 with 4, 15.6 with 8, 8192 tokens 68, 63, 63)
  int group = 1;
  while (group < 8 && group < kv && blocks * 2 * kv / (2 * group) >= 1024) group *= 2;
  const int64_t waves = (int64_t)a.tokens * slices + blocks * 2 * ((kv + group - 1) / group);
  hipLaunchKernelGGL((kv_append_kernel<E, D, TURN, Q8>), dim3((unsigned)((waves + WAVES - 1) / WAVES)), dim3(64 * WAVES), 0, s,
                     a, slices, slice, group);
  return hipGetLastError();
}
template <typename E, int D>
hipError_t append_d(const KvAppendArgs& a, hipStream_t s) {
  if (a.c.k_exps) return a.rot ? append<E, D, true, true>(a, s) : append<E, D, false, true>(a, s);
  return a.rot ? append<E, D, true, false>(a, s) : append<E, D, false, false>(a, s);
}
template <typename E>
hipError_t append_e(const KvAppendArgs& a, hipStream_t s) {
  return a.c.head_dim == 128 ? append_d<E, 128>(a, s) : append_d<E, 64>(a, s);
}

template <typename E, int D, bool Q8>
hipError_t read(const KvReadArgs& a, hipStream_t s) {
  hipLaunchKernelGGL((kv_read_kernel<E, D, Q8>), dim3((unsigned)((a.tokens + WAVES - 1) / WAVES)), dim3(64 * WAVES), 0, s, a);
  return hipGetLastError();
}
template <typename E>
hipError_t read_e(const KvReadArgs& a, hipStream_t s) {
  if (a.c.k_exps) return a.c.head_dim == 128 ? read<E, 128, true>(a, s) : read<E, 64, true>(a, s);
  return a.c.head_dim == 128 ? read<E, 128, false>(a, s) : read<E, 64, false>(a, s);
}

}  // namespace

hipError_t launch_kv_append(const KvAppendArgs& a, hipStream_t s) {
  return a.bf16 ? append_e<BF16>(a, s) : append_e<F16>(a, s);
}
hipError_t launch_kv_read(const KvReadArgs& a, hipStream_t s) { return a.bf16 ? read_e<BF16>(a, s) : read_e<F16>(a, s); }

}  // namespace qg
