// Root-mean-square norm of rows, with the residual's addition, and the result
// in 16 bits or in 8 bits with a scale per row.
//
// Mathematics.  h = x + r, y = h w / sqrt(sum h^2 / dim + eps); in 8 bits
// step = max |y| / 127, code = rint(y / step).
//
// Bound: memory (8 bytes an element with a residual), or for few rows the
// launch and two trips through the row's reduction.  A row is read once: WAVES
// waves hold it in registers as fp32 sums, HELD pieces of 8 elements a thread;
// what does not fit is read again in each later pass (nothing is written
// before the last one, so that outputs may take an input's place).  Two pieces
// a thread leave room for six waves a SIMD; with four, 5003 rows of 8192 took 72
// us instead of 66, and the 8-bit form for 16 waves did not fit its registers.
//
// Measured (bf16 or fp16, with a residual): 5003 rows of 8192 66 us (328 MB, 5.0
// TB/s, as a large copy), in 8 bits 68 us (287 MB), one row of 4096 3.2 us.  Outputs past the caches
// (non-temporal) took 62 us, but what reads them next lost that again.
#include "attn_common.hpp"
#include "step.hpp"

namespace qg {
namespace {

constexpr int HELD = 2;

__device__ __forceinline__ float wave_sum(float v) { return quarter_sum(group_sum<16>(v)); }
__device__ __forceinline__ float wave_max(float v) {
  v = fmaxf(v, dpp<DPP_QP_XOR1>(v));
  v = fmaxf(v, dpp<DPP_QP_XOR2>(v));
  v = fmaxf(v, dpp<DPP_ROR4>(v));
  v = fmaxf(v, dpp<DPP_ROR8>(v));
  return quarter_max(v);
}

__device__ __forceinline__ bool finite(float v) { return (__float_as_uint(v) & 0x7F800000u) != 0x7F800000u; }

__device__ __forceinline__ uint32_t low_bytes(uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
  return __builtin_amdgcn_perm(__builtin_amdgcn_perm(d, c, 0x0C0C0400u), __builtin_amdgcn_perm(b, a, 0x0C0C0400u), 0x05040100u);
}

// PW: elements of a piece, 8 (one 16-byte access) or 1 (any alignment).
// A workgroup has 16 waves or fewer: one row (WAVES > 1) or four (WAVES = 1).
template <typename E, int PW, int WAVES, bool Q8>
__global__ void __launch_bounds__(WAVES == 1 ? 256 : 64 * WAVES) rms_norm_kernel(NormArgs a) {
  constexpr int T = 64 * WAVES;
  constexpr int ROWS = WAVES == 1 ? 4 : 1;  // of a workgroup
  __shared__ float red[2][WAVES];
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int tid = WAVES == 1 ? lane : threadIdx.x;
  const int pieces = (a.dim + PW - 1) / PW;

  typedef uint32_t raw __attribute__((ext_vector_type(4)));
  auto load = [&](const uint16_t* p, int piece, float (&v)[PW]) {
    if constexpr (PW == 8) {
      const raw w = *reinterpret_cast<const raw*>(p + 8 * (int64_t)piece);
#pragma unroll
      for (int e = 0; e < 8; ++e) v[e] = E::value((uint16_t)(w[e / 2] >> (16 * (e & 1))));
    } else {
      v[0] = E::value(p[piece]);
    }
  };
  auto store = [&](uint16_t* p, int piece, const float (&v)[PW]) {
    if constexpr (PW == 8) {
      *reinterpret_cast<raw*>(p + 8 * (int64_t)piece) =
          raw{E::pack(v[0], v[1]), E::pack(v[2], v[3]), E::pack(v[4], v[5]), E::pack(v[6], v[7])};
    } else {
      p[piece] = (uint16_t)E::pack(v[0], 0.f);
    }
  };
  // a value of every wave of the row joined by f (in wave order)
  auto join = [&](float v, int which, auto f) {
    if constexpr (WAVES == 1) return v;
    if (lane == 0) red[which][wave] = v;
    __syncthreads();
    float r = red[which][0];
#pragma unroll
    for (int w = 1; w < WAVES; ++w) r = f(r, red[which][w]);
    return r;
  };

  for (int64_t row = (int64_t)blockIdx.x * ROWS + (WAVES == 1 ? wave : 0); row < a.rows; row += (int64_t)gridDim.x * ROWS) {
    const uint16_t* x = a.x + row * a.x_row;
    const uint16_t* r = a.residual ? a.residual + row * a.residual_row : nullptr;
    auto take = [&](int piece, float (&h)[PW]) {
      load(x, piece, h);
      if (r) {
        float y[PW];
        load(r, piece, y);
#pragma unroll
        for (int e = 0; e < PW; ++e) h[e] += y[e];
      }
    };
    float h[HELD][PW], w[HELD][PW];
#pragma unroll
    for (int i = 0; i < HELD; ++i)
      if (tid + T * i < pieces) take(tid + T * i, h[i]);
    // (the weights are on their way during the reduction)
#pragma unroll
    for (int i = 0; i < HELD; ++i)
      if (tid + T * i < pieces) load(a.weight, tid + T * i, w[i]);
    float sum = 0.f;
#pragma unroll
    for (int i = 0; i < HELD; ++i)
      if (tid + T * i < pieces)
#pragma unroll
        for (int e = 0; e < PW; ++e) sum = fmaf(h[i][e], h[i][e], sum);
    for (int p = tid + T * HELD; p < pieces; p += T) {
      float y[PW];
      take(p, y);
#pragma unroll
      for (int e = 0; e < PW; ++e) sum = fmaf(y[e], y[e], sum);
    }
    sum = join(wave_sum(sum), 0, [](float p, float q) { return p + q; });
    const float inv = 1.f / __builtin_sqrtf(sum / (float)a.dim + a.eps);

    float step = 0.f;
    if constexpr (Q8) {
      // (as whole numbers, magnitudes order alike, and infinities and NaN stand
      // above them all)
      uint32_t top = 0;
      auto look = [&](const float (&v)[PW], const float (&wt)[PW]) {
#pragma unroll
        for (int e = 0; e < PW; ++e) top = max(top, __float_as_uint(v[e] * inv * wt[e]) & 0x7FFFFFFFu);
      };
#pragma unroll
      for (int i = 0; i < HELD; ++i)
        if (tid + T * i < pieces) look(h[i], w[i]);
      for (int p = tid + T * HELD; p < pieces; p += T) {
        float y[PW], wt[PW];
        take(p, y);
        load(a.weight, p, wt);
        look(y, wt);
      }
      float most = wave_max(__uint_as_float(min(top, 0x7F800000u)));
      most = join(most, 1, [](float p, float q) { return fmaxf(p, q); });
      step = most / 127.0f;  // correctly rounded
      if (!finite(most)) step = __builtin_nanf("");
      if (tid == 0) a.step[row] = step;
    }
    // 1 / step, where the quotients below can be had from it
    const float by = Q8 && step > 0x1p-100f && step < 0x1p100f ? 1.f / step : 0.f;

    auto finish = [&](int piece, float (&v)[PW], const float (&wt)[PW]) {
      if (a.sum) store(a.sum + row * a.sum_row, piece, v);
#pragma unroll
      for (int e = 0; e < PW; ++e) v[e] = v[e] * inv * wt[e];
      if constexpr (Q8) {
        // y / step correctly rounded, so codes are those of the definition.  The
        // product with the correctly rounded reciprocal, corrected by its remainder,
        // is one of the quotient's two neighbours, and corrected once more its
        // rounding (Markstein's theorem; where a remainder would be subnormal, the
        // code is 0 with any rounding).  Adding 1.5 * 2^23 rounds to a whole number,
        // which then stands in the low byte.
        uint32_t c[PW];
        if (by != 0.f) {
#pragma unroll
          for (int e = 0; e < PW; ++e) {
            const float q = v[e] * by, near = fmaf(fmaf(-q, step, v[e]), by, q),
                        exact = fmaf(fmaf(-near, step, v[e]), by, near);
            c[e] = __float_as_uint(fminf(fmaxf(exact, -127.f), 127.f) + 12582912.f);
          }
        } else {
#pragma unroll
          for (int e = 0; e < PW; ++e)
            c[e] = step > 0.f ? (uint32_t)(int)rintf(fminf(fmaxf(v[e] / step, -127.f), 127.f)) : 0u;
        }
        int8_t* to = a.y8 + row * a.dim + (int64_t)piece * PW;
        if constexpr (PW == 8)
          *reinterpret_cast<u2*>(to) = u2{low_bytes(c[0], c[1], c[2], c[3]), low_bytes(c[4], c[5], c[6], c[7])};
        else
          *to = (int8_t)c[0];
      } else {
        store(a.y + row * a.y_row, piece, v);
      }
    };
#pragma unroll
    for (int i = 0; i < HELD; ++i)
      if (tid + T * i < pieces) finish(tid + T * i, h[i], w[i]);
    for (int p = tid + T * HELD; p < pieces; p += T) {
      float y[PW], wt[PW];
      take(p, y);
      load(a.weight, p, wt);
      finish(p, y, wt);
    }
    if constexpr (WAVES > 1) __syncthreads();  // `red` is free for the next row
  }
}

template <typename E, int PW, int WAVES, bool Q8>
hipError_t launch(const NormArgs& a, hipStream_t s) {
  constexpr int ROWS = WAVES == 1 ? 4 : 1;
  const int64_t groups = ((int64_t)a.rows + ROWS - 1) / ROWS;
  // (a launch stays under 2^32 threads; past it workgroups take several rows)
  hipLaunchKernelGGL((rms_norm_kernel<E, PW, WAVES, Q8>), dim3((unsigned)(groups < 1 << 20 ? groups : 1 << 20)),
                     dim3(WAVES == 1 ? 256 : 64 * WAVES), 0, s, a);
  return hipGetLastError();
}

template <typename E, int PW, bool Q8>
hipError_t launch_w(const NormArgs& a, hipStream_t s) {
  const int pieces = (a.dim + PW - 1) / PW;
  // Measured (fp16, with a residual, 16-bit results): 4096 rows of 1024 8.8 us with
  // one wave and 10.8 with 4, 128 rows 3.8 and 3.4; of 2048 13.8 with 4 and 16.8
  // with 8; of 4096 30 with either, one row 3.7 and 3.5; of 8192 56 with 8, 63 with
  // 4, 58 with 16; of 16384 114 with 8 and 106 with 16.
  if (pieces <= 128 && a.rows > 512) return launch<E, PW, 1, Q8>(a, s);
  if (pieces <= 256) return launch<E, PW, 4, Q8>(a, s);
  if (pieces <= 1024) return launch<E, PW, 8, Q8>(a, s);
  return launch<E, PW, 16, Q8>(a, s);
}

template <typename E, int PW>
hipError_t launch_q(const NormArgs& a, hipStream_t s) {
  return a.y8 ? launch_w<E, PW, true>(a, s) : launch_w<E, PW, false>(a, s);
}

template <typename E>
hipError_t launch_e(const NormArgs& a, hipStream_t s) {
  return a.vec ? launch_q<E, 8>(a, s) : launch_q<E, 1>(a, s);
}

}  // namespace

hipError_t launch_rms_norm(const NormArgs& a, hipStream_t s) { return a.bf16 ? launch_e<BF16>(a, s) : launch_e<F16>(a, s); }

}  // namespace qg
