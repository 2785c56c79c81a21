// Internal interface of the norm and sampling kernels (api_step.cpp calls the
// launchers; norm.hip and sample.hip hold the kernels).
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace qg {

struct NormArgs {
  int bf16, rows, dim;
  float eps;
  const uint16_t *x, *residual, *weight;
  uint16_t *sum, *y;
  int8_t* y8;   // 8-bit result ...
  float* step;  // ... and its row scales, or NULL
  int64_t x_row, residual_row, sum_row, y_row;
  int vec;  // every array can be taken in 16-byte pieces (y8 in 8-byte ones)
};
hipError_t launch_rms_norm(const NormArgs& a, hipStream_t s);

struct SampleArgs {
  int type;  // of the logits: 0 fp16, 1 bf16, 2 fp32
  int rows, vocab;
  const void* logits;
  int64_t row_bytes;
  const float *u, *temperature;
  const int32_t* top_k;
  const float *top_p, *min_p;  // (each of the settings may be NULL)
  int32_t* out;
  void* ws;
};
bool sample_fits(int rows, int vocab);  // launches stay in range
size_t sample_ws_bytes(int rows, int vocab);
hipError_t launch_sample(const SampleArgs& a, hipStream_t s);

}  // namespace qg
