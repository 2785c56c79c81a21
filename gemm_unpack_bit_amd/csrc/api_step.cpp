// C ABI of the norm, ready-row product and sampling calls (qgemv_step.h):
// argument checks and dispatch.  Host-only code; kernels live in norm.hip,
// gemv_w4a8.hip and sample.hip.
#include "qgemv_step.h"

#include <hip/hip_runtime.h>

#include <cmath>
#include <cstdint>

#include "kernels.hpp"
#include "spans.hpp"
#include "step.hpp"

namespace {

using qg::aligned;
using qg::overlap;
using qg::Span;
using qg::span;

constexpr int64_t STRIDE_MAX = (int64_t)1 << 40;
constexpr int DIM_MAX = 1 << 24, VOCAB_MAX = 1 << 21;

hipStream_t stream_of(qgemv_stream_t s) { return reinterpret_cast<hipStream_t>(s); }

// the array with a stride that leads anywhere
qgemv_rows used(const qgemv_rows* x, int rows) { return x ? qgemv_rows{x->data, rows > 1 ? x->row : 0} : qgemv_rows{nullptr, 0}; }
Span span_of(const qgemv_rows& x, int rows, int dim, int elem = 2) {
  return span(x.data, x.data && rows ? elem * ((rows - 1) * x.row + dim) : 0);
}
bool same(const qgemv_rows& a, const qgemv_rows& b) { return a.data == b.data && a.row == b.row; }
int check_rows(const qgemv_rows& x, int rows, int dim, bool output) {
  if (x.row < 0 || x.row > STRIDE_MAX || (double)rows * (double)x.row > 2e18) return QGEMV_ERR_SHAPE;
  return output && rows > 1 && x.row < dim ? QGEMV_ERR_SHAPE : QGEMV_OK;
}

int norm(int dtype, int rows, int dim, float eps, const qgemv_rows* x_, const qgemv_rows* r_, const uint16_t* weight,
         const qgemv_rows* s_, const qgemv_rows* y_, int8_t* y8, float* step, qgemv_stream_t stream) {
  const bool q8 = y_ == nullptr;
  if (!x_ || !x_->data || !weight || (r_ && !r_->data) || (s_ && !s_->data) || !r_ != !s_) return QGEMV_ERR_NULL;
  if (q8 ? !y8 || !step : !y_->data) return QGEMV_ERR_NULL;
  if (dtype != QGEMV_F16 && dtype != QGEMV_BF16) return QGEMV_ERR_UNSUPPORTED;
  if (rows < 0 || dim < 1 || dim > DIM_MAX) return QGEMV_ERR_SHAPE;
  const qgemv_rows x = used(x_, rows), r = used(r_, rows), sum = used(s_, rows), y = used(y_, rows);
  int rc;
  if ((rc = check_rows(x, rows, dim, false)) || (rc = check_rows(r, rows, dim, false)) ||
      (s_ && (rc = check_rows(sum, rows, dim, true))) || (!q8 && (rc = check_rows(y, rows, dim, true))))
    return rc;
  if (!std::isfinite(eps) || eps < 0.f) return QGEMV_ERR_VALUE;
  if (!aligned(x.data, 2) || !aligned(r.data, 2) || !aligned(weight, 2) || !aligned(sum.data, 2) || !aligned(y.data, 2) ||
      !aligned(step, 4))
    return QGEMV_ERR_ALIGN;
  const Span sx = span_of(x, rows, dim), sr = span_of(r, rows, dim), sw = span(weight, (int64_t)2 * dim),
             ss = span_of(sum, rows, dim), sy = q8 ? span(y8, (int64_t)rows * dim) : span_of(y, rows, dim),
             st = span(step, q8 ? (int64_t)4 * rows : 0);
  auto over = [&](const Span& out, const qgemv_rows& o, bool array, const Span& in, const qgemv_rows& i) {
    return overlap(out, in) && !(array && same(o, i));
  };
  if (overlap(ss, sw) || overlap(sy, sw) || overlap(st, sw) || overlap(ss, sy) || overlap(ss, st) || overlap(sy, st) ||
      overlap(st, sx) || overlap(st, sr) || over(ss, sum, true, sx, x) || over(ss, sum, true, sr, r) ||
      over(sy, y, !q8, sx, x) || over(sy, y, !q8, sr, r))
    return QGEMV_ERR_VALUE;
  if (!rows) return QGEMV_OK;
  qg::NormArgs a{};
  a.bf16 = dtype == QGEMV_BF16;
  a.rows = rows;
  a.dim = dim;
  a.eps = eps;
  a.x = x.data, a.x_row = x.row;
  a.residual = r.data, a.residual_row = r.row;
  a.weight = weight;
  a.sum = sum.data, a.sum_row = sum.row;
  a.y = y.data, a.y_row = y.row;
  a.y8 = y8;
  a.step = step;
  auto pieces = [](const qgemv_rows& v) { return aligned(v.data, 16) && v.row % 8 == 0; };
  a.vec = dim % 8 == 0 && pieces(x) && pieces(r) && pieces(sum) && pieces(y) && aligned(weight, 16) && aligned(y8, 8);
  return qg::hip_status(qg::launch_rms_norm(a, stream_of(stream)));
}

}  // namespace

extern "C" {

int qgemv_rms_norm(int dtype, int rows, int dim, float eps, const qgemv_rows* x, const qgemv_rows* residual,
                   const uint16_t* weight, const qgemv_rows* sum, const qgemv_rows* y, qgemv_stream_t stream) {
  if (!y) return QGEMV_ERR_NULL;
  return norm(dtype, rows, dim, eps, x, residual, weight, sum, y, nullptr, nullptr, stream);
}

int qgemv_rms_norm_q8(int dtype, int rows, int dim, float eps, const qgemv_rows* x, const qgemv_rows* residual,
                      const uint16_t* weight, const qgemv_rows* sum, int8_t* y8, float* step, qgemv_stream_t stream) {
  return norm(dtype, rows, dim, eps, x, residual, weight, sum, nullptr, y8, step, stream);
}

size_t qgemv_sample_workspace_bytes(int rows, int vocab) {
  if (rows < 1 || vocab < 1 || vocab > VOCAB_MAX || !qg::sample_fits(rows, vocab)) return 0;
  return qg::sample_ws_bytes(rows, vocab);
}

int qgemv_sample(int type, int rows, int vocab, const void* logits, int64_t row, const float* u, const float* temperature,
                 const int32_t* top_k, const float* top_p, const float* min_p, int32_t* token, void* ws, size_t ws_bytes,
                 qgemv_stream_t stream) {
  if (!logits || !u || !token) return QGEMV_ERR_NULL;
  if (type != QGEMV_F16 && type != QGEMV_BF16 && type != QGEMV_F32) return QGEMV_ERR_UNSUPPORTED;
  if (rows < 0 || vocab < 1 || vocab > VOCAB_MAX) return QGEMV_ERR_SHAPE;
  if (!rows) return QGEMV_OK;
  if (!qg::sample_fits(rows, vocab)) return QGEMV_ERR_SHAPE;
  const int64_t stride = rows > 1 ? row : 0, elem = type == QGEMV_F32 ? 4 : 2;
  if (stride < 0 || stride > STRIDE_MAX || (double)rows * (double)stride > 2e17) return QGEMV_ERR_SHAPE;
  if (!aligned(logits, elem) || !aligned(u, 4) || !aligned(temperature, 4) || !aligned(top_k, 4) || !aligned(top_p, 4) ||
      !aligned(min_p, 4) || !aligned(token, 4))
    return QGEMV_ERR_ALIGN;
  const size_t need = qg::sample_ws_bytes(rows, vocab);
  const int64_t each = (int64_t)4 * rows;
  const Span st = span(token, each), sw = span(ws, ws ? (int64_t)need : 0);
  const Span in[] = {span(logits, elem * ((rows - 1) * stride + vocab)), span(u, each), span(temperature, temperature ? each : 0),
                     span(top_k, top_k ? each : 0), span(top_p, top_p ? each : 0), span(min_p, min_p ? each : 0)};
  for (const Span& x : in)
    if (overlap(st, x) || overlap(sw, x)) return QGEMV_ERR_VALUE;
  if (overlap(st, sw)) return QGEMV_ERR_VALUE;
  if (!ws || ws_bytes < need) return QGEMV_ERR_WORKSPACE;
  if (!aligned(ws, 16)) return QGEMV_ERR_ALIGN;
  qg::SampleArgs a{type, rows, vocab, logits, stride * elem, u, temperature, top_k, top_p, min_p, token, ws};
  return qg::hip_status(qg::launch_sample(a, stream_of(stream)));
}

}  // extern "C"
