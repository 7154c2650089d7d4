// Host side of the rows' quantization and of the 8-bit product (include/mscl.h).
// Every entry point returns a status code; nothing here aborts or allocates.

#include <hip/hip_runtime.h>
#include <stdint.h>
#include <string.h>

#include <algorithm>

#include "../../include/mscl.h"
#include "failure.hpp"
#include "feedforward.hpp"
#include "forward.hpp"
#include "launch.hpp"
#include "linear.hpp"
#include "quantize.hpp"

namespace {

using namespace mscl;
using namespace mscl::launch;

mscl_status_t check_linear_quantized(const mscl_linear_quantized_t* c, Spans& s) {
  if (!c) return bad("call is null");
  mscl_status_t st = check_kinds(c->dtype, c->activation);
  if (st == MSCL_SUCCESS) st = check_sizes(c->rows, c->in_features, c->out_features);
  if (st == MSCL_SUCCESS) st = check_reach_of_sums(c->in_features);
  if (st != MSCL_SUCCESS) return st;
  const size_t e = bytes_of(c->dtype), m = c->rows, k = c->in_features, n = c->out_features;
  s.add("x", c->x, m, k, c->x_stride, 1, false, n != 0);
  s.add("x_scale", c->x_scale, 1, m, 0, 4, false, n != 0);
  s.add("w", c->w, n, k, c->w_stride, 1, false, m != 0);
  s.add("w_scale", c->w_scale, 1, n, 0, 4, false, m != 0);
  s.add("bias", c->bias, 1, n, 0, e, false, false);
  s.add("residual", c->residual, m, n, c->residual_stride, e, false, false);
  s.add("y", c->y, m, n, c->y_stride, e, true, true, "residual");
  return s.check();
}

ForwardPlan plan_linear_quantized(const mscl_linear_quantized_t& c) {
  const Operand w = operand(c.w, c.w_stride, c.out_features, c.in_features);
  return plan_forward(operand(c.x, c.x_stride, c.rows, c.in_features), &w, 1, c.rows, c.out_features, c.in_features, 1);
}

// ------------------------------------------------------------------ rows to 8 bits

// 16 elements a thread and chunk.  Few rows want the shortest way through a
// row, one chunk a thread; many rows want few threads with several in flight.
template <class C>
void launch_quantize(const QuantizeArgs& a, hipStream_t s) {
  const uint64_t chunks = ceil_div(a.width, 16);
  const uint32_t rows = static_cast<uint32_t>(a.rows), quads = static_cast<uint32_t>(ceil_div(a.rows, 4));
  if (chunks <= 64) return quantize_rows<C, 64, 1><<<quads, 256, 0, s>>>(a);
  if (a.rows <= 2 * kCus) {
    if (chunks <= 256) return quantize_rows<C, 256, 1><<<rows, 256, 0, s>>>(a);
    if (chunks <= 512) return quantize_rows<C, 512, 1><<<rows, 512, 0, s>>>(a);
    if (chunks <= 1024) return quantize_rows<C, 1024, 1><<<rows, 1024, 0, s>>>(a);
  }
  if (chunks <= 128) return quantize_rows<C, 64, 2><<<quads, 256, 0, s>>>(a);
  if (chunks <= 256) return quantize_rows<C, 256, 1><<<rows, 256, 0, s>>>(a);
  if (chunks <= 512) return quantize_rows<C, 256, 2><<<rows, 256, 0, s>>>(a);
  if (chunks <= 1024) return quantize_rows<C, 256, 4><<<rows, 256, 0, s>>>(a);
  if (chunks <= 2048) return quantize_rows<C, 512, 4><<<rows, 512, 0, s>>>(a);
  quantize_wide<C><<<rows, 1024, 0, s>>>(a);
}

mscl_status_t check_quantize(const mscl_quantize_t* c, Spans& s) {
  if (!c) return bad("call is null");
  if (!known_dtype(c->dtype)) return bad("unknown dtype");
  if (c->width == 0) return bad("width must be at least 1");
  if (c->rows > kMostGroups) return bad("too many rows");
  s.add("x", c->x, c->rows, c->width, c->x_stride, bytes_of(c->dtype), false, true);
  s.add("q", c->q, c->rows, c->width, c->q_stride, 1, true, true);
  s.add("scale", c->scale, 1, c->rows, 0, 4, true, true);
  return s.check();
}

}  // namespace

namespace mscl {
namespace launch {

mscl_status_t pack_int8(Operand* o, char* to, hipStream_t stream) {
  const PackArgs a{o->base, to, o->stride, packed_stride(o->cols), o->rows, o->cols};
  const uint64_t groups = std::min<uint64_t>(ceil_div(ceil_div(o->cols, 16) * o->rows, 256), 16 * kCus);
  linear_pack<I8><<<static_cast<uint32_t>(groups), 256, 0, stream>>>(a);
  *o = Operand{to, a.to_stride, o->rows, round_up(o->cols, 16)};
  return launched("linear_pack");
}

}  // namespace launch
}  // namespace mscl

extern "C" {

mscl_status_t mscl_quantize(const mscl_quantize_t* call, void* stream) {
  Spans spans;
  mscl_status_t st = check_quantize(call, spans);
  if (st != MSCL_SUCCESS) return st;
  const mscl_quantize_t& c = *call;
  if (c.rows == 0) return MSCL_SUCCESS;
  int cus = 0;
  if ((st = current_device(&cus)) != MSCL_SUCCESS) return st;
  // a launch has fewer than 2^32 threads, up to 1024 of them a row
  constexpr size_t kRowsOfLaunch = size_t(1) << 21;
  for (size_t first = 0; first < c.rows && st == MSCL_SUCCESS; first += kRowsOfLaunch) {
    const size_t rows = std::min(kRowsOfLaunch, c.rows - first);
    const QuantizeArgs a{bytes_at(c.x) + first * c.x_stride * bytes_of(c.dtype), c.q + first * c.q_stride, c.scale + first,
                         c.x_stride, c.q_stride, rows, c.width};
    st = with_codec(c.dtype, [&](auto t) {
      launch_quantize<decltype(t)>(a, static_cast<hipStream_t>(stream));
      return launched("quantize_rows");
    });
  }
  return st;
}

mscl_status_t mscl_linear_quantized_workspace(const mscl_linear_quantized_t* call, size_t* bytes) {
  if (!bytes) return bad("bytes is null");
  Spans spans;
  const mscl_status_t st = check_linear_quantized(call, spans);
  if (st != MSCL_SUCCESS) return st;
  *bytes = 0;
  if (call->rows == 0 || call->out_features == 0) return MSCL_SUCCESS;
  const ForwardPlan p = plan_linear_quantized(*call);
  *bytes = p.bytes;
  return check_threads(threads_of(p, call->rows, call->out_features, bytes_of(call->dtype)));
}

mscl_status_t mscl_linear_quantized(const mscl_linear_quantized_t* call, void* workspace, size_t workspace_bytes, void* stream) {
  Spans spans;
  mscl_status_t st = check_linear_quantized(call, spans);
  if (st != MSCL_SUCCESS) return st;
  const mscl_linear_quantized_t& c = *call;
  if (c.rows == 0 || c.out_features == 0) return MSCL_SUCCESS;
  const ForwardPlan p = plan_linear_quantized(c);
  if ((st = check_threads(threads_of(p, c.rows, c.out_features, bytes_of(c.dtype)))) != MSCL_SUCCESS) return st;
  if ((st = spans.check_workspace(workspace, workspace_bytes, p.bytes)) != MSCL_SUCCESS) return st;
  int cus = 0;
  if ((st = current_device(&cus)) != MSCL_SUCCESS) return st;
  return with_codec(c.dtype, [&](auto t) {
    Scaled<decltype(t)> e;
    memset(static_cast<void*>(&e), 0, sizeof e);
    e.bias = bytes_at(c.bias);
    e.residual = bytes_at(c.residual);
    e.residual_stride = c.residual_stride;
    e.y = bytes_at(c.y);
    e.y_stride = c.y_stride;
    e.m = c.rows;
    e.n = c.out_features;
    e.act = c.activation;
    e.row_scale = c.x_scale;
    e.col_scale = c.w_scale;
    return forward<I8>(p, operand(c.x, c.x_stride, c.rows, c.in_features),
                       operand(c.w, c.w_stride, c.out_features, c.in_features), c.in_features, e, bytes_at(workspace),
                       static_cast<hipStream_t>(stream));
  });
}

}  // extern "C"
