// Host side of the gated feed-forward block with 8-bit weights (include/mscl.h).
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

namespace {

using namespace mscl;
using namespace mscl::launch;

mscl_status_t check_gated_int8(const mscl_gated_linear_quantized_t* c, Spans& s) {
  if (!c) return bad("call is null");
  mscl_status_t st = check_kinds(c->dtype, c->activation);
  if (st == MSCL_SUCCESS) st = check_sizes(c->rows, c->in_features, c->out_features);
  if (st == MSCL_SUCCESS) st = check_reach_of_sums(c->in_features);
  if (st != MSCL_SUCCESS) return st;
  const size_t e = bytes_of(c->dtype), m = c->rows, k = c->in_features, n = c->out_features;
  s.add("x", c->x, m, k, c->x_stride, 1, false, n != 0);
  s.add("x_scale", c->x_scale, 1, m, 0, 4, false, n != 0);
  s.add("gate_w", c->gate_w, n, k, c->gate_w_stride, 1, false, m != 0);
  s.add("gate_scale", c->gate_scale, 1, n, 0, 4, false, m != 0);
  s.add("up_w", c->up_w, n, k, c->up_w_stride, 1, false, m != 0);
  s.add("up_scale", c->up_scale, 1, n, 0, 4, false, m != 0);
  s.add("gate_bias", c->gate_bias, 1, n, 0, e, false, false);
  s.add("up_bias", c->up_bias, 1, n, 0, e, false, false);
  s.add("y", c->y, m, n, c->y_stride, e, true, true);
  return s.check();
}

PairOperand weights_of(const mscl_gated_linear_quantized_t& c) {
  return pair_of(c.gate_w, c.gate_w_stride, c.up_w, c.up_w_stride, c.out_features, c.in_features);
}
ForwardPlan plan_gated_int8(const mscl_gated_linear_quantized_t& c) {
  return plan_forward(operand(c.x, c.x_stride, c.rows, c.in_features), weights_of(c).half, 2, c.rows, c.out_features,
                      c.in_features, 1);
}

}  // namespace

extern "C" {

mscl_status_t mscl_gated_linear_quantized_workspace(const mscl_gated_linear_quantized_t* call, size_t* bytes) {
  if (!bytes) return bad("bytes is null");
  Spans spans;
  const mscl_status_t st = check_gated_int8(call, spans);
  if (st != MSCL_SUCCESS) return st;
  *bytes = 0;
  if (call->rows == 0 || call->out_features == 0) return MSCL_SUCCESS;
  const ForwardPlan p = plan_gated_int8(*call);
  *bytes = p.bytes;
  return check_threads(threads_of(p, call->rows, call->out_features, bytes_of(call->dtype)));
}

mscl_status_t mscl_gated_linear_quantized(const mscl_gated_linear_quantized_t* call, void* workspace, size_t workspace_bytes,
                                     void* stream) {
  Spans spans;
  mscl_status_t st = check_gated_int8(call, spans);
  if (st != MSCL_SUCCESS) return st;
  const mscl_gated_linear_quantized_t& c = *call;
  if (c.rows == 0 || c.out_features == 0) return MSCL_SUCCESS;
  const ForwardPlan p = plan_gated_int8(c);
  if ((st = check_threads(threads_of(p, c.rows, c.out_features, bytes_of(c.dtype)))) != MSCL_SUCCESS) return st;
  if ((st = spans.check_workspace(workspace, workspace_bytes, p.bytes)) != MSCL_SUCCESS) return st;
  int cus = 0;
  if ((st = current_device(&cus)) != MSCL_SUCCESS) return st;
  return with_codec(c.dtype, [&](auto t) {
    Gated<decltype(t)> e;
    memset(&e, 0, sizeof e);
    e.bias[0] = bytes_at(c.gate_bias);
    e.bias[1] = bytes_at(c.up_bias);
    e.y = bytes_at(c.y);
    e.y_stride = c.y_stride;
    e.m = c.rows;
    e.n = c.out_features;
    e.act = c.activation;
    e.row_scale = c.x_scale;
    e.col_scale[0] = c.gate_scale;
    e.col_scale[1] = c.up_scale;
    return forward<I8>(p, operand(c.x, c.x_stride, c.rows, c.in_features), weights_of(c), c.in_features, e,
                       bytes_at(workspace), static_cast<hipStream_t>(stream));
  });
}

}  // extern "C"
