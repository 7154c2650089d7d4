// Host side of the gated feed-forward block, forward and backward
// (include/mscl.h).  Every entry point returns a status code; nothing here
// aborts or allocates.

#include <hip/hip_runtime.h>
#include <stdint.h>
#include <string.h>

#include <algorithm>

#include "../../include/mscl.h"
#include "failure.hpp"
#include "feedforward.hpp"
#include "forward.hpp"
#include "gated.hpp"
#include "launch.hpp"
#include "linear.hpp"

namespace {

using namespace mscl;
using namespace mscl::launch;

mscl_status_t check_gated(const mscl_gated_linear_t* c, Spans& s) {
  if (!c) return bad("call is null");
  mscl_status_t st = check_kinds(c->dtype, c->activation);
  if (st == MSCL_SUCCESS) st = check_sizes(c->rows, c->in_features, c->out_features);
  if (st != MSCL_SUCCESS) return st;
  const size_t e = bytes_of(c->dtype), m = c->rows, k = c->in_features, n = c->out_features;
  s.add("x", c->x, m, k, c->x_stride, e, false, n != 0);
  s.add("gate_w", c->gate_w, n, k, c->gate_w_stride, e, false, m != 0);
  s.add("up_w", c->up_w, n, k, c->up_w_stride, e, false, m != 0);
  s.add("gate_bias", c->gate_bias, 1, n, 0, e, false, false);
  s.add("up_bias", c->up_bias, 1, n, 0, e, false, false);
  s.add("y", c->y, m, n, c->y_stride, e, true, true);
  s.add("gate", c->gate, m, n, c->gate_stride, e, true, false);
  s.add("up", c->up, m, n, c->up_stride, e, true, false);
  return s.check();
}

PairOperand weights_of(const mscl_gated_linear_t& c) {
  return pair_of(c.gate_w, c.gate_w_stride, c.up_w, c.up_w_stride, c.out_features, c.in_features);
}
// A binary32 operand's parts in a workspace.
size_t part_bytes(const Operand& o) { return packed_bytes(o); }
Operand parts_at(const Operand& o, const char* at) {
  return Operand{at, packed_stride(o.cols), o.rows, round_up(o.cols, 8)};
}
mscl_status_t split_operand(const Operand& o, char* to, hipStream_t s) {
  const SplitArgs a{o, to, packed_stride(o.cols), part_bytes(o)};
  const uint64_t groups = std::min<uint64_t>(ceil_div(ceil_div(o.cols, 8) * o.rows, 256), 16 * kCus);
  split_parts<<<static_cast<uint32_t>(groups), 256, 0, s>>>(a);
  return launched("split_parts");
}
// How a product of binary32 operands in parts runs, if at all.  Its tiles of
// 256 x 256 take 6 x 1.4 us a block of k whether or not they fill the device, so
// k is split where they would leave much of it idle, and the shares' sums (and
// the parts themselves, 10 bytes a value) are a pass over memory at 5 TB/s.
// forward_tile, which takes operands into parts in every tile, reaches 130 to 165
// TFLOP/s.  Forward, us by parts and by those tiles: 1024 x 4096 -> 4096
// 376 and 509, 2048 x 2048 -> 2048 203 and 260, 512 x 4096 -> 4096 249 and 205.
struct PartsPlan {
  bool on = false;
  uint32_t blocks = 0, blocks_per_share = 0, shares = 1;
  uint64_t partial_stride = 0;
  size_t partial_bytes = 0;  // of one product
};

// `products` of m x n with `blocks` blocks of k each, from `values` values of
// operands; `flops` in all.
PartsPlan plan_parts(int dtype, uint64_t tiles, uint64_t products, uint64_t m, uint64_t n, uint64_t blocks, double values,
                     double flops, uint64_t a_stride, uint64_t b_stride) {
  PartsPlan p;
  const uint64_t limit = uint64_t(1) << 22;  // elements of 2 bytes within a tile's 31-bit offsets
  if (dtype != MSCL_FLOAT32 || a_stride >= limit || b_stride >= limit || blocks < 4 || blocks >= (1u << 24)) return p;
  double best = flops / 160e6;  // us
  for (uint64_t shares = 1; shares <= 8 && 4 * shares <= blocks; ++shares) {
    const uint64_t per = ceil_div(blocks, shares);
    if (ceil_div(blocks, per) != shares) continue;
    double us = static_cast<double>(ceil_div(tiles * products * shares, kCus)) * per * 6 * 1.4 + values * 10 / 5e6 + 8;
    if (shares > 1) us += 8.0 * shares * products * m * n / 5e6 + 4;
    if (us >= best) continue;
    best = us;
    p.on = true;
    p.shares = static_cast<uint32_t>(shares);
    p.blocks_per_share = static_cast<uint32_t>(per);
  }
  p.blocks = static_cast<uint32_t>(blocks);
  p.partial_stride = round_up(n, 8);
  if (p.on && p.shares > 1) p.partial_bytes = round_up(p.shares * m * p.partial_stride * 4, 256);
  return p;
}

struct GatedPlan {
  PartsPlan parts;
  ForwardPlan tiles;
  size_t a_part = 0, b_part = 0;  // bytes of one part of x, of a weight
  size_t bytes = 0;
};

GatedPlan plan_gated(const mscl_gated_linear_t& c) {
  GatedPlan p;
  const Operand x = operand(c.x, c.x_stride, c.rows, c.in_features);
  const PairOperand w = weights_of(c);
  const uint64_t stride = packed_stride(c.in_features);
  const double m = c.rows, k = c.in_features, n = c.out_features;
  p.parts = plan_parts(c.dtype, ceil_div(c.rows, 256) * ceil_div(c.out_features, 128), 1, c.rows, 2 * c.out_features,
                       ceil_div(c.in_features, 64), (m + 2 * n) * k, 4 * m * n * k, stride, stride);
  if (p.parts.on) {
    p.a_part = part_bytes(x);
    p.b_part = part_bytes(w.half[0]);
    p.parts.partial_stride = 2 * round_up(c.out_features, 8);
    if (p.parts.shares > 1)
      p.parts.partial_bytes = round_up(p.parts.shares * c.rows * p.parts.partial_stride * 4, 256);
    p.bytes = 3 * p.a_part + 6 * p.b_part + p.parts.partial_bytes;
    return p;
  }
  p.tiles = plan_forward(x, w.half, 2, c.rows, c.out_features, c.in_features, bytes_of(c.dtype));
  p.bytes = p.tiles.bytes;
  return p;
}

double threads_of(const GatedPlan& p, const mscl_gated_linear_t& c) {
  if (!p.parts.on) return threads_of(p.tiles, c.rows, c.out_features, bytes_of(c.dtype));
  const double tiles = static_cast<double>(ceil_div(c.rows, 256)) * ceil_div(c.out_features, 128) * p.parts.shares;
  return std::max(512 * tiles, join_threads(c.rows, c.out_features, 4));
}

mscl_status_t gated_by_parts(const GatedPlan& p, const mscl_gated_linear_t& c, Gated<F32> e, char* ws, hipStream_t s) {
  const Operand x = operand(c.x, c.x_stride, c.rows, c.in_features);
  const PairOperand w = weights_of(c);
  char* w_at = ws + 3 * p.a_part;
  mscl_status_t st = split_operand(x, ws, s);
  for (int h = 0; h < 2 && st == MSCL_SUCCESS; ++h) st = split_operand(w.half[h], w_at + 3 * h * p.b_part, s);
  if (st != MSCL_SUCCESS) return st;
  const uint64_t tm = ceil_div(c.rows, 256), tn = ceil_div(c.out_features, 128);
  const hipError_t err = allow_lds<&gated_parts_big>(kBigLds);
  if (err != hipSuccess) return failed_hip(err, "hipFuncSetAttribute");
  if (p.parts.shares > 1) e.partial = reinterpret_cast<float*>(w_at + 6 * p.b_part);
  e.partial_stride = p.parts.partial_stride;
  GatedPartsArgs a;
  a.parts = {parts_at(x, ws), PairOperand{{parts_at(w.half[0], w_at), parts_at(w.half[1], w_at + 3 * p.b_part)}}, e,
             round_up(c.in_features, 8), static_cast<uint32_t>(tm), static_cast<uint32_t>(tn)};
  a.of = {p.a_part, p.b_part, p.parts.blocks, p.parts.blocks_per_share};
  a.a = x;
  a.b = w;
  a.k = c.in_features;
  gated_parts_big<<<static_cast<uint32_t>(tm * tn * p.parts.shares), 512, kBigLds, s>>>(a);
  st = launched("gated_parts_big");
  return st != MSCL_SUCCESS || p.parts.shares == 1 ? st : join_forward<F32>(e, p.parts.shares, s);
}

// ------------------------------------------------------------------ backward pass

// Parts of a backward call's workspace, each from a 256-byte boundary.
struct GatedBackwardPlan {
  uint64_t half = 0;     // columns of dz and of dv in the workspace
  bool products = false; // dx or a weight's gradient is wanted
  bool dx_big = false, pack_w = false, dw_big = false;
  ProductPlan dx, dw;    // dx as tiles: of one weight's half
  uint32_t groups = 0, rows_per_group = 0;  // of the bias gradients' partial sums
  PairOperand w;
  Operand x;
  size_t w_bytes = 0;    // of one weight laid out anew, or of one part of it
  // large binary32 products: bytes of one part of d and of x
  bool parts = false;
  PartsPlan dx_parts, dw_parts;
  size_t d_part = 0, x_part = 0;
  size_t d_at = 0, sums_at = 0, parts_at = 0, dx_at = 0, dw_at = 0, bytes = 0;
};

// Two shares of the blocks of k of a product m x n.
void halve(ProductPlan* p, uint64_t m, uint64_t n, uint64_t blocks) {
  p->shares = 2;
  p->blocks_per_share = static_cast<uint32_t>(ceil_div(blocks, 2));
  p->partial_stride = round_up(n, 8);
  p->partial_bytes = round_up(2 * m * p->partial_stride * 4, 256);
}

GatedBackwardPlan plan_gated_backward(const mscl_gated_linear_backward_t& c) {
  GatedBackwardPlan p;
  const size_t e = bytes_of(c.dtype);
  const uint64_t m = c.rows, k = c.in_features, n = c.out_features;
  const bool want_dw = c.dgate_w || c.dup_w;
  const size_t dws = (c.dgate_w ? 1 : 0) + (c.dup_w ? 1 : 0);
  p.products = c.dx || want_dw;
  p.half = round_up(n, 128);  // whole tiles of the weights' gradients, whatever their size
  size_t at = 0;
  if (p.products) at = round_up(m * 2 * p.half * e, 256);
  plan_groups(m, ceil_div(p.half, 64 * (16 / e)), &p.groups, &p.rows_per_group);
  p.sums_at = at;
  if (c.dgate_bias || c.dup_bias) at = round_up(at + size_t(p.groups) * 2 * n * 4, 256);
  // The plans go by sizes and layouts, not by which gradients are wanted, so a
  // gradient has the same bits alone; except that the layouts of what is not given
  // are taken as plain, where odd ones could send a large product to other tiles.
  const Operand none{nullptr, k, n, k};
  p.w = c.dx ? pair_of(c.gate_w, c.gate_w_stride, c.up_w, c.up_w_stride, n, k) : PairOperand{{none, none}};
  p.x = want_dw ? operand(c.x, c.x_stride, m, k) : Operand{nullptr, k, m, k};
  const Operand d{nullptr, 2 * p.half, m, 2 * p.half};
  const uint64_t big_m = ceil_div(m, 256), big_n = ceil_div(k, 256), turn = p.half / 64;
  if (e == 2 && big_m * big_n >= kCus / 2 && turn >= 2) {
    p.pack_w = !lies_well(p.w.half[0]) || !lies_well(p.w.half[1]) || p.w.half[0].stride != p.w.half[1].stride;
    p.dx_big = (!p.pack_w || big_m >= 4) && within_reach(d.stride, d.cols, true) &&
               within_reach(p.pack_w ? packed_stride(k) : p.w.half[0].stride, k, false);
    if (!p.dx_big) p.pack_w = false;
  }
  if (m && n && k) {
    p.dw = plan_product(Operand{nullptr, 2 * p.half, m, round_up(n, 8)}, false, p.x, false, n, k, m, c.dtype);
    p.dw_big = p.dw.kind == ProductPlan::kBig;
  }
  if (c.dtype == MSCL_FLOAT32 && m && n && k) {
    const double M = m, N = n, K = k;
    const uint64_t stride = packed_stride(k);
    p.dx_parts = plan_parts(c.dtype, big_m * big_n, 1, m, k, 2 * turn, 2 * N * (M + K), 4 * M * N * K, d.stride, stride);
    p.dw_parts = plan_parts(c.dtype, ceil_div(n, 256) * big_n, 2, n, k, ceil_div(m, 64), M * (2 * N + K), 4 * M * N * K,
                            d.stride, stride);
    p.dx_big = p.dx_parts.on;
    p.dw_big = p.dw_parts.on;
    p.parts = (p.dx_big && c.dx) || (p.dw_big && want_dw);
  }
  // what runs as tiles runs in one launch
  const uint64_t across = ceil_div(k, 128);
  const uint64_t large = 2 * across * ((p.dx_big ? 0 : ceil_div(m, 128)) + (p.dw_big ? 0 : ceil_div(n, 128)));
  choose_tile(&p.dx, large, c.dtype);
  const uint64_t steps = 2 * ((p.dx_big ? 0 : ceil_div(m, p.dx.tile_m) * turn) +
                              (p.dw_big ? 0 : ceil_div(n, p.dx.tile_m) * ceil_div(m, 64))) * ceil_div(k, p.dx.tile_n);
  if (!p.dw_big) {
    const ProductPlan shape = p.dx;
    p.dw = shape;
    choose_shares(&p.dw, n, k, m, steps);
  }
  if (!p.dx_big) choose_shares(&p.dx, m, k, n, steps);
  // Two workgroups on a compute unit split and multiply in turn: 512 x 1025 ->
  // 770 fp32, 306 workgroups, 75 us, in halves of k 52 us; with 768 workgroups
  // (1024 x 2048 -> 1024) 132 us, in halves 149.
  const uint64_t of_tiles = (p.dx_big ? 0 : ceil_div(m, p.dx.tile_m) * ceil_div(k, p.dx.tile_n)) +
                            (p.dw_big ? 0 : 2 * ceil_div(n, p.dx.tile_m) * ceil_div(k, p.dx.tile_n));
  if (e == 4 && of_tiles <= 2 * kCus) {
    if (!p.dx_big && p.dx.shares == 1 && turn >= 8) halve(&p.dx, m, k, ceil_div(n, 64));
    if (!p.dw_big && p.dw.shares == 1 && m >= 512) halve(&p.dw, n, k, ceil_div(m, 64));
  }
  if (p.parts) {
    p.parts_at = at;
    p.d_part = part_bytes(d);
    at += 3 * p.d_part;
  }
  p.dx_at = at;
  if (c.dx && p.dx_big && e == 4) {
    p.w_bytes = part_bytes(p.w.half[0]);
    at += 6 * p.w_bytes + p.dx_parts.partial_bytes;
  } else if (c.dx) {
    if (p.pack_w) p.w_bytes = packed_bytes(p.w.half[0]);
    if (p.dx_big)
      at += 2 * p.w_bytes;
    else if (p.dx.shares > 1)
      at += round_up(2 * size_t(p.dx.shares) * m * p.dx.partial_stride * 4, 256);
  }
  p.dw_at = at;
  if (want_dw && p.dw_big && e == 4) {
    p.x_part = part_bytes(p.x);
    at += 3 * p.x_part + dws * p.dw_parts.partial_bytes;
  } else if (want_dw) {
    at += p.dw_big ? p.dw.bytes() : dws * p.dw.partial_bytes;
  }
  p.bytes = at;
  return p;
}

// Threads of the largest launch of a backward call.
double threads_of(const GatedBackwardPlan& p, const mscl_gated_linear_backward_t& c) {
  const size_t e = bytes_of(c.dtype);
  const uint64_t m = c.rows, k = c.in_features, n = c.out_features;
  const double dws = (c.dgate_w ? 1 : 0) + (c.dup_w ? 1 : 0), across = ceil_div(k, 256);
  double tiles = 0, joins = 0;
  double most = 256.0 * ceil_div(p.half, 64 * (16 / e));  // the slopes
  if (c.dx && p.dx_big) {
    most = std::max(most, 512 * across * ceil_div(m, 256) * p.dx_parts.shares);
    if (p.dx_parts.shares > 1) joins += join_threads(m, k, e);
  } else if (c.dx) {
    tiles += static_cast<double>(ceil_div(m, p.dx.tile_m)) * ceil_div(k, p.dx.tile_n) * p.dx.shares * (p.dx.shares > 1 ? 2 : 1);
    if (p.dx.shares > 1) joins += join_threads(m, k, e);
  }
  if (dws && p.dw_big) {
    most = std::max(most, 512 * across * ceil_div(n, 256) * p.dw_parts.shares * dws);
    if (p.dw_parts.shares > 1) joins += dws * join_threads(n, k, e);
  } else if (dws) {
    tiles += static_cast<double>(ceil_div(n, p.dx.tile_m)) * ceil_div(k, p.dx.tile_n) * p.dw.shares * dws;
    if (p.dw.shares > 1) joins += dws * join_threads(n, k, e);
  }
  if (c.dgate_bias || c.dup_bias) {
    const double of_biases = static_cast<double>(ceil_div(n, 32));
    if (tiles > 0)
      tiles += 2 * of_biases;
    else
      most = std::max(most, 256 * of_biases);
  }
  return std::max({most, 256 * tiles, joins});
}

mscl_status_t check_gated_backward(const mscl_gated_linear_backward_t* c, Spans& s) {
  if (!c) return bad("call is null");
  mscl_status_t st = check_kinds(c->dtype, c->activation);
  if (st == MSCL_SUCCESS) st = check_sizes(c->rows, c->in_features, c->out_features);
  if (st != MSCL_SUCCESS) return st;
  const size_t e = bytes_of(c->dtype), m = c->rows, k = c->in_features, n = c->out_features;
  const bool dw = c->dgate_w || c->dup_w, some = c->dx || dw || c->dgate_bias || c->dup_bias;
  s.add("dy", c->dy, m, n, c->dy_stride, e, false, some);
  if (dw) s.add("x", c->x, m, k, c->x_stride, e, false, n != 0);
  if (c->dx) {
    s.add("gate_w", c->gate_w, n, k, c->gate_w_stride, e, false, m != 0);
    s.add("up_w", c->up_w, n, k, c->up_w_stride, e, false, m != 0);
  }
  s.add("gate", c->gate, m, n, c->gate_stride, e, false, some);
  s.add("up", c->up, m, n, c->up_stride, e, false, some);
  s.add("dx", c->dx, m, k, c->dx_stride, e, true, false);
  s.add("dgate_w", c->dgate_w, n, k, c->dgate_w_stride, e, true, false);
  s.add("dup_w", c->dup_w, n, k, c->dup_w_stride, e, true, false);
  s.add("dgate_bias", c->dgate_bias, 1, n, 0, e, true, false);
  s.add("dup_bias", c->dup_bias, 1, n, 0, e, true, false);
  return s.check();
}

template <class C, int kBM, int kBN>
mscl_status_t launch_gated_back(const GatedBackArgs& a, uint32_t groups, hipStream_t stream) {
  constexpr int kLds = std::max(tile_lds<C, true, false, kBM, kBN>(), tile_lds<C, false, false, kBM, kBN>());
  const hipError_t err = allow_lds<&gated_back<C, kBM, kBN>>(kLds);
  if (err != hipSuccess) return failed_hip(err, "hipFuncSetAttribute");
  gated_back<C, kBM, kBN><<<groups, 256, kLds, stream>>>(a);
  return launched("gated_back");
}

// The joins of up to three products; one of fewer than two shares has none.
template <class C>
mscl_status_t join_gradients(GatedJoinArgs& j, hipStream_t s) {
  uint64_t joins = 0;
  for (int i = 0; i < 3; ++i) {
    if (j.shares[i] < 2) continue;
    const uint64_t of_it = ceil_div(ceil_div(j.e[i].n, C::V) * j.e[i].m, 256);
    joins += of_it;
    j.groups[i] = static_cast<uint32_t>(of_it);
  }
  if (joins == 0) return MSCL_SUCCESS;
  gated_join<C><<<static_cast<uint32_t>(joins), 256, 0, s>>>(j);
  return launched("gated_join");
}

FittedArgs fitted(const TileArgs& t) {
  FittedArgs f;
  f.a = t.a;
  f.b = t.b;
  static_cast<Epilogue&>(f.e) = t.e;
  f.k = t.k;
  f.tiles_m = t.tiles_m;
  f.tiles_n = t.tiles_n;
  f.blocks_per_share = t.blocks_per_share;
  return f;
}

Epilogue results(void* y, uint64_t stride, uint64_t m, uint64_t n) {
  Epilogue e;
  memset(&e, 0, sizeof e);
  e.y = bytes_at(y);
  e.y_stride = stride;
  e.m = m;
  e.n = n;
  return e;
}

template <class C>
mscl_status_t dx_by_large_tiles(const GatedBackwardPlan& p, const Operand& d, const Epilogue& e, int dtype, char* ws,
                                hipStream_t s) {
  PairOperand w = p.w;
  if (p.pack_w) {
    mscl_status_t st = pack_operand(dtype, &w.half[0], ws + p.dx_at, s);
    if (st == MSCL_SUCCESS) st = pack_operand(dtype, &w.half[1], ws + p.dx_at + p.w_bytes, s);
    if (st != MSCL_SUCCESS) return st;
  }
  const uint64_t tm = ceil_div(e.m, 256), tn = ceil_div(e.n, 256);
  const hipError_t err = allow_lds<&gated_dx_big<C>>(kBigLds);
  if (err != hipSuccess) return failed_hip(err, "hipFuncSetAttribute");
  const GatedDxArgs a{d, w, e, static_cast<uint32_t>(p.half / 64), static_cast<uint32_t>(tm), static_cast<uint32_t>(tn)};
  gated_dx_big<C><<<static_cast<uint32_t>(tm * tn), 512, kBigLds, s>>>(a);
  return launched("gated_dx_big");
}

// dx of binary32 operands; d's parts are there.
mscl_status_t dx_by_parts(const GatedBackwardPlan& p, const mscl_gated_linear_backward_t& c, const Operand& d, char* ws,
                          hipStream_t s) {
  char* w_at = ws + p.dx_at;
  for (int h = 0; h < 2; ++h) {
    const mscl_status_t st = split_operand(p.w.half[h], w_at + 3 * h * p.w_bytes, s);
    if (st != MSCL_SUCCESS) return st;
  }
  const uint64_t tm = ceil_div(c.rows, 256), tn = ceil_div(c.in_features, 256);
  const hipError_t err = allow_lds<&gated_dx_parts_big>(kBigLds);
  if (err != hipSuccess) return failed_hip(err, "hipFuncSetAttribute");
  Epilogue e = results(c.dx, c.dx_stride, c.rows, c.in_features);
  if (p.dx_parts.shares > 1) e.partial = reinterpret_cast<float*>(w_at + 6 * p.w_bytes);
  e.partial_stride = p.dx_parts.partial_stride;
  GatedDxPartsArgs a;
  a.parts = {parts_at(d, ws + p.parts_at),
             PairOperand{{parts_at(p.w.half[0], w_at), parts_at(p.w.half[1], w_at + 3 * p.w_bytes)}},
             e, static_cast<uint32_t>(p.half / 64), static_cast<uint32_t>(tm), static_cast<uint32_t>(tn)};
  a.of = {p.d_part, p.w_bytes, p.dx_parts.blocks, p.dx_parts.blocks_per_share};
  for (int h = 0; h < 2; ++h) a.a[h] = Operand{d.base + h * p.half * 4, d.stride, c.rows, c.out_features};
  a.b = p.w;
  a.k = c.out_features;
  gated_dx_parts_big<<<static_cast<uint32_t>(tm * tn * p.dx_parts.shares), 512, kBigLds, s>>>(a);
  const mscl_status_t st = launched("gated_dx_parts_big");
  GatedJoinArgs j;
  memset(&j, 0, sizeof j);
  j.e[0] = e;
  j.shares[0] = p.dx_parts.shares;
  return st != MSCL_SUCCESS ? st : join_gradients<F32>(j, s);
}

// The weights' gradients that are wanted; d's parts are there.
mscl_status_t dw_by_parts(const GatedBackwardPlan& p, const mscl_gated_linear_backward_t& c, const Operand& d, char* ws,
                          hipStream_t s) {
  mscl_status_t st = split_operand(p.x, ws + p.dw_at, s);
  if (st != MSCL_SUCCESS) return st;
  const uint64_t tm = ceil_div(c.out_features, 256), tn = ceil_div(c.in_features, 256);
  const hipError_t err = allow_lds<&gated_dw_parts_big>(kBigLds);
  if (err != hipSuccess) return failed_hip(err, "hipFuncSetAttribute");
  GatedDwPartsArgs a;
  memset(&a, 0, sizeof a);
  for (int h = 0; h < 2; ++h) {
    void* to = h ? c.dup_w : c.dgate_w;
    if (!to) continue;
    const uint32_t i = a.count++;
    a.a[i] = Operand{ws + p.parts_at + h * p.half * 2, 2 * p.half, c.rows, round_up(c.out_features, 8)};
    a.a32[i] = Operand{d.base + h * p.half * 4, d.stride, c.rows, c.out_features};
    a.e[i] = results(to, h ? c.dup_w_stride : c.dgate_w_stride, c.out_features, c.in_features);
    if (p.dw_parts.shares > 1)
      a.e[i].partial = reinterpret_cast<float*>(ws + p.dw_at + 3 * p.x_part + i * p.dw_parts.partial_bytes);
    a.e[i].partial_stride = p.dw_parts.partial_stride;
  }
  a.b = parts_at(p.x, ws + p.dw_at);
  a.b32 = p.x;
  a.of = {p.d_part, p.x_part, p.dw_parts.blocks, p.dw_parts.blocks_per_share};
  a.k = c.rows;
  a.tiles_m = static_cast<uint32_t>(tm);
  a.tiles_n = static_cast<uint32_t>(tn);
  gated_dw_parts_big<<<static_cast<uint32_t>(a.count * tm * tn * p.dw_parts.shares), 512, kBigLds, s>>>(a);
  if ((st = launched("gated_dw_parts_big")) != MSCL_SUCCESS) return st;
  GatedJoinArgs j;
  memset(&j, 0, sizeof j);
  for (uint32_t i = 0; i < a.count; ++i) {
    j.e[i] = a.e[i];
    j.shares[i] = p.dw_parts.shares;
  }
  return join_gradients<F32>(j, s);
}

// dx, both weights' gradients and the bias gradients' last sums, as far as they
// run as tiles.
template <class C>
mscl_status_t back_by_tiles(const GatedBackwardPlan& p, const mscl_gated_linear_backward_t& c, bool dx, bool dw, bool db,
                            const Operand& d, const JoinArgs& join, char* ws, hipStream_t s) {
  const uint64_t m = c.rows, k = c.in_features, n = c.out_features;
  constexpr size_t e = C::kElemBytes;
  GatedBackArgs a;
  GatedJoinArgs j;
  memset(&a, 0, sizeof a);
  memset(&j, 0, sizeof j);
  a.db = join;
  const uint64_t dx_tiles = ceil_div(m, p.dx.tile_m) * ceil_div(k, p.dx.tile_n);
  const uint64_t dw_tiles = ceil_div(n, p.dx.tile_m) * ceil_div(k, p.dx.tile_n);
  uint64_t groups = 0;
  const bool chained = p.dx.shares == 1;
  a.dx_parts = chained ? 1 : 2;
  for (int h = 0; h < 2; ++h) {
    if (dx) {
      const Operand side{d.base + h * p.half * e, d.stride, m, round_up(n, C::V)};
      a.dx[h] = fitted(tile_args(p.dx, side, p.w.half[h], n, results(c.dx, c.dx_stride, m, k), nullptr));
      a.dx[h].e.partial =
          chained ? nullptr : reinterpret_cast<float*>(ws + p.dx_at) + h * p.dx.shares * m * p.dx.partial_stride;
    }
    void* to = h ? c.dup_w : c.dgate_w;
    const uint64_t stride = h ? c.dup_w_stride : c.dgate_w_stride;
    if (dw && to) {
      // whole tiles of columns: those past the last one meet only rows that are not stored
      const Operand side{d.base + h * p.half * e, d.stride, m, p.half};
      const uint32_t i = a.dw_count++;
      a.dw[i] = fitted(tile_args(p.dw, side, p.x, m, results(to, stride, n, k), ws + p.dw_at + i * p.dw.partial_bytes));
    }
  }
  if (dx) {
    a.dx_tiles = static_cast<uint32_t>(dx_tiles);
    a.dx_groups = static_cast<uint32_t>(dx_tiles * p.dx.shares);
    j.e[0] = a.dx[0].e;
    j.shares[0] = chained ? 1 : 2 * p.dx.shares;
  }
  if (dw) {
    a.dw_tiles = static_cast<uint32_t>(dw_tiles);
    a.dw_groups = static_cast<uint32_t>(dw_tiles * p.dw.shares);
    for (uint32_t i = 0; i < a.dw_count; ++i) {
      j.e[1 + i] = a.dw[i].e;
      j.shares[1 + i] = p.dw.shares;
    }
  }
  groups = uint64_t(a.dx_parts) * a.dx_groups + uint64_t(a.dw_count) * a.dw_groups;
  a.db_blocks = static_cast<uint32_t>(std::max<uint64_t>(1, ceil_div(n, 32)));
  if (db) groups += 2 * uint64_t(a.db_blocks);
  if (groups == 0) return MSCL_SUCCESS;
  mscl_status_t st;
  if (p.dx.tile_m == 128)
    st = launch_gated_back<C, 128, e == 4 ? 64 : 128>(a, static_cast<uint32_t>(groups), s);
  else
    st = launch_gated_back<C, 64, 64>(a, static_cast<uint32_t>(groups), s);
  if (st != MSCL_SUCCESS) return st;
  return join_gradients<C>(j, s);
}

}  // namespace

extern "C" {

mscl_status_t mscl_gated_linear_workspace(const mscl_gated_linear_t* call, size_t* bytes) {
  if (!bytes) return bad("bytes is null");
  Spans spans;
  const mscl_status_t st = check_gated(call, spans);
  if (st != MSCL_SUCCESS) return st;
  *bytes = 0;
  if (call->rows == 0 || call->out_features == 0) return MSCL_SUCCESS;
  const GatedPlan p = plan_gated(*call);
  *bytes = p.bytes;
  return check_threads(threads_of(p, *call));
}

mscl_status_t mscl_gated_linear(const mscl_gated_linear_t* call, void* workspace, size_t workspace_bytes, void* stream) {
  Spans spans;
  mscl_status_t st = check_gated(call, spans);
  if (st != MSCL_SUCCESS) return st;
  const mscl_gated_linear_t& c = *call;
  if (c.rows == 0 || c.out_features == 0) return MSCL_SUCCESS;
  const GatedPlan p = plan_gated(c);
  if ((st = check_threads(threads_of(p, c))) != MSCL_SUCCESS) return st;
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
    e.z[0] = bytes_at(c.gate);
    e.z[1] = bytes_at(c.up);
    e.z_stride[0] = c.gate_stride;
    e.z_stride[1] = c.up_stride;
    e.m = c.rows;
    e.n = c.out_features;
    e.act = c.activation;
    if constexpr (std::is_same<decltype(t), F32>::value)
      if (p.parts.on) return gated_by_parts(p, c, e, bytes_at(workspace), static_cast<hipStream_t>(stream));
    return forward<decltype(t)>(p.tiles, operand(c.x, c.x_stride, c.rows, c.in_features), weights_of(c), c.in_features, e,
                                bytes_at(workspace), static_cast<hipStream_t>(stream));
  });
}

mscl_status_t mscl_gated_linear_backward_workspace(const mscl_gated_linear_backward_t* call, size_t* bytes) {
  if (!bytes) return bad("bytes is null");
  Spans spans;
  const mscl_status_t st = check_gated_backward(call, spans);
  if (st != MSCL_SUCCESS) return st;
  const GatedBackwardPlan p = plan_gated_backward(*call);
  *bytes = p.bytes;
  return check_threads(threads_of(p, *call));
}

mscl_status_t mscl_gated_linear_backward(const mscl_gated_linear_backward_t* call, void* workspace,
                                         size_t workspace_bytes, void* stream) {
  Spans spans;
  mscl_status_t st = check_gated_backward(call, spans);
  if (st != MSCL_SUCCESS) return st;
  const mscl_gated_linear_backward_t& c = *call;
  const GatedBackwardPlan p = plan_gated_backward(c);
  if ((st = check_threads(threads_of(p, c))) != MSCL_SUCCESS) return st;
  if ((st = spans.check_workspace(workspace, workspace_bytes, p.bytes)) != MSCL_SUCCESS) return st;
  const bool dx = c.dx && c.rows && c.in_features;
  const bool dw = (c.dgate_w || c.dup_w) && c.out_features && c.in_features;
  const bool db = (c.dgate_bias || c.dup_bias) && c.out_features;
  if (!dx && !dw && !db) return MSCL_SUCCESS;
  int cus = 0;
  if ((st = current_device(&cus)) != MSCL_SUCCESS) return st;
  const hipStream_t s = static_cast<hipStream_t>(stream);
  char* ws = bytes_at(workspace);
  const size_t e = bytes_of(c.dtype);

  GatedSlopeArgs g;
  g.dy = bytes_at(c.dy);
  g.z = bytes_at(c.gate);
  g.v = bytes_at(c.up);
  g.d = dx || dw ? ws + p.d_at : nullptr;
  g.sums = db ? reinterpret_cast<float*>(ws + p.sums_at) : nullptr;
  g.dy_stride = c.dy_stride;
  g.z_stride = c.gate_stride;
  g.v_stride = c.up_stride;
  g.half = p.half;
  g.rows = c.rows;
  g.cols = c.out_features;
  g.rows_per_group = p.rows_per_group;
  g.act = c.activation;
  const uint64_t blocks = ceil_div(p.half, 64 * (16 / e));
  if (blocks) {
    st = with_codec(c.dtype, [&](auto t) {
      gated_slope<decltype(t)><<<dim3(static_cast<uint32_t>(blocks), p.groups), 256, 0, s>>>(g);
      return launched("gated_slope");
    });
    if (st != MSCL_SUCCESS) return st;
  }
  const JoinArgs join =
      join_args(g.sums, c.out_features, c.out_features, p.groups, c.dgate_bias, c.dup_bias, 2);
  const Operand d{ws + p.d_at, 2 * p.half, c.rows, 2 * p.half};
  const bool dx_tiles = dx && !p.dx_big, dw_tiles = dw && !p.dw_big;
  const bool db_with_tiles = db && (dx_tiles || dw_tiles);
  if (db && !db_with_tiles && (st = join_columns(c.dtype, join, 2, s)) != MSCL_SUCCESS) return st;
  if (p.parts && (dx || dw) && (st = split_operand(d, ws + p.parts_at, s)) != MSCL_SUCCESS) return st;
  if (dx && p.dx_big && e == 4) {
    if ((st = dx_by_parts(p, c, d, ws, s)) != MSCL_SUCCESS) return st;
  } else if (dx && p.dx_big) {
    const Epilogue ex = results(c.dx, c.dx_stride, c.rows, c.in_features);
    st = c.dtype == MSCL_FLOAT16 ? dx_by_large_tiles<F16>(p, d, ex, c.dtype, ws, s)
                                 : dx_by_large_tiles<BF16>(p, d, ex, c.dtype, ws, s);
    if (st != MSCL_SUCCESS) return st;
  }
  if (dw && p.dw_big && e == 4) {
    if ((st = dw_by_parts(p, c, d, ws, s)) != MSCL_SUCCESS) return st;
  } else if (dw && p.dw_big) {
    ProductPlan dw_plan = p.dw;
    Operand x = p.x;
    char* at = ws + p.dw_at;
    if (dw_plan.pack_b) {  // once for both
      if ((st = pack_operand(c.dtype, &x, at, s)) != MSCL_SUCCESS) return st;
      dw_plan.pack_b = false;
    }
    for (int h = 0; h < 2; ++h) {
      void* to = h ? c.dup_w : c.dgate_w;
      if (!to) continue;
      const Operand side{d.base + h * p.half * e, d.stride, c.rows, round_up(c.out_features, 8)};
      st = weight_gradient(c.dtype, dw_plan, side, x, c.rows,
                           results(to, h ? c.dup_w_stride : c.dgate_w_stride, c.out_features, c.in_features), at, s);
      if (st != MSCL_SUCCESS) return st;
    }
  }
  if (!dx_tiles && !dw_tiles) return MSCL_SUCCESS;
  return with_codec(c.dtype, [&](auto t) {
    return back_by_tiles<decltype(t)>(p, c, dx_tiles, dw_tiles, db_with_tiles, d, join, ws, s);
  });
}

}  // extern "C"
