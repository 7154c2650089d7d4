// Host side that the gated feed-forward block and the 8-bit products share:
// checks, and the plans and launches of the kernels in feedforward.hpp.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include <algorithm>
#include <cmath>
#include <type_traits>

#include "../../include/mscl.h"
#include "failure.hpp"
#include "feedforward.hpp"
#include "launch.hpp"
#include "linear.hpp"

namespace mscl {
namespace __attribute__((visibility("hidden"))) launch {

// An 8-bit operand laid out anew at `to`; defined in quantized.hip.
mscl_status_t pack_int8(Operand* o, char* to, hipStream_t stream);

inline mscl_status_t check_sizes(size_t rows, size_t in, size_t out) {
  if (rows > kMostGroups || in > kMostGroups || out > kMostGroups) return bad("the matrices are too large");
  return MSCL_SUCCESS;
}

inline mscl_status_t check_kinds(int dtype, int activation) {
  if (!known_dtype(dtype)) return bad("unknown dtype");
  if (activation < MSCL_ACT_NONE || activation > MSCL_ACT_SILU) return bad("unknown activation");
  return MSCL_SUCCESS;
}

inline mscl_status_t check_reach_of_sums(size_t in) {
  // 128 * 128 * 131071 < 2^31
  return in > 131071 ? bad("in_features must be at most 131071") : MSCL_SUCCESS;
}

inline PairOperand pair_of(const void* gate, size_t gate_stride, const void* up, size_t up_stride, uint64_t n, uint64_t k) {
  return PairOperand{{operand(gate, gate_stride, n, k), operand(up, up_stride, n, k)}};
}
// ------------------------------------------------------------------ forward products

// Threads that add the shares of k of m x n results of `out` bytes each: 16 bytes a thread.
inline double join_threads(uint64_t m, uint64_t n, size_t out) {
  return 256 * std::ceil(static_cast<double>(ceil_div(n, 16 / out)) * m / 256);
}

// How the products of m rows with one weight or a pair of n x k run.
struct ForwardPlan {
  enum { kTile, kBig, kFew } kind = kTile;
  int tile_m = 64;   // rows of a tile
  int outs = 64;     // outputs of a tile, of each weight
  bool pack_a = false, pack_b = false;  // operands laid out anew for forward_big
  uint32_t shares = 1, blocks_per_share = 1;
  uint64_t partial_stride = 0;
  size_t a_bytes = 0, b_bytes = 0, partial_bytes = 0;  // b: of each weight
  size_t bytes = 0;
};

// Elements of k in a block of the tiles.
inline uint64_t block_of(size_t e) { return e == 1 ? 128 : 64; }

inline void share_k(ForwardPlan* p, uint64_t shares, uint64_t steps, uint64_t m, uint64_t n, int parts) {
  p->blocks_per_share = static_cast<uint32_t>(std::max<uint64_t>(1, ceil_div(steps, shares)));
  p->shares = static_cast<uint32_t>(std::max<uint64_t>(1, ceil_div(steps, p->blocks_per_share)));
  p->partial_stride = parts * round_up(n, 8);
  if (p->shares > 1) p->partial_bytes = round_up(p->shares * m * p->partial_stride * 4, 256);
  p->bytes = p->partial_bytes;
}

// forward_tile's tile, and the shares of k, by what a launch of them takes.  A
// workgroup alone on its compute unit takes 4 us and, for each block of k (us,
// from products of 8 to 128 blocks)
//                          64 rows   128 rows
//   8 bits                   0.285     0.69      (64 and 128 columns)
//   pairs of 8 or 16 bits    0.43      0.69      (64 of each)
//   pairs of binary32        1.35      2.35      (32 of each)
// and r of them at once take 0.92 r times as long (0.75 r, binary32, whose
// operands' splitting and products overlap).  Shares shorten the run of blocks,
// and cost a launch and a write and a read of their sums at 4 TB/s.  us, without
// shares and with two: 512 x 512 -> 4096 pairs of bf16 11 and 28, 1024 x 2048 ->
// 1024 8 bits 8.9 and 15; the other way 64 x 8192 -> 4096 pairs of bf16 59 and
// 38 (four 29), 1024 x 2048 -> 1024 pairs of binary32 82 and 70.
inline void choose_tiles(ForwardPlan* p, uint64_t m, uint64_t n, uint64_t k, int parts, size_t e) {
  const uint64_t steps = ceil_div(k, block_of(e));
  double best = 0;
  uint64_t best_shares = 1;
  for (const int rows : {64, 128}) {
    const int outs = e == 4 ? 64 / parts : (parts == 1 ? rows : 64);
    const double block = e == 4 ? (rows == 64 ? 1.35 : 2.35) : (rows == 128 ? 0.69 : (parts == 1 ? 0.285 : 0.43));
    const uint64_t tiles = ceil_div(m, rows) * ceil_div(n, outs);
    for (const uint64_t shares : {1, 2, 3, 4, 6, 8, 12, 16, 24, 32}) {
      if (shares > 1 && 2 * shares > steps) break;
      const double at_once = static_cast<double>(ceil_div(tiles * shares, kCus));
      double us = 4 + block * ceil_div(steps, shares) * std::max(1.0, (e == 4 ? 0.75 : 0.92) * at_once);
      if (shares > 1) us += 4 + 8.0 * shares * m * parts * n / 4e6;
      if (best > 0 && us >= best) continue;
      best = us;
      best_shares = shares;
      p->tile_m = rows;
      p->outs = outs;
    }
  }
  share_k(p, best_shares, steps, m, n, parts);
}

inline ForwardPlan plan_forward(const Operand& a, const Operand* b, int parts, uint64_t m, uint64_t n, uint64_t k, size_t e) {
  ForwardPlan p;
  const uint64_t block = 128 / e, blocks = ceil_div(k, block);
  const uint64_t big_m = ceil_div(m, 256), big_n = ceil_div(n, 256 / parts);
  auto lies = [&](const Operand& o) {
    return reinterpret_cast<uintptr_t>(o.base) % 16 == 0 && o.stride * e % 16 == 0 && o.cols * e % 16 == 0;
  };
  auto reach = [&](uint64_t stride) {
    const uint64_t limit = (uint64_t(1) << 31) / e;
    return stride < limit / 256 && k < limit - 256 * stride;
  };
  if (e <= 2 && big_m * big_n >= kCus / 2 && blocks >= 4 && !mostly_empty(true, m, n * parts, big_m * big_n)) {
    p.pack_a = !lies(a);
    p.pack_b = !lies(b[0]) || (parts == 2 && (!lies(b[1]) || b[0].stride != b[1].stride));
    if ((!p.pack_a || big_n >= 4) && (!p.pack_b || big_m >= 4) && reach(p.pack_a ? packed_stride(k) : a.stride) &&
        reach(p.pack_b ? packed_stride(k) : b[0].stride)) {
      p.kind = ForwardPlan::kBig;
      p.tile_m = 256;
      p.outs = 256 / parts;
      if (p.pack_a) p.a_bytes = packed_bytes(a, e);
      if (p.pack_b) p.b_bytes = packed_bytes(b[0], e);
      p.bytes = p.a_bytes + parts * p.b_bytes;
      return p;
    }
    p.pack_a = p.pack_b = false;
  }
  if (m <= 32 && k > 0) {
    const uint64_t whole = std::max<uint64_t>(1, k / block);
    p.kind = ForwardPlan::kFew;
    p.tile_m = 32;
    p.outs = parts == 1 && (m > 16 || (m > 8 && ceil_div(n, 32) >= kCus)) ? 32 : 16;
    const uint64_t groups = ceil_div(n, p.outs);
    const uint64_t shares = groups < kCus ? std::max<uint64_t>(1, std::min(kCus / groups, whole / 32)) : 1;
    share_k(&p, shares, whole, m, n, parts);
    return p;
  }
  choose_tiles(&p, m, n, k, parts, e);
  return p;
}

// Threads of the largest launch of a plan whose results take `out` bytes each.
inline double threads_of(const ForwardPlan& p, uint64_t m, uint64_t n, size_t out) {
  const double tiles = static_cast<double>(ceil_div(m, p.tile_m)) * ceil_div(n, p.outs);
  const double products = p.kind == ForwardPlan::kTile ? 256 * tiles * p.shares : 512 * tiles;
  return p.shares > 1 ? std::max(products, join_threads(m, n, out)) : products;
}

template <class C>
mscl_status_t pack_any(Operand* o, char* to, hipStream_t stream) {
  if constexpr (C::kElemBytes == 2)
    return pack_operand(std::is_same<C, F16>::value ? MSCL_FLOAT16 : MSCL_BFLOAT16, o, to, stream);
  return pack_int8(o, to, stream);
}

template <class C, class B>
mscl_status_t pack_weights(B* b, size_t bytes, char* to, hipStream_t stream) {
  if constexpr (B::kParts == 1) {
    return pack_any<C>(b, to, stream);
  } else {
    const mscl_status_t st = pack_any<C>(&b->half[0], to, stream);
    return st != MSCL_SUCCESS ? st : pack_any<C>(&b->half[1], to + bytes, stream);
  }
}

template <class C, int kBM, int kBN, class B, class E>
mscl_status_t launch_forward_tile(const TileArgsOf<B, E>& t, uint32_t groups, hipStream_t stream) {
  constexpr int kLds = tile_lds<C, true, true, kBM, kBN>();
  const hipError_t err = allow_lds<&forward_tile<C, kBM, kBN, B, E>>(kLds);
  if (err != hipSuccess) return failed_hip(err, "hipFuncSetAttribute");
  forward_tile<C, kBM, kBN, B, E><<<groups, 256, kLds, stream>>>(t);
  return launched("forward_tile");
}

// Adds the shares of k at e.partial and finishes the sums.
template <class C, class E>
mscl_status_t join_forward(const E& e, uint32_t shares, hipStream_t stream) {
  const uint64_t joins = ceil_div(ceil_div(e.n, OutOf<E>::V) * e.m, 256);
  forward_join<C, E><<<static_cast<uint32_t>(joins), 256, 0, stream>>>(e, static_cast<int>(shares));
  return launched("forward_join");
}

// threads_of(p) have passed check_threads().
template <class C, class B, class E>
mscl_status_t forward(const ForwardPlan& p, Operand a, B b, uint64_t k, E e, char* workspace, hipStream_t stream) {
  const uint64_t tm = ceil_div(e.m, p.tile_m), tn = ceil_div(e.n, p.outs);
  const uint32_t groups = static_cast<uint32_t>(tm * tn);
  if constexpr (C::kElemBytes <= 2) {
    if (p.kind == ForwardPlan::kBig) {
      mscl_status_t st = MSCL_SUCCESS;
      if (p.pack_a) st = pack_any<C>(&a, workspace, stream);
      if (st == MSCL_SUCCESS && p.pack_b) st = pack_weights<C>(&b, p.b_bytes, workspace + p.a_bytes, stream);
      if (st != MSCL_SUCCESS) return st;
      const hipError_t err = allow_lds<&forward_big<C, B, E>>(kBigLds);
      if (err != hipSuccess) return failed_hip(err, "hipFuncSetAttribute");
      const BigArgsOf<B, E> t{a, b, e, round_up(k, C::V), static_cast<uint32_t>(tm), static_cast<uint32_t>(tn)};
      forward_big<C, B, E><<<groups, 512, kBigLds, stream>>>(t);
      return launched("forward_big");
    }
  }
  e.partial = p.shares > 1 ? reinterpret_cast<float*>(workspace) : nullptr;
  e.partial_stride = p.partial_stride;
  const TileArgsOf<B, E> t{a, b, e, k, static_cast<uint32_t>(tm), static_cast<uint32_t>(tn), p.blocks_per_share};
  mscl_status_t st = MSCL_SUCCESS;
  if (p.kind == ForwardPlan::kFew) {
    const dim3 grid(groups, p.shares);
    if (e.m > 16)
      forward_few<C, 2, 2, 1, B, E><<<grid, 512, 0, stream>>>(t);
    else if (p.outs * B::kParts == 32)
      forward_few<C, 1, 2, 1, B, E><<<grid, 512, 0, stream>>>(t);
    else if constexpr (B::kParts == 1)
      forward_few<C, 1, 1, 2, B, E><<<grid, 512, 0, stream>>>(t);
    st = launched("forward_few");
  } else if constexpr (C::kElemBytes == 4) {
    if (p.tile_m == 128)
      st = launch_forward_tile<C, 128, 64>(t, groups * p.shares, stream);
    else
      st = launch_forward_tile<C, 64, 64>(t, groups * p.shares, stream);
  } else if (p.tile_m == 128) {
    st = launch_forward_tile<C, 128, 128>(t, groups * p.shares, stream);
  } else {
    st = launch_forward_tile<C, 64, 64 * B::kParts>(t, groups * p.shares, stream);
  }
  return st != MSCL_SUCCESS || p.shares == 1 ? st : join_forward<C>(e, p.shares, stream);
}

}  // namespace launch
}  // namespace mscl
