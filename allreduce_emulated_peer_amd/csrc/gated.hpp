// Kernels of the gated feed-forward block alone: its backward pass, and large
// binary32 products.  The other forward kernels are feedforward.hpp's.
//
//   gated_slope        both sums' gradients, side by side in the workspace, and
//                      the bias gradients' partial sums
//   gated_dx_big       input gradient, one product over both weights
//   gated_back         tiles of all three products in one launch
//   gated_join         adds their shares of k
//   split_parts        a binary32 operand as three of bfloat16
//   gated_parts_big, gated_dx_parts_big, gated_dw_parts_big
//                      large products of binary32 operands in parts
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "../../include/mscl.h"
#include "codec.hpp"
#include "feedforward.hpp"
#include "linear.hpp"

namespace mscl {

// ------------------------------------------------------------------ large binary32 products

// A binary32 operand as linear.hpp's three bfloat16 parts, each a matrix of its
// own in the workspace.  The parts are taken apart once and not in every tile
// that uses them, and a product is then one of 16 bits whose k is six times as
// long: block t is block t / 6 of k, of the parts that pair t % 6 names, the
// smaller products first.
constexpr int kPairs = 6;
constexpr uint32_t kPartsOfA = 0 | 1 << 2 | 2 << 4 | 0 << 6 | 1 << 8 | 0 << 10;
constexpr uint32_t kPartsOfB = 2 | 1 << 2 | 0 << 4 | 1 << 6 | 0 << 8 | 0 << 10;

struct SplitArgs {
  Operand from;
  char* to;            // three parts, `part_bytes` apart
  uint64_t to_stride;  // elements: rows at 128-byte boundaries
  uint64_t part_bytes;
};

// 8 values a thread, past the row's end zeros up to a whole vector.  A pass
// over memory: 4 bytes read and 6 written for each value.
__global__ __launch_bounds__(256) void split_parts(const SplitArgs a) {
  const uint64_t per_row = (a.from.cols + 7) / 8, total = per_row * a.from.rows;
  for (uint64_t id = static_cast<uint64_t>(blockIdx.x) * 256 + threadIdx.x; id < total;
       id += static_cast<uint64_t>(gridDim.x) * 256) {
    const uint64_t row = id / per_row, col = id % per_row * 8;
    const int valid = a.from.cols - col < 8 ? static_cast<int>(a.from.cols - col) : 8;
    const char* p = a.from.base + (row * a.from.stride + col) * 4;
    const u32x4 lo = load_upto<F32>(p, valid), hi = load_upto<F32>(p + 16, valid - 4);
    const Parts o = split(lo, hi);
#pragma unroll
    for (int i = 0; i < 3; ++i)
      *reinterpret_cast<u32x4*>(a.to + i * a.part_bytes + (row * a.to_stride + col) * 2) = o.part[i];
  }
}

// The copies of an operand that lies in parts, from block `first` of k on.
template <class Inner>
struct PartCopier {
  Inner in;
  uint64_t part_bytes;
  uint32_t parts;  // 2 bits for each pair
  uint32_t first;
  __device__ inline void copy(uint32_t lds, int h, uint32_t t, int wave) const {
    const uint32_t block = t / kPairs, pair = t - block * kPairs;
    Inner from = in;
    from.shift((parts >> (2 * pair) & 3) * part_bytes);
    from.copy(lds, h, first + block, wave);
  }
};

struct PartsOf {
  uint64_t a_bytes, b_bytes;  // of one part
  uint32_t blocks;            // of k, and of one share of it
  uint32_t blocks_per_share;
};

// Blocks [first, first + count) of k: one share's.
struct ShareOf {
  uint32_t first, count;
  __device__ inline ShareOf(const PartsOf& o, uint32_t share) {
    first = share * o.blocks_per_share;
    count = o.blocks - first < o.blocks_per_share ? o.blocks - first : o.blocks_per_share;
  }
};

template <class A, class B>
__device__ inline void take_parts(PartCopier<A>& a, PartCopier<B>& b, const PartsOf& o, const ShareOf& s) {
  a.part_bytes = o.a_bytes;
  b.part_bytes = o.b_bytes;
  a.parts = kPartsOfA;
  b.parts = kPartsOfB;
  a.first = b.first = s.first;
}

// A wave's sums of parts to those of the values; where one of the m x n is not
// finite, all of them again in binary32 from the operands themselves.  What lies
// past the matrix may be anything and is not looked at.  at(p) is where quarter p
// begins, a_of(h) and b_of(h, p) its operands in the h-th run of `turn` blocks of
// k, of which k_end exist.
template <bool kAAlong, bool kBAlong, class At, class OfA, class OfB>
__device__ inline void finish_parts(f32x4 (&acc)[4][4][2], uint64_t m, uint64_t n, uint64_t k_end, uint32_t turn,
                                    const ShareOf& share, At&& at, OfA&& a_of, OfB&& b_of) {
  const int lane = threadIdx.x & 63, r = lane & 15, g = lane >> 4;
  bool odd = false;
#pragma unroll
  for (int p = 0; p < 4; ++p) {
    const Corner c = at(p);
    const int rows = c.first >= m ? 0 : (m - c.first < 64 ? static_cast<int>(m - c.first) : 64);
    const int cols = c.second >= n ? 0 : (n - c.second < 32 ? static_cast<int>(n - c.second) : 32);
#pragma unroll
    for (int x = 0; x < 4; ++x)
#pragma unroll
      for (int y = 0; y < 2; ++y) {
#pragma unroll
        for (int i = 0; i < 4; ++i)
          if (16 * x + r < rows && 16 * y + 4 * g + i < cols) odd |= !(fabsf(acc[p][x][y][i]) < INFINITY);
        acc[p][x][y] *= kSplitBack;
      }
  }
  if (!__any(odd)) return;
#pragma unroll
  for (int p = 0; p < 4; ++p) {
#pragma unroll
    for (int x = 0; x < 4; ++x)
#pragma unroll
      for (int y = 0; y < 2; ++y) acc[p][x][y] = f32x4{0.f, 0.f, 0.f, 0.f};
    const Corner c = at(p);
    for (uint32_t step = 0; step < share.count * 16; ++step) {
      const uint32_t block = share.first + step / 16, h = block / turn;
      const uint64_t k = static_cast<uint64_t>(block % turn) * 64 + step % 16 * 4;
      float a[4], b[2];
#pragma unroll
      for (int x = 0; x < 4; ++x) a[x] = value_at<kAAlong>(a_of(h), c.first + 16 * x + r, k + g, k_end);
#pragma unroll
      for (int y = 0; y < 2; ++y) b[y] = value_at<kBAlong>(b_of(h, p), c.second + 16 * y + r, k + g, k_end);
#pragma unroll
      for (int x = 0; x < 4; ++x)
#pragma unroll
        for (int y = 0; y < 2; ++y) acc[p][x][y] = __builtin_amdgcn_mfma_f32_16x16x4f32(b[y], a[x], acc[p][x][y], 0, 0, 0);
    }
  }
}

// forward_big of a pair of binary32 weights in parts; a and b are the operands
// themselves.
struct GatedPartsArgs {
  BigArgsOf<PairOperand, Gated<F32>> parts;
  PartsOf of;
  Operand a;
  PairOperand b;
  uint64_t k;
};

// 4096 x 4096 -> 4096: 1190 to 1215 us with the parts (226 to 232 TFLOP/s; a
// binary32 library product 153).
__global__ __launch_bounds__(512, 2) void gated_parts_big(const GatedPartsArgs args) {
  const auto& t = args.parts;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int wm = wave >> 2, wn = wave & 3;
  const uint32_t tiles = t.tiles_m * t.tiles_n, id = xcd_run(blockIdx.x, gridDim.x);
  const TileAt at(id % tiles, t.tiles_m, t.tiles_n);
  const ShareOf share(args.of, id / tiles);
  const uint64_t m0 = static_cast<uint64_t>(at.m) * 256, n0 = static_cast<uint64_t>(at.n) * 128;
  PartCopier<Copier<BF16, true>> ca;
  PartCopier<PairCopier<BF16>> cb;
  ca.in.init(t.a, m0, t.k, args.of.blocks, wave);
  cb.in.init(t.b, n0, t.k, args.of.blocks, wave);
  take_parts(ca, cb, args.of, share);
  f32x4 acc[4][4][2];
  big_sums<BF16, true, true>(ca, cb, kPairs * share.count, wave, acc);
  finish_parts<true, true>(
      acc, t.e.m, t.e.n, args.k, args.of.blocks, share, [&](int p) { return Corner{m0 + (p >> 1) * 128 + wm * 64, n0 + wn * 32}; },
      [&](int) -> const Operand& { return args.a; }, [&](int, int p) -> const Operand& { return args.b.half[p & 1]; });
  if (t.e.partial) {
    using G = Groups<F32, 4, 2>;
#pragma unroll
    for (int p = 0; p < 4; ++p)
#pragma unroll
      for (int q = 0; q < G::kCount; ++q) {
        float v[4];
        G::sums(acc[p], q, v);
        keep_share(t.e, id / tiles, G::row(m0 + (p >> 1) * 128 + wm * 64, q), G::column(n0 + wn * 32, q), p & 1, v);
      }
    return;
  }
  finish_blocks<F32, 4, 2, 2>(
      t.e, [&](int b, int p) -> const f32x4(&)[4][2] { return acc[2 * b + p]; },
      [&](int b) { return Corner{m0 + b * 128 + wm * 64, n0 + wn * 32}; });
}

// ------------------------------------------------------------------ backward pass

struct GatedSlopeArgs {
  const char *dy, *z, *v;  // z: the gate's sums, v: the other's
  char* d;      // null: not wanted; else rows of dz and dv, `half` columns each
  float* sums;  // null: no bias gradients; else [gridDim.y][2][cols]
  uint64_t dy_stride, z_stride, v_stride, half;
  uint64_t rows, cols;
  uint32_t rows_per_group;
  int act;
};

// dz = dy v act'(z) and dv = dy act(z), and each column's sums of both over
// this workgroup's rows, in binary32 from the unrounded values: a pass over
// memory as linear_slope.  Both are rounded to the element type, which is what
// the matrix units multiply; columns from the last one to `half` become 0.
// 8192 x 4096 bf16: 70 us (335 MB, 4.8 TB/s).
template <class C>
__global__ __launch_bounds__(256) void gated_slope(const GatedSlopeArgs a) {
  constexpr int V = C::V;
  constexpr bool kFast = C::kElemBytes == 2;
  __shared__ float part[2][4][64 * V];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const uint64_t n = (static_cast<uint64_t>(blockIdx.x) * 64 + lane) * V;
  const uint64_t first = static_cast<uint64_t>(blockIdx.y) * a.rows_per_group;
  uint64_t end = first + a.rows_per_group;
  if (end > a.rows) end = a.rows;
  const int valid = n >= a.cols ? 0 : (a.cols - n < V ? static_cast<int>(a.cols - n) : V);
  float sum[2][V];
#pragma unroll
  for (int i = 0; i < V; ++i) sum[0][i] = sum[1][i] = 0.0f;
  with_activation(a.act, [&](auto act) {
    with_edges(n - lane * V + 64 * V <= a.cols, [&](auto full) {
      constexpr int kAct = decltype(act)::value;
      constexpr bool kFull = decltype(full)::value;
      constexpr int kRows = 4;  // in flight
      // A lane at a row's end loads the vector that ends there and moves it down,
      // a lane behind it the row's first and drops it, so that no load hangs on a
      // branch and all are in flight together; rows shorter than a vector are
      // loaded element by element.
      const bool whole = kFull || a.cols >= V;
      const uint32_t back = kFull || valid == V ? 0 : (valid > 0 ? (V - valid) * C::kElemBytes : 16);
      const uint64_t from = kFull || valid == V ? n : (valid > 0 ? a.cols - V : 0);
      auto fetch = [&](const char* base, uint64_t m, uint64_t stride) {
        if (!whole) return load_upto<C>(base + (m * stride + n) * C::kElemBytes, valid);
        return load_loose<C>(base + (m * stride + from) * C::kElemBytes);
      };
      for (uint64_t m0 = first + wave; m0 < end; m0 += 4 * kRows) {
        u32x4 dy[kRows], z[kRows], v[kRows];
#pragma unroll
        for (int q = 0; q < kRows; ++q) {
          const uint64_t m = m0 + 4 * q < end ? m0 + 4 * q : end - 1;
          dy[q] = fetch(a.dy, m, a.dy_stride);
          z[q] = fetch(a.z, m, a.z_stride);
          v[q] = fetch(a.v, m, a.v_stride);
        }
        if (!kFull && whole) {
#pragma unroll
          for (int q = 0; q < kRows; ++q) {
            dy[q] = moved_down(dy[q], back);
            z[q] = moved_down(z[q], back);
            v[q] = moved_down(v[q], back);
          }
        }
#pragma unroll
        for (int q = 0; q < kRows; ++q) {
          if (m0 + 4 * q >= end) continue;
          float g[V], t[V], w[V];
          C::unpack(dy[q], g);
          C::unpack(z[q], t);
          C::unpack(v[q], w);
#pragma unroll
          for (int i = 0; i < V; ++i) {
            const float dz = g[i] * w[i] * slope<kAct, kFast>(t[i]);
            w[i] = g[i] * activate<kAct, kFast>(t[i]);
            g[i] = dz;
            sum[0][i] += g[i];
            sum[1][i] += w[i];
          }
          if (a.d && (kFull || n < a.half)) {
            char* to = a.d + ((m0 + 4 * q) * 2 * a.half + n) * C::kElemBytes;
            *reinterpret_cast<u32x4*>(to) = C::pack(g);
            *reinterpret_cast<u32x4*>(to + a.half * C::kElemBytes) = C::pack(w);
          }
        }
      }
    });
  });
  if (!a.sums) return;
#pragma unroll
  for (int i = 0; i < V; ++i) {
    part[0][wave][lane * V + i] = sum[0][i];
    part[1][wave][lane * V + i] = sum[1][i];
  }
  __syncthreads();
  float* out = a.sums + static_cast<uint64_t>(blockIdx.y) * 2 * a.cols;
  for (int c = threadIdx.x; c < 2 * 64 * V; c += 256) {
    const int p = c / (64 * V), i = c % (64 * V);
    const uint64_t col = static_cast<uint64_t>(blockIdx.x) * 64 * V + i;
    if (col < a.cols) out[p * a.cols + col] = (part[p][0][i] + part[p][1][i]) + (part[p][2][i] + part[p][3][i]);
  }
}

// The copies of two weights as one operand whose k runs down the first's rows
// and then the second's, `turn` blocks each: rows past a weight's end, and whole
// blocks of them, read as 0.
template <class C>
struct ChainCopier {
  Copier<C, false> first;
  const char* base;  // of the second weight's tile
  uint64_t left;
  uint32_t turn;

  __device__ inline void init(const PairOperand& b, uint64_t n, uint32_t turn_, int wave) {
    first.init(b.half[0], n, 0, static_cast<uint32_t>((b.half[0].rows + 63) / 64), wave);
    turn = turn_;
    const Operand& o = b.half[1];
    const uint64_t at = n * C::kElemBytes;
    base = o.base + at;
    left = (o.rows - 1) * o.stride * C::kElemBytes + o.cols * C::kElemBytes - at;
  }
  __device__ inline void shift(uint64_t bytes) {
    first.base += bytes;
    base += bytes;
  }
  __device__ inline void copy(uint32_t lds, int h, uint32_t t, int wave) const {
    Copier<C, false> from = first;
    const bool second = t >= turn;
    from.base = second ? base : first.base;
    from.left = second ? left : first.left;
    from.copy(lds, h, second ? t - turn : t, wave);
  }
};

struct GatedDxArgs {
  Operand a;      // dz and dv side by side
  PairOperand b;  // the weights, rows equally far apart
  Epilogue e;
  uint32_t turn;  // blocks of 64 of one weight's rows
  uint32_t tiles_m, tiles_n;
};

// dx = dz wg + dv wu: one product whose k runs over both, so that no sums are
// written and read again in between.  8192 x 8192 x 4096 bf16: 746 to 777 us
// (1415 to 1470 TFLOP/s), bounded as linear_big.
template <class C>
__global__ __launch_bounds__(512, 2) void gated_dx_big(const GatedDxArgs args) {
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int wm = wave >> 2, wn = wave & 3;
  const TileAt at(xcd_run(blockIdx.x, args.tiles_m * args.tiles_n), args.tiles_m, args.tiles_n);
  const uint64_t m0 = static_cast<uint64_t>(at.m) * 256, n0 = static_cast<uint64_t>(at.n) * 256;
  Copier<C, true> ca;
  ChainCopier<C> cb;
  ca.init(args.a, m0, args.a.cols, 2 * args.turn, wave);
  cb.init(args.b, n0, args.turn, wave);
  f32x4 acc[4][4][2];
  big_sums<C, true, false>(ca, cb, 2 * args.turn, wave, acc);
  finish_all<C, true>(args.e, acc, [&](int p) {
    return Corner{m0 + (p >> 1) * 128 + wm * 64, n0 + (p & 1) * 128 + wn * 32};
  });
}

// A gradient's sums, or those of one share of k.
template <class At>
__device__ inline void finish_share(const Epilogue& e, uint32_t share, const f32x4 (&acc)[4][4][2], At&& at) {
  if (!e.partial) return finish_all<F32, true>(e, acc, at);
  using G = Groups<F32, 4, 2>;
#pragma unroll
  for (int p = 0; p < 4; ++p)
#pragma unroll
    for (int q = 0; q < G::kCount; ++q) {
      float v[4];
      G::sums(acc[p], q, v);
      keep_partial<F32>(e, share, G::row(at(p).first, q), G::column(at(p).second, q), v);
    }
}

// The same of binary32 operands in parts; a[h] and b are the operands themselves.
struct GatedDxPartsArgs {
  GatedDxArgs parts;
  PartsOf of;
  Operand a[2];
  PairOperand b;
  uint64_t k;  // of one weight
};

__global__ __launch_bounds__(512, 2) void gated_dx_parts_big(const GatedDxPartsArgs args) {
  const auto& t = args.parts;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int wm = wave >> 2, wn = wave & 3;
  const uint32_t tiles = t.tiles_m * t.tiles_n, id = xcd_run(blockIdx.x, gridDim.x);
  const TileAt at(id % tiles, t.tiles_m, t.tiles_n);
  const ShareOf share(args.of, id / tiles);
  const uint64_t m0 = static_cast<uint64_t>(at.m) * 256, n0 = static_cast<uint64_t>(at.n) * 256;
  PartCopier<Copier<BF16, true>> ca;
  PartCopier<ChainCopier<BF16>> cb;
  ca.in.init(t.a, m0, t.a.cols, 2 * t.turn, wave);
  cb.in.init(t.b, n0, t.turn, wave);
  take_parts(ca, cb, args.of, share);
  f32x4 acc[4][4][2];
  big_sums<BF16, true, false>(ca, cb, kPairs * share.count, wave, acc);
  auto corner = [&](int p) { return Corner{m0 + (p >> 1) * 128 + wm * 64, n0 + (p & 1) * 128 + wn * 32}; };
  finish_parts<true, false>(
      acc, t.e.m, t.e.n, args.k, t.turn, share, corner, [&](int h) -> const Operand& { return args.a[h]; },
      [&](int h, int) -> const Operand& { return args.b.half[h]; });
  finish_share(t.e, id / tiles, acc, corner);
}

// The weights' gradients, those of the two that are wanted, of binary32 operands
// in parts.
struct GatedDwPartsArgs {
  Operand a[2], b;    // parts of dz, dv and x
  Epilogue e[2];
  uint32_t count;
  PartsOf of;
  Operand a32[2], b32;
  uint64_t k;
  uint32_t tiles_m, tiles_n;  // of one gradient
};

__global__ __launch_bounds__(512, 2) void gated_dw_parts_big(const GatedDwPartsArgs args) {
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int wm = wave >> 2, wn = wave & 3;
  const uint32_t tiles = args.tiles_m * args.tiles_n, id = xcd_run(blockIdx.x, gridDim.x), h = id / tiles % args.count;
  const TileAt at(id % tiles, args.tiles_m, args.tiles_n);
  const ShareOf share(args.of, id / (args.count * tiles));
  const uint64_t m0 = static_cast<uint64_t>(at.m) * 256, n0 = static_cast<uint64_t>(at.n) * 256;
  PartCopier<Copier<BF16, false>> ca, cb;
  ca.in.init(args.a[h], m0, args.k, args.of.blocks, wave);
  cb.in.init(args.b, n0, args.k, args.of.blocks, wave);
  take_parts(ca, cb, args.of, share);
  f32x4 acc[4][4][2];
  big_sums<BF16, false, false>(ca, cb, kPairs * share.count, wave, acc);
  auto corner = [&](int p) { return Corner{m0 + (p >> 1) * 128 + wm * 64, n0 + (p & 1) * 128 + wn * 32}; };
  finish_parts<false, false>(
      acc, args.e[h].m, args.e[h].n, args.k, args.of.blocks, share, corner, [&](int) -> const Operand& { return args.a32[h]; },
      [&](int, int) -> const Operand& { return args.b32; });
  finish_share(args.e[h], id / (args.count * tiles), acc, corner);
}

// A gradient's sums, whose last tile of columns ends where the matrix does.
struct Fitted : Epilogue {
  static constexpr bool kFit = true;
};
using FittedArgs = TileArgsOf<Operand, Fitted>;

template <class C, bool kPlain, int kM, int kN>
__device__ inline void finish_tile(const Fitted& e, uint64_t share, const f32x4 (&acc)[1][kM][kN], uint64_t m0,
                                   uint64_t n0) {
  finish_tile<C, kPlain>(static_cast<const Epilogue&>(e), share, acc, m0, n0);
}

// The same of a wave some of whose columns, those before `own`, are the tile
// before's to store: element by element.  One wave of two at most a row of tiles.
template <class C, bool kPlain, int kM, int kN>
__device__ inline void finish_tile(const Fitted& e, uint64_t share, const f32x4 (&acc)[1][kM][kN], uint64_t m0, uint64_t n0,
                                   uint64_t own) {
  using G = Groups<C, kM, kN>;
  if (n0 + 16 * kN <= own) return;
#pragma unroll
  for (int q = 0; q < G::kCount; ++q) {
    const uint64_t m = G::row(m0, q), n = G::column(n0, q);
    float v[C::V];
    G::sums(acc[0], q, v);
    if (m >= e.m) continue;
#pragma unroll
    for (int c = 0; c < C::V; ++c) {
      if (n + c < own || n + c >= e.n) continue;
      if (e.partial)
        e.partial[(share * e.m + m) * e.partial_stride + n + c] = v[c];
      else
        reinterpret_cast<typename C::Bits*>(e.y)[m * e.y_stride + n + c] = C::narrow(v[c]);
    }
  }
}

// Tiles of the three products and the bias gradients' last sums in one launch:
// small products leave the device half empty, and each launch costs 3 us on the
// host.  515 x 1025 x 770 fp16: 20 us, 32 x 54 -> 189 bf16 8 us.
// A tile of dx walks over both weights, or, where there are few tiles, over a
// share of one of them: dx[h] then writes shares of its own.
struct GatedBackArgs {
  FittedArgs dx[2], dw[2];
  JoinArgs db;
  uint32_t dx_tiles, dx_groups;  // groups of one of the two: tiles x shares
  uint32_t dw_tiles, dw_groups, dw_count;  // dw_count: of the two, those that are wanted
  uint32_t db_blocks;
  uint32_t dx_parts;  // 2; 1: both weights in one tile
};

template <class C, int kBM, int kBN>
__global__ __launch_bounds__(256, 2) void gated_back(const GatedBackArgs p) {
  extern __shared__ __align__(16) char lds[];
  uint32_t id = blockIdx.x;
  if (id < p.dx_parts * p.dx_groups) {
    id = xcd_run(id, p.dx_parts * p.dx_groups);
    const uint32_t h = id / p.dx_groups, r = id % p.dx_groups;
    any_tile<C, true, false, kBM, kBN>(p.dx[h], r % p.dx_tiles, r / p.dx_tiles, lds, 3 - static_cast<int>(p.dx_parts));
    return;
  }
  id -= p.dx_parts * p.dx_groups;
  if (id < p.dw_count * p.dw_groups) {
    id = xcd_run(id, p.dw_count * p.dw_groups);
    const uint32_t h = id / p.dw_groups, r = id % p.dw_groups;
    any_tile<C, false, false, kBM, kBN>(p.dw[h], r % p.dw_tiles, r / p.dw_tiles, lds);
    return;
  }
  id -= p.dw_count * p.dw_groups;
  join_block<C>(p.db, id % p.db_blocks, id / p.db_blocks);
}

struct GatedJoinArgs {
  Epilogue e[3];
  uint32_t shares[3];
  uint32_t groups[3];  // workgroups of each; 0: nothing to join
};

template <class C>
__global__ __launch_bounds__(256) void gated_join(const GatedJoinArgs p) {
  uint32_t id = blockIdx.x;
  int i = 0;
  while (i < 2 && id >= p.groups[i]) id -= p.groups[i++];
  const Epilogue& e = p.e[i];
  constexpr int V = C::V;
  const uint64_t per_row = (e.n + V - 1) / V, at = static_cast<uint64_t>(id) * 256 + threadIdx.x;
  if (at >= per_row * e.m) return;
  const uint64_t m = at / per_row, n = at % per_row * V;
  f32x4 s[V / 4];
  add_shares<V / 4>(e.partial + m * e.partial_stride + n, e.m * e.partial_stride, static_cast<int>(p.shares[i]), s);
  float v[V];
#pragma unroll
  for (int c = 0; c < V; ++c) v[c] = s[c / 4][c % 4];
  store_row<C>(e.y, e.y_stride, m, n, e.m, e.n, v);
}

}  // namespace mscl
