// Kernels of the gated feed-forward block and of 8-bit products on gfx950.
//
// The products are those of linear.hpp, with its tiles, copies and splits of k;
// here are the other weights they take and what becomes of their sums:
//
//   gated    y = act(x wg^T + bg) * (x wu^T + bu).  A tile has the same columns
//            of both weights, and a lane ends up with both sums of its columns
//            (PairOperand), so the product of the two never leaves registers.
//   8 bits   v_mfma_i32_16x16x64_i8: an operand register holds 16 bytes of 16
//            rows, as for 16 bits, and has twice as many k; sums are exact
//            32-bit integers (k up to 131071) and become (sum * row's scale) *
//            column's scale in binary32.
//
//   forward_big    256 x 256 (256 x 128 + 128) tiles of large products
//   forward_tile   small tiles of any size, stride and alignment
//   forward_few    up to 32 rows
//   forward_join   adds the shares of k of the two above
//   gated_slope    both sums' gradients, side by side in the workspace, and the
//                  bias gradients' partial sums
//   gated_dx_big   input gradient, one product over both weights
//   gated_back     tiles of all three products in one launch
//   quantize_rows  a row's largest size, its scale and its 8-bit integers
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "../../include/mscl.h"
#include "codec.hpp"
#include "linear.hpp"

namespace mscl {

// ------------------------------------------------------------------ epilogues

// One 8-bit product: + bias, activation, + residual, rounded to Out.
template <class Out>
struct Scaled : Epilogue {
  using Type = Out;
  static constexpr int kParts = 1;
  const float* row_scale;
  const float* col_scale;
  __device__ inline const float* scale_of(int) const { return col_scale; }
};

// A pair of products, gate first.  The scales are of 8-bit operands.
template <class Out>
struct Gated {
  using Type = Out;
  static constexpr int kParts = 2;
  const char* bias[2];
  char* y;
  char* z[2];  // the sums with their biases, kept for a backward pass, or null
  float* partial;
  uint64_t y_stride, z_stride[2], partial_stride;
  uint64_t m, n;
  int act;
  const float* row_scale;
  const float* col_scale[2];
  __device__ inline const float* scale_of(int p) const { return col_scale[p]; }
};

// The element type of an epilogue's results.
template <class E>
using OutOf = typename E::Type;

// V neighbouring values of a column's vector from column n on.
template <class T>
__device__ inline u32x4 column_values(const char* base, uint64_t n, uint64_t end) {
  if (!base || n >= end) return u32x4{0u, 0u, 0u, 0u};
  return load_upto<T>(base + n * T::kElemBytes, end - n < T::V ? static_cast<int>(end - n) : T::V);
}

// What V columns need of one part, fetched before the sums are at hand.
template <class C, class Out>
struct Columns {
  static constexpr int V = Out::V;
  u32x4 bias;
  u32x4 scale[C::kElemBytes == 1 ? V / 4 : 1];

  __device__ inline void fetch(const char* bias_, const float* scale_, uint64_t n, uint64_t end) {
    bias = column_values<Out>(bias_, n, end);
    if constexpr (C::kElemBytes == 1)
#pragma unroll
      for (int i = 0; i < V; i += 4) scale[i / 4] = column_values<F32>(reinterpret_cast<const char*>(scale_), n + i, end);
  }
  // Sums (of integers, their bits) to values, bias and all.
  __device__ inline void apply(float* v, float row_scale, bool with_bias) const {
    if constexpr (C::kElemBytes == 1)
#pragma unroll
      for (int i = 0; i < V; ++i) {
        const uint32_t s = scale[i / 4][i % 4];
        v[i] = static_cast<float>(__builtin_bit_cast(int32_t, v[i])) * row_scale * __builtin_bit_cast(float, s);
      }
    if (with_bias) {
      float b[V];
      Out::unpack(bias, b);
#pragma unroll
      for (int i = 0; i < V; ++i) v[i] += b[i];
    }
  }
};

template <class C, class E>
__device__ inline float row_scale_of(const E& e, uint64_t m) {
  if constexpr (C::kElemBytes == 1) return m < e.m ? e.row_scale[m] : 0.0f;
  return 1.0f;
}

template <class Out>
__device__ inline void store_row(char* base, uint64_t stride, uint64_t m, uint64_t n, uint64_t rows, uint64_t cols,
                                 const float* v) {
  if (m < rows && n < cols)
    store_upto<Out>(base + (m * stride + n) * Out::kElemBytes, v, cols - n < Out::V ? static_cast<int>(cols - n) : Out::V);
}

// One group of V columns: v (and w, of the second part) are the finished sums.
template <int kAct, class Out>
__device__ inline void finish_group(const Scaled<Out>& e, uint64_t m, uint64_t n, float* v, const float*,
                                    const u32x4& residual) {
#pragma unroll
  for (int i = 0; i < Out::V; ++i) v[i] = activate<kAct, Out::kElemBytes == 2>(v[i]);
  keep_result<Out>(e, m, n, v, residual);
}
template <int kAct, class Out>
__device__ inline void finish_group(const Gated<Out>& e, uint64_t m, uint64_t n, float* v, const float* w, const u32x4&) {
  if (e.z[0]) store_row<Out>(e.z[0], e.z_stride[0], m, n, e.m, e.n, v);
  if (e.z[1]) store_row<Out>(e.z[1], e.z_stride[1], m, n, e.m, e.n, w);
#pragma unroll
  for (int i = 0; i < Out::V; ++i) v[i] = activate<kAct, Out::kElemBytes == 2>(v[i]) * w[i];
  store_row<Out>(e.y, e.y_stride, m, n, e.m, e.n, v);
}

template <class Out>
__device__ inline const char* bias_of(const Scaled<Out>& e, int) {
  return e.bias;
}
template <class Out>
__device__ inline const char* bias_of(const Gated<Out>& e, int p) {
  return e.bias[p];
}
template <class Out>
__device__ inline u32x4 residual_of(const Scaled<Out>& e, uint64_t m, uint64_t n) {
  return fetch_residual<Out>(e, m, n);
}
template <class Out>
__device__ inline u32x4 residual_of(const Gated<Out>&, uint64_t, uint64_t) {
  return u32x4{0u, 0u, 0u, 0u};
}

// All of it for one group whose sums (integers as their bits) are at hand.
template <class C, class E>
__device__ inline void finish_one(const E& e, uint64_t m, uint64_t n, float (&v)[E::kParts][OutOf<E>::V]) {
  using Out = OutOf<E>;
  const float rs = row_scale_of<C>(e, m);
  const u32x4 residual = residual_of(e, m, n);
#pragma unroll
  for (int p = 0; p < E::kParts; ++p) {
    Columns<C, Out> c;
    c.fetch(bias_of(e, p), e.scale_of(p), n, e.n);
    c.apply(v[p], rs, bias_of(e, p) != nullptr);
  }
  with_activation(e.act, [&](auto act) {
    finish_group<decltype(act)::value>(e, m, n, v[0], v[E::kParts - 1], residual);
  });
}

// A wave's blocks of tiles: kBlocks of them, block b of part p in acc(b, p), at
// at(b).  A column's bias and scale are fetched once for all of its rows.
template <class C, int kM, int kN, int kBlocks, class E, class Acc, class At>
__device__ inline void finish_blocks(const E& e, Acc&& acc, At&& at) {
  using Out = OutOf<E>;
  using G = Groups<Out, kM, kN>;
  with_activation(e.act, [&](auto act) {
#pragma unroll
    for (int b = 0; b < kBlocks; ++b) {
      Columns<C, Out> c[E::kParts][G::kPerRow];
      u32x4 residual[G::kCount];
      float rs[G::kCount / G::kPerRow];
#pragma unroll
      for (int q = 0; q < G::kPerRow; ++q)
#pragma unroll
        for (int p = 0; p < E::kParts; ++p)
          c[p][q].fetch(bias_of(e, p), e.scale_of(p), G::column(at(b).second, q), e.n);
#pragma unroll
      for (int q = 0; q < G::kCount; ++q) {
        residual[q] = residual_of(e, G::row(at(b).first, q), G::column(at(b).second, q));
        if (q % G::kPerRow == 0) rs[q / G::kPerRow] = row_scale_of<C>(e, G::row(at(b).first, q));
      }
#pragma unroll
      for (int q = 0; q < G::kCount; ++q) {
        float v[E::kParts][Out::V];
#pragma unroll
        for (int p = 0; p < E::kParts; ++p) {
          G::sums(acc(b, p), q, v[p]);
          c[p][q % G::kPerRow].apply(v[p], rs[q / G::kPerRow], bias_of(e, p) != nullptr);
        }
        finish_group<decltype(act)::value>(e, G::row(at(b).first, q), G::column(at(b).second, q), v[0],
                                           v[E::kParts - 1], residual[q]);
      }
    }
  });
}

// V neighbouring sums of one share of k (integers as their bits).  A partial
// row holds one part's columns after the other's, each padded to whole groups.
template <class E>
__device__ inline float* partial_at(const E& e, uint64_t share, uint64_t m, uint64_t n, int p) {
  return e.partial + (share * e.m + m) * e.partial_stride + p * (e.partial_stride / E::kParts) + n;
}
template <class E>
__device__ inline void keep_share(const E& e, uint64_t share, uint64_t m, uint64_t n, int p, const float* v) {
  if (m >= e.m || n >= e.n) return;
  float* to = partial_at(e, share, m, n, p);
#pragma unroll
  for (int i = 0; i < OutOf<E>::V; i += 4) *reinterpret_cast<f32x4*>(to + i) = f32x4{v[i], v[i + 1], v[i + 2], v[i + 3]};
}

// What linear.hpp's tiles call for these epilogues.
template <class C, bool kPlain, int kM, int kN, class E>
__device__ inline void finish_tile(const E& e, uint64_t share, const Sums<C> (&acc)[E::kParts][kM][kN], uint64_t m0,
                                   uint64_t n0) {
  using G = Groups<OutOf<E>, kM, kN>;
  if (e.partial) {
#pragma unroll
    for (int p = 0; p < E::kParts; ++p)
#pragma unroll
      for (int q = 0; q < G::kCount; ++q) {
        float v[OutOf<E>::V];
        G::sums(acc[p], q, v);
        keep_share(e, share, G::row(m0, q), G::column(n0, q), p, v);
      }
    return;
  }
  finish_blocks<C, kM, kN, 1>(
      e, [&](int, int p) -> const Sums<C>(&)[kM][kN] { return acc[p]; }, [&](int) { return Corner{m0, n0}; });
}

template <class C, int kM, int kN, class E, int kSize>
__device__ inline void finish_few(const E& e, const SumOf<C> (&sums)[4][kSize], uint64_t n0) {
  constexpr int V = OutOf<E>::V;
  constexpr int kPitch = 16 * kN + 4, kColumns = 16 * kN / E::kParts;
  for (int id = threadIdx.x; id < 16 * kM * kColumns / V; id += 512) {
    const int m = id / (kColumns / V), n = id % (kColumns / V) * V;
    float v[E::kParts][V];
#pragma unroll
    for (int p = 0; p < E::kParts; ++p)
#pragma unroll
      for (int c = 0; c < V; ++c) {
        const int at = m * kPitch + p * kColumns + n + c;
        const SumOf<C> s = (sums[0][at] + sums[1][at]) + (sums[2][at] + sums[3][at]);
        v[p][c] = __builtin_bit_cast(float, s);
      }
    if (!e.partial) {
      finish_one<C>(e, m, n0 + n, v);
      continue;
    }
#pragma unroll
    for (int p = 0; p < E::kParts; ++p) keep_share(e, blockIdx.y, m, n0 + n, p, v[p]);
  }
}

// ------------------------------------------------------------------ forward kernels

template <class C, int kBM, int kBN, class B, class E>
__global__ __launch_bounds__(256, 2) void forward_tile(const TileArgsOf<B, E> t) {
  extern __shared__ __align__(16) char lds[];
  const uint32_t id = xcd_run(blockIdx.x, gridDim.x), tiles = t.tiles_m * t.tiles_n;
  any_tile<C, true, true, kBM, kBN>(t, id % tiles, id / tiles, lds);
}

template <class C, int kM, int kN, int kDeep, class B, class E>
__global__ __launch_bounds__(512) void forward_few(const TileArgsOf<B, E> t) {
  few_body<C, kM, kN, kDeep>(t);
}

// Adds the shares of k in their order and finishes a group of V columns.
template <class C, class E>
__global__ __launch_bounds__(256) void forward_join(const E e, int shares) {
  constexpr int V = OutOf<E>::V;
  const uint64_t per_row = (e.n + V - 1) / V, id = static_cast<uint64_t>(blockIdx.x) * 256 + threadIdx.x;
  if (id >= per_row * e.m) return;
  const uint64_t m = id / per_row, n = id % per_row * V;
  Sums<C> s[E::kParts][V / 4];
#pragma unroll
  for (int p = 0; p < E::kParts; ++p)
#pragma unroll
    for (int i = 0; i < V / 4; ++i) s[p][i] = Sums<C>{0, 0, 0, 0};
  for (int share = 0; share < shares; ++share)
#pragma unroll
    for (int p = 0; p < E::kParts; ++p)
#pragma unroll
      for (int i = 0; i < V / 4; ++i)
        s[p][i] += *reinterpret_cast<const Sums<C>*>(partial_at(e, share, m, n, p) + 4 * i);
  float v[E::kParts][V];
#pragma unroll
  for (int p = 0; p < E::kParts; ++p)
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const SumOf<C> one = s[p][i / 4][i % 4];
      v[p][i] = __builtin_bit_cast(float, one);
    }
  finish_one<C>(e, m, n, v);
}

// The copies of a pair of weights whose rows are equally far apart: half h of a
// block is 128 rows of weight h.
template <class C>
struct PairCopier {
  Copier<C, true> gate;
  const char* base;  // of the second weight's tile
  uint64_t left;

  __device__ inline void init(const PairOperand& b, uint64_t first, uint64_t k, uint32_t blocks, int wave) {
    gate.init(b.half[0], first, k, blocks, wave);
    const Operand& o = b.half[1];
    const uint64_t at = first * gate.stride;
    base = o.base + at;
    left = (o.rows - 1) * gate.stride + o.cols * C::kElemBytes - at;
  }
  __device__ inline void copy(uint32_t lds, int h, uint32_t t, int wave) const {
    Copier<C, true> from = gate;
    if (h) {
      from.base = base;
      from.left = left;
    }
    from.copy(lds, 0, t, wave);
  }
};
template <class C>
__device__ inline Copier<C, true> copier_of(const Operand&) {
  return {};
}
template <class C>
__device__ inline PairCopier<C> copier_of(const PairOperand&) {
  return {};
}

// linear.hpp's 256 x 256 tiles with these operands and epilogues.  Of a pair a
// tile has 128 columns of each weight, in quarters (i, 0) and (i, 1).
template <class C, class B, class E>
__global__ __launch_bounds__(512, 2) void forward_big(const BigArgsOf<B, E> args) {
  extern __shared__ __align__(16) char lds[];
  constexpr int kParts = B::kParts;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int wm = wave >> 2, wn = wave & 3;
  const TileAt at(xcd_run(blockIdx.x, args.tiles_m * args.tiles_n), args.tiles_m, args.tiles_n);
  const uint64_t m0 = static_cast<uint64_t>(at.m) * 256, n0 = static_cast<uint64_t>(at.n) * (256 / kParts);
  constexpr int kBlock = 8 * C::V;
  const uint32_t blocks = static_cast<uint32_t>((args.k + kBlock - 1) / kBlock);
  Copier<C, true> ca;
  auto cb = copier_of<C>(args.b);
  ca.init(args.a, m0, args.k, blocks, wave);
  cb.init(args.b, n0, args.k, blocks, wave);
  Sums<C> acc[4][4][2];
  big_sums<C, true, true>(ca, cb, blocks, lds, wave, acc);
  // block b is quarter b, or with a pair quarters (b, 0) and (b, 1)
  finish_blocks<C, 4, 2, 4 / kParts>(
      args.e, [&](int b, int p) -> const Sums<C>(&)[4][2] { return acc[kParts * b + p]; },
      [&](int b) {
        const int i = kParts == 1 ? b >> 1 : b, j = kParts == 1 ? b & 1 : 0;
        return Corner{m0 + i * 128 + wm * 64, n0 + j * 128 + wn * 32};
      });
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
      for (uint64_t m0 = first + wave; m0 < end; m0 += 4 * kRows) {
        u32x4 dy[kRows], z[kRows], v[kRows];
#pragma unroll
        for (int q = 0; q < kRows; ++q) {
          const uint64_t m = m0 + 4 * q < end ? m0 + 4 * q : end - 1;
          const int there = kFull ? V : valid;
          dy[q] = load_upto<C>(a.dy + (m * a.dy_stride + n) * C::kElemBytes, there);
          z[q] = load_upto<C>(a.z + (m * a.z_stride + n) * C::kElemBytes, there);
          v[q] = load_upto<C>(a.v + (m * a.v_stride + n) * C::kElemBytes, there);
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
// and then the second's, `turn` blocks each: rows past a weight's end read as 0.
template <class C>
struct ChainCopier {
  Copier<C, false> first;
  const char* base;  // of the second weight's tile
  uint64_t left;
  uint32_t turn;

  __device__ inline void init(const PairOperand& b, uint64_t n, uint32_t turn_, int wave) {
    first.init(b.half[0], n, 0, turn_, wave);
    turn = turn_;
    const Operand& o = b.half[1];
    const uint64_t at = n * C::kElemBytes;
    base = o.base + at;
    left = (o.rows - 1) * o.stride * C::kElemBytes + o.cols * C::kElemBytes - at;
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

// dx = dz wg + dv wu: one product whose k runs over both.
template <class C>
__global__ __launch_bounds__(512, 2) void gated_dx_big(const GatedDxArgs args) {
  extern __shared__ __align__(16) char lds[];
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int wm = wave >> 2, wn = wave & 3;
  const TileAt at(xcd_run(blockIdx.x, args.tiles_m * args.tiles_n), args.tiles_m, args.tiles_n);
  const uint64_t m0 = static_cast<uint64_t>(at.m) * 256, n0 = static_cast<uint64_t>(at.n) * 256;
  Copier<C, true> ca;
  ChainCopier<C> cb;
  ca.init(args.a, m0, args.a.cols, 2 * args.turn, wave);
  cb.init(args.b, n0, args.turn, wave);
  f32x4 acc[4][4][2];
  big_sums<C, true, false>(ca, cb, 2 * args.turn, lds, wave, acc);
  finish_all<C, true>(args.e, acc, [&](int p) {
    return Corner{m0 + (p >> 1) * 128 + wm * 64, n0 + (p & 1) * 128 + wn * 32};
  });
}

// Tiles of the three products and the bias gradients' last sums in one launch.
// dx is summed over shares of k of either weight: dx[h] writes its own shares.
struct GatedBackArgs {
  TileArgs dx[2], dw[2];
  JoinArgs db;
  uint32_t dx_tiles, dx_groups;  // groups of one of the two: tiles x shares
  uint32_t dw_tiles, dw_groups;
  uint32_t db_blocks;
};

template <class C, int kBM, int kBN>
__global__ __launch_bounds__(256, 2) void gated_back(const GatedBackArgs p) {
  extern __shared__ __align__(16) char lds[];
  uint32_t id = blockIdx.x;
  if (id < 2 * p.dx_groups) {
    id = xcd_run(id, 2 * p.dx_groups);
    const uint32_t h = id / p.dx_groups, r = id % p.dx_groups;
    any_tile<C, true, false, kBM, kBN>(p.dx[h], r % p.dx_tiles, r / p.dx_tiles, lds);
    return;
  }
  id -= 2 * p.dx_groups;
  if (id < 2 * p.dw_groups) {
    id = xcd_run(id, 2 * p.dw_groups);
    const uint32_t h = id / p.dw_groups, r = id % p.dw_groups;
    any_tile<C, false, false, kBM, kBN>(p.dw[h], r % p.dw_tiles, r / p.dw_tiles, lds);
    return;
  }
  id -= 2 * p.dw_groups;
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
  join_shares<C>(p.e[i], static_cast<int>(p.shares[i]), static_cast<uint64_t>(id) * 256 + threadIdx.x);
}

// ------------------------------------------------------------------ rows to 8 bits

struct QuantizeArgs {
  const char* x;
  int8_t* q;
  float* scale;
  uint64_t x_stride, q_stride;
  uint64_t rows, width;
};

// A row's largest size counts as at least this when its scale is chosen, so
// that neither the scale nor 127 over the size leaves the normal numbers.
constexpr float kLeastSize = 0x1p-100f;

// 16 elements, the last of a row fewer.
template <class C>
struct Sixteen {
  static constexpr int kVecs = 16 / C::V;
  u32x4 v[kVecs];

  __device__ inline void load(const char* p, int valid) {
#pragma unroll
    for (int i = 0; i < kVecs; ++i) v[i] = load_upto<C>(p + 16 * i, valid - i * C::V);
  }
  __device__ inline void values(float (&f)[16]) const {
#pragma unroll
    for (int i = 0; i < kVecs; ++i) C::unpack(v[i], f + i * C::V);
  }
  // The largest size's bits: NaN above infinity above all numbers.
  __device__ inline uint32_t largest() const {
    float f[16];
    values(f);
    uint32_t most = 0;
#pragma unroll
    for (int i = 0; i < 16; ++i) most = max(most, __builtin_bit_cast(uint32_t, f[i]) & 0x7fffffffu);
    return most;
  }
  // rint(x by) of each, 4 to a register.
  __device__ inline u32x4 integers(float by) const {
    float f[16];
    values(f);
    u32x4 o = {0u, 0u, 0u, 0u};
#pragma unroll
    for (int i = 0; i < 16; ++i)
      o[i / 4] |= (static_cast<uint32_t>(static_cast<int32_t>(rintf(f[i] * by))) & 0xffu) << (8 * (i % 4));
    return o;
  }
};

// 127 / size and size / 127 of a row, from its largest size's bits.  A row with
// an infinity or NaN has the scale NaN, and 0 for its integers.
struct RowScale {
  float by, scale;
  bool finite;
  __device__ inline explicit RowScale(uint32_t most) {
    finite = most < 0x7f800000u;
    const float size = fmaxf(__builtin_bit_cast(float, most), kLeastSize);
    by = 127.0f / size;
    scale = finite ? size / 127.0f : __builtin_nanf("");
  }
};

__device__ inline void store_integers(int8_t* q, const u32x4& v, int valid) {
  if (valid >= 16) {
    *reinterpret_cast<u32x4_by1*>(q) = v;
    return;
  }
#pragma unroll
  for (int i = 0; i < 16; ++i)
    if (i < valid) q[i] = static_cast<int8_t>(v[i / 4] >> (8 * (i % 4)));
}

// The largest of kThreads threads' values, in all of them.
template <int kThreads>
__device__ inline uint32_t largest_of(uint32_t v, uint32_t* lds) {
#pragma unroll
  for (int d = 32; d >= 1; d >>= 1) v = max(v, static_cast<uint32_t>(__shfl_xor(static_cast<int>(v), d)));
  if constexpr (kThreads > 64) {
    const int wave = threadIdx.x >> 6;
    if ((threadIdx.x & 63) == 0) lds[wave] = v;
    __syncthreads();
    v = lds[0];
#pragma unroll
    for (int i = 1; i < kThreads / 64; ++i) v = max(v, lds[i]);
  }
  return v;
}

// A row by kThreads threads, held in registers, kChunks times 16 elements each.
template <class C, int kThreads, int kChunks>
__global__ __launch_bounds__(kThreads < 256 ? 256 : kThreads) void quantize_rows(const QuantizeArgs a) {
  constexpr int kBlock = kThreads < 256 ? 256 : kThreads;
  constexpr int kRows = kBlock / kThreads;
  static_assert(kThreads == 64 || kRows == 1, "a row is a wave's or a workgroup's");
  __shared__ uint32_t lds[kBlock / 64];
  const uint64_t row = static_cast<uint64_t>(blockIdx.x) * kRows + threadIdx.x / kThreads;
  if (row >= a.rows) return;  // whole waves, and whole workgroups where they meet in LDS
  const int t = threadIdx.x % kThreads;
  const char* x = a.x + row * a.x_stride * C::kElemBytes;
  int8_t* q = a.q + row * a.q_stride;
  Sixteen<C> held[kChunks];
#pragma unroll
  for (int i = 0; i < kChunks; ++i) {
    const uint64_t n = (static_cast<uint64_t>(i) * kThreads + t) * 16;
    const int valid = n >= a.width ? 0 : (a.width - n < 16 ? static_cast<int>(a.width - n) : 16);
    held[i].load(x + n * C::kElemBytes, valid);
  }
  uint32_t most = 0;
#pragma unroll
  for (int i = 0; i < kChunks; ++i) most = max(most, held[i].largest());
  const RowScale s(largest_of<kThreads>(most, lds));
#pragma unroll
  for (int i = 0; i < kChunks; ++i) {
    const uint64_t n = (static_cast<uint64_t>(i) * kThreads + t) * 16;
    const int valid = n >= a.width ? 0 : (a.width - n < 16 ? static_cast<int>(a.width - n) : 16);
    const u32x4 none = {0u, 0u, 0u, 0u};
    if (valid > 0) store_integers(q + n, s.finite ? held[i].integers(s.by) : none, valid);
  }
  if (t == 0) a.scale[row] = s.scale;
}

// Rows too wide for the registers: read twice.
template <class C>
__global__ __launch_bounds__(1024) void quantize_wide(const QuantizeArgs a) {
  __shared__ uint32_t lds[16];
  const uint64_t row = blockIdx.x;
  const char* x = a.x + row * a.x_stride * C::kElemBytes;
  int8_t* q = a.q + row * a.q_stride;
  uint32_t most = 0;
  Sixteen<C> held;
  for (uint64_t n = threadIdx.x * 16; n < a.width; n += 1024 * 16) {
    held.load(x + n * C::kElemBytes, a.width - n < 16 ? static_cast<int>(a.width - n) : 16);
    most = max(most, held.largest());
  }
  const RowScale s(largest_of<1024>(most, lds));
  for (uint64_t n = threadIdx.x * 16; n < a.width; n += 1024 * 16) {
    const int valid = a.width - n < 16 ? static_cast<int>(a.width - n) : 16;
    held.load(x + n * C::kElemBytes, valid);
    const u32x4 none = {0u, 0u, 0u, 0u};
    store_integers(q + n, s.finite ? held.integers(s.by) : none, valid);
  }
  if (threadIdx.x == 0) a.scale[row] = s.scale;
}

}  // namespace mscl
