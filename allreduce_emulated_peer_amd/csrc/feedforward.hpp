// Forward kernels of the gated feed-forward block and of 8-bit products on gfx950.
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
  static constexpr bool kFit = true;
  const float* row_scale;
  const float* col_scale;
  __device__ inline const float* scale_of(int) const { return col_scale; }
};

// A pair of products, gate first.  The scales are of 8-bit operands.
template <class Out>
struct Gated {
  using Type = Out;
  static constexpr int kParts = 2;
  static constexpr bool kFit = true;
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
__device__ __forceinline__ void finish_one(const E& e, uint64_t m, uint64_t n, float (&v)[E::kParts][OutOf<E>::V]) {
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
__device__ __forceinline__ void finish_blocks(const E& e, Acc&& acc, At&& at) {
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
__device__ __forceinline__ void finish_tile(const E& e, uint64_t share, const Sums<C> (&acc)[E::kParts][kM][kN], uint64_t m0,
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
__device__ __forceinline__ void finish_few(const E& e, const SumOf<C> (&sums)[4][kSize], uint64_t n0) {
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

// Any sizes, strides and alignments.  1024 x 2048 -> 1024 8 bits 9.1 us, pairs of
// bf16 17.5; 1001 x 2047 -> 1537 at odd addresses 20 us (8 bits), pairs of binary32
// 97 us (131 TFLOP/s), where splitting and multiplying share the time.
template <class C, int kBM, int kBN, class B, class E>
__global__ __launch_bounds__(256, 2) void forward_tile(const TileArgsOf<B, E> t) {
  extern __shared__ __align__(16) char lds[];
  const uint32_t id = xcd_run(blockIdx.x, gridDim.x), tiles = t.tiles_m * t.tiles_n;
  any_tile<C, true, true, kBM, kBN>(t, id % tiles, id / tiles, lds);
}

// The pass over the weights bounds it: a pair of bf16 1 x 8192 -> 4096 25 us from
// memory (5.4 TB/s), 8 bits 9.0 (3.7 TB/s), a pair of 8 bits with 32 rows 17.6.
// Twice the loads in flight gained nothing, and cost 4 to 13% at k = 4096.
template <class C, int kM, int kN, int kDeep, class B, class E>
__global__ __launch_bounds__(512) void forward_few(const TileArgsOf<B, E> t) {
  few_body<C, kM, kN, kDeep>(t);
}

// The sums of kGroups times four neighbouring values of the shares, in their
// order, `apart` values between one share and the next; eight shares' loads are
// in flight together.
template <int kGroups, class S>
__device__ inline void add_shares(const float* at, uint64_t apart, int shares, S (&sum)[kGroups]) {
#pragma unroll
  for (int i = 0; i < kGroups; ++i) sum[i] = S{0, 0, 0, 0};
  for (int first = 0; first < shares; first += 8) {
    S held[8][kGroups];
#pragma unroll
    for (int q = 0; q < 8; ++q) {
      const int share = first + q < shares ? first + q : shares - 1;
#pragma unroll
      for (int i = 0; i < kGroups; ++i) held[q][i] = *reinterpret_cast<const S*>(at + share * apart + 4 * i);
    }
#pragma unroll
    for (int q = 0; q < 8; ++q)
      if (first + q < shares)
#pragma unroll
        for (int i = 0; i < kGroups; ++i) sum[i] += held[q][i];
  }
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
    add_shares<V / 4>(partial_at(e, 0, m, n, p), e.m * e.partial_stride, shares, s[p]);
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
  __device__ inline void shift(uint64_t bytes) {
    gate.base += bytes;
    base += bytes;
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
// tile has 128 columns of each weight, in quarters (i, 0) and (i, 1).  What
// bounds it is the matrix units: 8192 x 8192 -> 4096 pairs of bf16 with both sums
// kept 735 to 780 us (1410 to 1500 TFLOP/s, MFMA busy 79% of the cycles), of 8
// bits 370 to 400 us (2.75 to 3.0 POP/s); 8 bits 8192 x 4096 -> 8192 with a
// residual 241 to 252 us, where stores and residual take a fifth.
template <class C, class B, class E>
__global__ __launch_bounds__(512, 2) void forward_big(const BigArgsOf<B, E> args) {
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
  big_sums<C, true, true>(ca, cb, blocks, wave, acc);
  // block b is quarter b, or with a pair quarters (b, 0) and (b, 1)
  finish_blocks<C, 4, 2, 4 / kParts>(
      args.e, [&](int b, int p) -> const Sums<C>(&)[4][2] { return acc[kParts * b + p]; },
      [&](int b) {
        const int i = kParts == 1 ? b >> 1 : b, j = kParts == 1 ? b & 1 : 0;
        return Corner{m0 + i * 128 + wm * 64, n0 + j * 128 + wn * 32};
      });
}

}  // namespace mscl
