// Matrix products of the linear layer and of its backward pass on gfx950.
//
// Every product here is  C[m][n] = sum_k A(m, k) B(n, k)  with binary32 sums:
//   forward            y = x w^T     A = x  (k along its rows)   B = w  (k along its rows)
//   input gradient    dx = dz w      A = dz (k along its rows)   B = w  (k down its columns)
//   weight gradient   dw = dz^T x    A = dz (k down its columns) B = x  (k down its columns)
// An operand whose k runs along its memory rows is kAlong, the other form
// kDown; both are read from memory as they lie, and a kDown tile of 16-bit
// elements is turned while it goes from LDS to registers.
//
// The products run on the matrix units: v_mfma_f32_16x16x32_{bf16,f16} for
// the 16-bit types, and for binary32 too, whose values are split into three
// bfloat16 parts (with few rows, where memory bounds, v_mfma_f32_16x16x4_f32).
// The B tile is given as the instruction's first operand, so a lane ends up
// with four neighbouring columns n of one row m; v_permlane16_swap of two
// neighbouring tiles makes eight, one 16-byte store of a 16-bit type.
//
//   linear_big    256 x 256 tiles of large 16-bit products
//   linear_tile   64 x 64, 128 x 64 and 128 x 128 tiles of all others, of any
//                 size, stride and alignment, k split over workgroups where
//                 the tiles are few (linear_join adds the shares)
//   linear_pair   both gradients' tiles in one launch
//   linear_few    up to 32 rows, but for 17 and more of 16-bit types and 65281 or
//                 more outputs, which linear_big takes
//   linear_slope  dz and the bias gradient's partial sums
//   linear_pack   an operand laid out anew for linear_big
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include <type_traits>

#include "../../include/mscl.h"
#include "codec.hpp"

namespace mscl {

typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef _Float16 f16x8 __attribute__((ext_vector_type(8)));
typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
typedef short s16x4 __attribute__((ext_vector_type(4)));
typedef __attribute__((address_space(3))) s16x4 lds_s16x4;

// 16 bytes at the alignment of one element: gfx950 loads and stores them at
// any element's address with one instruction.
typedef u32x4 u32x4_by2 __attribute__((aligned(2)));
typedef u32x4 u32x4_by4 __attribute__((aligned(4)));

template <class C>
__device__ inline u32x4 load_loose(const char* p) {
  if constexpr (C::kElemBytes == 4) return *reinterpret_cast<const u32x4_by4*>(p);
  return *reinterpret_cast<const u32x4_by2*>(p);
}
template <class C>
__device__ inline void store_loose(char* p, const u32x4& v) {
  if constexpr (C::kElemBytes == 4)
    *reinterpret_cast<u32x4_by4*>(p) = v;
  else
    *reinterpret_cast<u32x4_by2*>(p) = v;
}

// V elements from `p`, of which the first `valid` exist; the others read as 0.
template <class C>
__device__ inline u32x4 load_upto(const char* p, int valid) {
  if (valid >= C::V) return load_loose<C>(p);
  u32x4 v = {0u, 0u, 0u, 0u};
  if (valid > 0) v = load_partial<C>(p, 0, valid);
  return v;
}

// Rounds V values and stores the first `valid` of them.
template <class C>
__device__ inline void store_upto(char* p, const float* v, int valid) {
  const u32x4 b = C::pack(v);
  if (valid >= C::V)
    store_loose<C>(p, b);
  else if (valid > 0)
    store_partial<C>(p, 0, b, valid);
}

// Runs fn with whether a whole workgroup's columns exist as a constant.
template <class Fn>
__device__ inline void with_edges(bool full, Fn&& fn) {
  if (full)
    fn(std::true_type{});
  else
    fn(std::false_type{});
}

// ------------------------------------------------------------------ activations

// Activations and their slopes in binary32.  kFast is taken where the result
// is rounded to 16 bits: the hardware's exp2 and reciprocal (1 ulp each), and
// a polynomial for the Gaussian tail, against roundings of up to 2^-8 (bf16)
// and 2^-11 (fp16) of a result.  binary32 results use the math library.
// The Gaussian tail is computed as erfc(|z|), never as 1 + erf(z), so small
// values at negative z keep their relative accuracy: the polynomial's is 1.2e-5
// of the tail (and 5.6e-7 where the tail is not small), to which exp adds 2^-23
// of its argument, 1e-5 at z = -12.  A tail or sigmoid below 2^-126 may be 0.
template <bool kFast>
__device__ inline float exp_of(float x) {
  if constexpr (kFast) return __builtin_amdgcn_exp2f(x * 1.44269504088896340736f);
  return expf(x);
}
template <bool kFast>
__device__ inline float reciprocal(float x) {
  if constexpr (kFast) return __builtin_amdgcn_rcpf(x);
  return 1.0f / x;
}
template <bool kFast>
__device__ inline float sigmoid(float x) {
  return reciprocal<kFast>(1.0f + exp_of<kFast>(-x));
}

// Phi(z), the normal distribution's integral up to z; *bell = exp(-z^2 / 2).
template <bool kFast>
__device__ inline float normal_cdf(float z, float* bell) {
  *bell = exp_of<kFast>(-0.5f * z * z);
  if constexpr (kFast) {
    // erfc(u) exp(u^2) = t P(t), t = 1 / (1 + 0.425 u).  P is fitted (linear
    // programming over 5000 points of u in [0, 10], for this kernel) so that its
    // relative error is at most 5.6e-7 / erfc(u), and 1.12e-5 far out; with a
    // degree less these are 6.6 times as large.
    const float u = fabsf(z) * 0.70710678118654752440f;
    const float t = __builtin_amdgcn_rcpf(fmaf(0.425f, u, 1.0f));
    float p = fmaf(-0.158399324f, t, 0.44051643f);
    p = fmaf(p, t, -0.0426700415f);
    p = fmaf(p, t, 0.292943433f);
    p = fmaf(p, t, 0.226971731f);
    p = fmaf(p, t, 0.240637183f);
    // t -> 0 and bell -> 0 at infinity, where 0 is the limit
    const float tail = 0.5f * p * t * *bell;
    return z >= 0.0f ? 1.0f - tail : (z < 0.0f ? tail : z);
  }
  return 0.5f * erfcf(-z * 0.70710678118654752440f);
}

constexpr float kTanhScale = 0.79788456080286535588f;  // sqrt(2 / pi)
constexpr float kTanhCubic = 0.044715f;

template <int kAct, bool kFast>
__device__ inline float activate(float z) {
  if constexpr (kAct == MSCL_ACT_RELU) return z > 0.0f ? z : (z <= 0.0f ? 0.0f : z);  // NaN stays NaN
  if constexpr (kAct == MSCL_ACT_GELU) {
    float bell;
    const float p = normal_cdf<kFast>(z, &bell);
    return p == 0.0f ? 0.0f : z * p;  // the limit at -inf
  }
  if constexpr (kAct == MSCL_ACT_GELU_TANH) {
    // 0.5 (1 + tanh u) = sigmoid(2 u)
    const float q = sigmoid<kFast>(2.0f * kTanhScale * (z + kTanhCubic * z * z * z));
    return q == 0.0f ? 0.0f : z * q;
  }
  if constexpr (kAct == MSCL_ACT_SILU) {
    const float q = sigmoid<kFast>(z);
    return q == 0.0f ? 0.0f : z * q;
  }
  return z;
}

template <int kAct, bool kFast>
__device__ inline float slope(float z) {
  if constexpr (kAct == MSCL_ACT_RELU) return z > 0.0f ? 1.0f : 0.0f;
  if constexpr (kAct == MSCL_ACT_GELU) {
    float bell;
    const float p = normal_cdf<kFast>(z, &bell);
    return bell == 0.0f ? p : fmaf(z * 0.39894228040143267794f, bell, p);  // 1 / sqrt(2 pi)
  }
  if constexpr (kAct == MSCL_ACT_GELU_TANH) {
    const float s = sigmoid<kFast>(2.0f * kTanhScale * (z + kTanhCubic * z * z * z));
    const float du = kTanhScale * (1.0f + 3.0f * kTanhCubic * z * z);
    const float bend = 2.0f * s * (1.0f - s);  // 0.5 (1 - tanh^2)
    return bend == 0.0f ? s : fmaf(z * bend, du, s);
  }
  if constexpr (kAct == MSCL_ACT_SILU) {
    const float q = sigmoid<kFast>(z);
    const float bend = q * (1.0f - q);
    return bend == 0.0f ? q : fmaf(z, bend, q);
  }
  return 1.0f;
}

// ------------------------------------------------------------------ epilogue

// What happens to a product's sums: + bias, (kept as z), activation,
// + residual, one rounding to the element type.  `partial` instead takes the
// raw sums of one share of k (rows of `partial_stride` binary32 values, one
// matrix after the other), which linear_join adds up.
struct Epilogue {
  const char* bias;
  const char* residual;
  char* y;
  char* z;
  float* partial;
  uint64_t residual_stride, y_stride, z_stride, partial_stride;
  uint64_t m, n;
  int act;
};

// Runs fn(activation as a constant) for a value known only at run time, so
// that the choice is made once and not for every element.
template <class Fn>
__device__ inline void with_activation(int act, Fn&& fn) {
  switch (act) {
    case MSCL_ACT_RELU: fn(std::integral_constant<int, MSCL_ACT_RELU>{}); break;
    case MSCL_ACT_GELU: fn(std::integral_constant<int, MSCL_ACT_GELU>{}); break;
    case MSCL_ACT_GELU_TANH: fn(std::integral_constant<int, MSCL_ACT_GELU_TANH>{}); break;
    case MSCL_ACT_SILU: fn(std::integral_constant<int, MSCL_ACT_SILU>{}); break;
    default: fn(std::integral_constant<int, MSCL_ACT_NONE>{}); break;
  }
}

// What the epilogue adds to V neighbouring sums.  A wave fetches the residual of
// many tiles before it finishes the first one: fetched one by one, each would
// wait a memory latency behind the stores of the one before (8192 x 4096 x
// 8192 fp16 with a residual: 482 us one by one, 441 us ahead).
template <class C>
__device__ inline u32x4 fetch_bias(const Epilogue& e, uint64_t n) {
  if (!e.bias || n >= e.n) return u32x4{0u, 0u, 0u, 0u};
  return load_upto<C>(e.bias + n * C::kElemBytes, e.n - n < C::V ? static_cast<int>(e.n - n) : C::V);
}
template <class C>
__device__ inline u32x4 fetch_residual(const Epilogue& e, uint64_t m, uint64_t n) {
  if (!e.residual || m >= e.m || n >= e.n) return u32x4{0u, 0u, 0u, 0u};
  return load_upto<C>(e.residual + (m * e.residual_stride + n) * C::kElemBytes,
                      e.n - n < C::V ? static_cast<int>(e.n - n) : C::V);
}

// V neighbouring sums of row m from column n on: + bias, kept as z if wanted.
template <class C>
__device__ inline void keep_preact(const Epilogue& e, uint64_t m, uint64_t n, float* v, const u32x4& bias) {
  if (e.bias) {
    float t[C::V];
    C::unpack(bias, t);
#pragma unroll
    for (int i = 0; i < C::V; ++i) v[i] += t[i];
  }
  if (e.z && m < e.m && n < e.n)
    store_upto<C>(e.z + (m * e.z_stride + n) * C::kElemBytes, v, e.n - n < C::V ? static_cast<int>(e.n - n) : C::V);
}

// V neighbouring activated values: + residual, stored as y.
template <class C>
__device__ inline void keep_result(const Epilogue& e, uint64_t m, uint64_t n, float* v, const u32x4& residual) {
  if (e.residual) {
    float t[C::V];
    C::unpack(residual, t);
#pragma unroll
    for (int i = 0; i < C::V; ++i) v[i] += t[i];
  }
  if (m < e.m && n < e.n)
    store_upto<C>(e.y + (m * e.y_stride + n) * C::kElemBytes, v, e.n - n < C::V ? static_cast<int>(e.n - n) : C::V);
}

// All three steps for one group.
template <class C>
__device__ inline void finish(const Epilogue& e, uint64_t m, uint64_t n, float* v) {
  const u32x4 bias = fetch_bias<C>(e, n), residual = fetch_residual<C>(e, m, n);
  keep_preact<C>(e, m, n, v, bias);
  with_activation(e.act, [&](auto act) {
#pragma unroll
    for (int i = 0; i < C::V; ++i) v[i] = activate<decltype(act)::value, C::kElemBytes == 2>(v[i]);
  });
  keep_result<C>(e, m, n, v, residual);
}

// V neighbouring sums of one share of k.  Partial rows are padded to whole
// 32-byte groups, so the store never needs a bound on n beyond the group's.
template <class C>
__device__ inline void keep_partial(const Epilogue& e, uint64_t share, uint64_t m, uint64_t n, const float* v) {
  if (m >= e.m || n >= e.n) return;
  float* p = e.partial + (share * e.m + m) * e.partial_stride + n;
#pragma unroll
  for (int i = 0; i < C::V; i += 4) *reinterpret_cast<f32x4*>(p + i) = f32x4{v[i], v[i + 1], v[i + 2], v[i + 3]};
}

// Swaps lanes 16..31 (48..63) of a with lanes 0..15 (32..47) of b.
__device__ inline void swap_rows16(float& a, float& b) {
  const auto r = __builtin_amdgcn_permlane16_swap(__builtin_bit_cast(uint32_t, a), __builtin_bit_cast(uint32_t, b), false, false);
  const uint32_t x = r[0], y = r[1];
  a = __builtin_bit_cast(float, x);
  b = __builtin_bit_cast(float, y);
}

// Where the V sums of group q of a wave's kM x kN tiles of 16 x 16 lie (tile
// (i, j) at row m0 + 16 i, column n0 + 16 j).  In tile (i, j) lane l holds row
// l % 16, columns 4 (l / 16) .. + 3; for a 16-bit type two neighbouring tiles
// trade halves, so that each lane holds eight columns.
template <class C, int kM, int kN>
struct Groups {
  static constexpr int kPerRow = C::V == 4 ? kN : kN / 2;
  static constexpr int kCount = kM * kPerRow;
  static_assert(C::V == 4 || kN % 2 == 0, "16-bit tiles come in pairs");

  static __device__ inline uint64_t row(uint64_t m0, int q) { return m0 + 16 * (q / kPerRow) + (threadIdx.x & 15); }
  static __device__ inline uint64_t column(uint64_t n0, int q) {
    const int g = (threadIdx.x & 63) >> 4, j = q % kPerRow;
    if constexpr (C::V == 4) return n0 + 16 * j + 4 * g;
    return n0 + 16 * (2 * j + (g & 1)) + 8 * (g >> 1);
  }
  static __device__ inline void sums(const f32x4 (&acc)[kM][kN], int q, float* v) {
    const int i = q / kPerRow, j = q % kPerRow;
    if constexpr (C::V == 4) {
#pragma unroll
      for (int c = 0; c < 4; ++c) v[c] = acc[i][j][c];
    } else {
#pragma unroll
      for (int c = 0; c < 4; ++c) {
        float a = acc[i][2 * j][c], b = acc[i][2 * j + 1][c];
        swap_rows16(a, b);
        v[c] = a;
        v[4 + c] = b;
      }
    }
  }
};

// Finishes and stores a wave's kParts blocks of tiles, block p at (m0, n0) of
// at(p).  kPlain: a gradient's product, of which nothing but the sums is
// wanted (its kernels have half the code and need fewer registers).
template <class C, bool kPlain, int kM, int kN, int kParts, class At>
__device__ inline void finish_all(const Epilogue& e, const f32x4 (&acc)[kParts][kM][kN], At&& at) {
  using G = Groups<C, kM, kN>;
  if constexpr (kPlain) {
#pragma unroll
    for (int p = 0; p < kParts; ++p)
#pragma unroll
      for (int q = 0; q < G::kCount; ++q) {
        const uint64_t m = G::row(at(p).first, q), n = G::column(at(p).second, q);
        float v[C::V];
        G::sums(acc[p], q, v);
        if (m < e.m && n < e.n)
          store_upto<C>(e.y + (m * e.y_stride + n) * C::kElemBytes, v, e.n - n < C::V ? static_cast<int>(e.n - n) : C::V);
      }
    return;
  }
  u32x4 bias[kParts][G::kPerRow], residual[kParts][G::kCount];
#pragma unroll
  for (int p = 0; p < kParts; ++p) {
#pragma unroll
    for (int q = 0; q < G::kPerRow; ++q) bias[p][q] = fetch_bias<C>(e, G::column(at(p).second, q));
#pragma unroll
    for (int q = 0; q < G::kCount; ++q)
      residual[p][q] = fetch_residual<C>(e, G::row(at(p).first, q), G::column(at(p).second, q));
  }
  with_activation(e.act, [&](auto act) {
#pragma unroll
    for (int p = 0; p < kParts; ++p)
#pragma unroll
      for (int q = 0; q < G::kCount; ++q) {
        const uint64_t m = G::row(at(p).first, q), n = G::column(at(p).second, q);
        float v[C::V];
        G::sums(acc[p], q, v);
        keep_preact<C>(e, m, n, v, bias[p][q % G::kPerRow]);
#pragma unroll
        for (int c = 0; c < C::V; ++c) v[c] = activate<decltype(act)::value, C::kElemBytes == 2>(v[c]);
        keep_result<C>(e, m, n, v, residual[p][q]);
      }
  });
}

struct Corner {
  uint64_t first, second;
};

// ------------------------------------------------------------------ column sums

struct JoinArgs {
  const float* sums;  // [groups][kinds][stride]
  char* out[2];       // null: not wanted
  uint64_t stride, width;
  uint32_t groups, kinds;
};

// Adds the groups' column sums of one kind in a fixed order and rounds them:
// 32 columns a workgroup, 8 threads a column.
template <class P>
__device__ inline void join_block(const JoinArgs& a, uint64_t block, uint32_t kind) {
  __shared__ float part[8][33];
  const int c = threadIdx.x & 31, q = threadIdx.x >> 5;
  const uint64_t col = block * 32 + c;
  float s = 0.0f;
  if (col < a.width)
#pragma unroll 4
    for (uint32_t g = q; g < a.groups; g += 8) s += a.sums[(static_cast<uint64_t>(g) * a.kinds + kind) * a.stride + col];
  part[q][c] = s;
  __syncthreads();
  if (q == 0 && col < a.width && a.out[kind]) {
    float t = 0.0f;
#pragma unroll
    for (int i = 0; i < 8; ++i) t += part[i][c];
    reinterpret_cast<typename P::Bits*>(a.out[kind])[col] = P::narrow(t);
  }
}

template <class P>
__global__ __launch_bounds__(256) void column_join(const JoinArgs a) {
  join_block<P>(a, blockIdx.x, blockIdx.y);
}

// ------------------------------------------------------------------ general tile kernel

// Workgroup w of a launch runs on XCD w % 8, and each XCD has an L2 of its
// own.  This hands each XCD one run of neighbouring work items out of `total`.
__device__ inline uint32_t xcd_run(uint32_t w, uint32_t total) {
  const uint32_t per = total / 8, more = total % 8, x = w % 8, i = w / 8;
  return x * per + (x < more ? x : more) + i;
}

// Tile `id` in bands of 8 tile rows, down each band's columns: what is in
// flight on one XCD then shares rows of A and columns of B in its L2.
struct TileAt {
  uint32_t m, n;
  __device__ inline TileAt(uint32_t id, uint32_t tiles_m, uint32_t tiles_n) {
    constexpr uint32_t kBand = 8;
    const uint32_t band = id / (kBand * tiles_n), in_band = id % (kBand * tiles_n);
    const uint32_t high = tiles_m - band * kBand < kBand ? tiles_m - band * kBand : kBand;
    m = band * kBand + in_band % high;
    n = in_band / high;
  }
};

struct Operand {
  const char* base;
  uint64_t stride;  // elements between memory rows
  uint64_t rows;    // memory rows: m or n (kAlong), k (kDown)
  uint64_t cols;    // elements of a memory row: k (kAlong), m or n (kDown)
};

struct TileArgs {
  Operand a, b;
  Epilogue e;
  uint64_t k;
  uint32_t tiles_m, tiles_n;
  uint32_t blocks_per_share;  // blocks of k that one share sums
};

// Where one operand's kT x (64 k) tiles of a run of k come from: a thread's
// 8-element chunks, block after block, kParts 16-byte loads each.  Rows
// (kAlong) and columns (kDown) past the matrix meet only results that are not
// stored: a row past the end repeats the last one.
// The whole blocks' loads hang on no branch, or the compiler could not count
// which of the loads in flight a use has to wait for, and would wait for all:
// addresses are set up once and advance, past the last whole block by 0.
template <class C, bool kAlong, int kT, int kThreads, int kParts>
struct Feed {
  static constexpr int kChunks = kT * 8 / kThreads;
  static constexpr int kPerRow = kAlong ? 8 : kT / 8;  // chunks per LDS row
  static constexpr int e = C::kElemBytes;
  // kAlong: each chunk's address; kDown: the first one's, the others lie `apart`
  const char* p[kAlong ? kChunks : 1];
  uint64_t apart;
  uint64_t step;      // bytes between blocks
  uint64_t cols;      // kDown: columns from the tile's first on
  uint32_t left = 0;  // whole blocks not yet loaded

  __device__ inline void init(const Operand& o, uint64_t first, uint64_t k) {
    step = kAlong ? 64 * e : 64 * o.stride * e;
    cols = kAlong ? 0 : o.cols - first;
    apart = kThreads / kPerRow * o.stride * e;
#pragma unroll
    for (int i = 0; i < (kAlong ? kChunks : 1); ++i) {
      const int id = i * kThreads + threadIdx.x;
      const int r = id / kPerRow, c = id % kPerRow;
      uint64_t row = (kAlong ? first : k) + r;
      if (kAlong && row >= o.rows) row = o.rows - 1;
      p[i] = o.base + (row * o.stride + (kAlong ? k : first) + static_cast<uint64_t>(c) * 8) * e;
    }
  }
  __device__ inline const char* chunk(int i) const {
    if constexpr (kAlong) return p[i];
    return p[0] + i * apart;
  }
  // Whether all of the tile's columns exist.
  __device__ inline bool whole() const { return kAlong || cols >= kT; }

  // fn(chunk, part, address, how many of the part's elements exist) for the
  // next whole block.
  template <class Fn>
  __device__ inline void next(Fn&& fn) {
#pragma unroll
    for (int i = 0; i < kChunks; ++i)
#pragma unroll
      for (int q = 0; q < kParts; ++q) fn(i, q, chunk(i) + q * 16, C::V);
    const uint64_t by = left > 1 ? step : 0;
    if (left > 1) --left;
#pragma unroll
    for (int i = 0; i < (kAlong ? kChunks : 1); ++i) p[i] += by;
  }

  // The same for a block at k of which k_end - k may be less than 64, or
  // whose columns may end.
  template <class Fn>
  __device__ inline void edge(const Operand& o, uint64_t first, uint64_t k, uint64_t k_end, Fn&& fn) {
    init(o, first, k);
#pragma unroll
    for (int i = 0; i < kChunks; ++i) {
      const int id = i * kThreads + threadIdx.x;
      const int r = id / kPerRow, c = id % kPerRow;
      int64_t valid;
      if constexpr (kAlong)
        valid = static_cast<int64_t>(k_end - k) - c * 8;
      else
        valid = k + r < k_end ? static_cast<int64_t>(cols) - c * 8 : 0;
      const int n = valid < 0 ? 0 : (valid > 8 ? 8 : static_cast<int>(valid));
#pragma unroll
      for (int q = 0; q < kParts; ++q) fn(i, q, chunk(i) + q * 16, n - q * C::V);
    }
  }
};

// Walks over the blocks of k of a tile: kDeep whole blocks' loads in flight,
// then what is left one by one.  store(d, block) puts set d into the block's
// LDS buffer, compute(block) multiplies it; kBuffers LDS buffers alternate.
template <int kDeep, int kBuffers, class FA, class FB, class SA, class SB, class Store, class Compute>
__device__ inline void walk(const TileArgs& t, uint64_t m0, uint64_t n0, uint64_t k_first, uint64_t k_end, FA& feed_a,
                            FB& feed_b, SA (&sa)[kDeep], SB (&sb)[kDeep], Store&& store, Compute&& compute) {
  feed_a.init(t.a, m0, k_first);
  feed_b.init(t.b, n0, k_first);
  uint64_t k = k_first;
  const uint32_t blocks =
      k_end > k_first && feed_a.whole() && feed_b.whole() ? static_cast<uint32_t>((k_end - k_first) / 64) : 0;
  if (blocks > 0) {
    feed_a.left = feed_b.left = blocks;
#pragma unroll
    for (int d = 0; d < kDeep; ++d) {
      sa[d].load(feed_a);
      sb[d].load(feed_b);
      __builtin_amdgcn_sched_barrier(0);  // in this order, as the loop's waits count on it
    }
    // whole groups of kDeep blocks, so that the loop has one way out, then the rest
    uint32_t block = 0;
    for (; block + kDeep <= blocks; block += kDeep) {
#pragma unroll
      for (int d = 0; d < kDeep; ++d) {
        store(d, block + d);
        __syncthreads();
        sa[d].load(feed_a);
        sb[d].load(feed_b);
        __builtin_amdgcn_sched_barrier(0);
        compute(block + d);
        if constexpr (kBuffers == 1) __syncthreads();
      }
    }
#pragma unroll
    for (int d = 0; d + 1 < kDeep; ++d) {
      if (block + d < blocks) {
        store(d, block + d);
        __syncthreads();
        compute(block + d);
        if constexpr (kBuffers == 1) __syncthreads();
      }
    }
    k += static_cast<uint64_t>(blocks) * 64;
  }
  for (; k < k_end; k += 64) {
    sa[0].load_edge(feed_a, t.a, m0, k, k_end);
    sb[0].load_edge(feed_b, t.b, n0, k, k_end);
    __syncthreads();
    store(0, 0);
    __syncthreads();
    compute(0);
  }
}

// One operand's kT x (64 k) tile of a 16-bit type, from memory through
// registers into LDS.  kAlong: kT rows of 128 bytes, 16-byte chunk c of row r
// at chunk c ^ (r % 8), so that eight neighbouring rows' equal chunks lie in
// different banks.  kDown: one row of kT elements for each k, read
// transposed; 32-byte segments are xored with bits of k so that the rows that
// one instruction reads lie in different banks.
template <class C, bool kAlong, int kT, int kThreads>
struct Stage {
  static constexpr int V = C::V;
  static_assert(V == 8, "binary32 operands are split first");
  static constexpr int kBlock = 64;  // k
  static constexpr int kChunks = kT * 8 / kThreads;  // 16-byte chunks per thread
  static constexpr int kBytes = kT * 128;
  static constexpr int kPerRow = kAlong ? 8 : kT / V;  // chunks per LDS row
  u32x4 held[kChunks];

  static __device__ inline int swizzle(int row, int chunk) {
    if constexpr (kAlong) return chunk ^ (row & 7);
    // segments of 2 chunks; rows k .. k + 3 and k + 8 .. k + 11 are read at once
    constexpr int kSegs = kT / 16;
    const int key = kSegs >= 8 ? ((row & 3) | ((row >> 3 & 1) << 2)) : ((row >> 1 & 1) | ((row >> 3 & 1) << 1));
    return chunk ^ ((key & (kSegs - 1)) << 1);
  }

  __device__ inline void load(Feed<C, kAlong, kT, kThreads, 1>& f) {
    f.next([&](int i, int, const char* p, int valid) { held[i] = load_upto<C>(p, valid); });
  }
  __device__ inline void load_edge(Feed<C, kAlong, kT, kThreads, 1>& f, const Operand& o, uint64_t first, uint64_t k,
                                   uint64_t k_end) {
    f.edge(o, first, k, k_end, [&](int i, int, const char* p, int valid) { held[i] = load_upto<C>(p, valid); });
  }
  __device__ inline void store(char* lds) const {
#pragma unroll
    for (int i = 0; i < kChunks; ++i) {
      const int id = i * kThreads + threadIdx.x;
      const int r = id / kPerRow, c = id % kPerRow;
      *reinterpret_cast<u32x4*>(lds + (r * kPerRow + swizzle(r, c)) * 16) = held[i];
    }
  }

  // The 16 x (16-byte) operand tile of rows (kAlong) or columns `p` .. + 15,
  // step s of the block's two: lane l holds element p + l % 16 and the k of
  // its quarter l / 16 of the step.
  static __device__ inline u32x4 fragment(const char* lds, int p, int s) {
    const int lane = threadIdx.x & 63;
    const int r = lane & 15, g = lane >> 4;
    if constexpr (kAlong) {
      return *reinterpret_cast<const u32x4*>(lds + ((p + r) * 8 + swizzle(p + r, 4 * s + g)) * 16);
    } else {
      // lane l gives the address of row k + (l % 16) / 4, columns 4 (l % 4) .. + 3
      // of its quarter's 4 x 16 square and receives column l % 16
      u32x4 out;
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const int k = 32 * s + 8 * g + 4 * h + (r >> 2);
        const int col = p + 4 * (r & 3);
        const char* at = lds + (k * kPerRow + swizzle(k, col >> 3)) * 16 + (col & 7) * 2;
        const s16x4 q = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4*)at);
        const u32x2 w = __builtin_bit_cast(u32x2, q);
        out[2 * h] = w[0];
        out[2 * h + 1] = w[1];
      }
      return out;
    }
  }
};

// acc += (16 rows of b) x (16 rows of a) over the k of one fragment.
template <class C>
__device__ inline f32x4 multiply(const u32x4& b, const u32x4& a, f32x4 acc) {
  if constexpr (C::kElemBytes == 4) {
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const uint32_t x = b[j], y = a[j];
      acc = __builtin_amdgcn_mfma_f32_16x16x4f32(__builtin_bit_cast(float, x), __builtin_bit_cast(float, y), acc, 0, 0, 0);
    }
    return acc;
  } else if constexpr (std::is_same<C, BF16>::value) {
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, b), __builtin_bit_cast(bf16x8, a), acc, 0, 0, 0);
  } else {
    return __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(f16x8, b), __builtin_bit_cast(f16x8, a), acc, 0, 0, 0);
  }
}

// Any sizes, strides and alignments of a 16-bit type: kBM x kBN tiles by 4
// waves in a square, 64 k at a time, two LDS buffers.  The next kDeep blocks'
// loads are in flight in registers.
template <class C, bool kAAlong, bool kBAlong, int kBM, int kBN, int kDeep>
__device__ inline void tile_body(const TileArgs& t, uint32_t tile, uint32_t share, char* lds) {
  using SA = Stage<C, kAAlong, kBM, 256>;
  using SB = Stage<C, kBAlong, kBN, 256>;
  constexpr int kWM = kBM / 2 / 16, kWN = kBN / 2 / 16;
  const TileAt at(tile, t.tiles_m, t.tiles_n);
  const uint64_t m0 = static_cast<uint64_t>(at.m) * kBM, n0 = static_cast<uint64_t>(at.n) * kBN;
  const int wave = threadIdx.x >> 6;
  const int wm = (wave & 1) * (kBM / 2), wn = (wave >> 1) * (kBN / 2);
  const uint64_t k_first = static_cast<uint64_t>(share) * t.blocks_per_share * SA::kBlock;
  uint64_t k_end = k_first + static_cast<uint64_t>(t.blocks_per_share) * SA::kBlock;
  if (k_end > t.k) k_end = t.k;

  f32x4 acc[1][kWM][kWN];
#pragma unroll
  for (int i = 0; i < kWM; ++i)
#pragma unroll
    for (int j = 0; j < kWN; ++j) acc[0][i][j] = f32x4{0.f, 0.f, 0.f, 0.f};

  SA sa[kDeep];
  SB sb[kDeep];
  Feed<C, kAAlong, kBM, 256, 1> feed_a;
  Feed<C, kBAlong, kBN, 256, 1> feed_b;
  auto buffer = [&](uint32_t block) { return lds + (block & 1) * (SA::kBytes + SB::kBytes); };
  walk<kDeep, 2>(
      t, m0, n0, k_first, k_end, feed_a, feed_b, sa, sb,
      [&](int d, uint32_t block) {
        sa[d].store(buffer(block));
        sb[d].store(buffer(block) + SA::kBytes);
      },
      [&](uint32_t block) {
        const char* la = buffer(block);
        const char* lb = la + SA::kBytes;
#pragma unroll
        for (int s = 0; s < 2; ++s) {
          u32x4 fa[kWM], fb[kWN];
#pragma unroll
          for (int i = 0; i < kWM; ++i) fa[i] = SA::fragment(la, wm + 16 * i, s);
#pragma unroll
          for (int j = 0; j < kWN; ++j) fb[j] = SB::fragment(lb, wn + 16 * j, s);
#pragma unroll
          for (int i = 0; i < kWM; ++i)
#pragma unroll
            for (int j = 0; j < kWN; ++j) acc[0][i][j] = multiply<C>(fb[j], fa[i], acc[0][i][j]);
        }
      });
  if (t.e.partial) {
    using G = Groups<C, kWM, kWN>;
#pragma unroll
    for (int q = 0; q < G::kCount; ++q) {
      float v[C::V];
      G::sums(acc[0], q, v);
      keep_partial<C>(t.e, share, G::row(m0 + wm, q), G::column(n0 + wn, q), v);
    }
  } else {
    finish_all<C, !(kAAlong && kBAlong)>(t.e, acc, [&](int) { return Corner{m0 + wm, n0 + wn}; });
  }
}

// ------------------------------------------------------------------ large products of 16-bit types

// 256 x 256 tiles by 8 waves (2 x 4; a wave has 4 x 2 tiles of 16 x 16 in each
// quarter of the tile), 64 k at a time, memory to LDS without registers in
// between.  A block of k lies in LDS as four halves: rows 0..127 and
// 128..255 of A, and of B, 16 KiB each, in Stage's layout; two blocks fill
// 128 KiB, so one workgroup runs on a compute unit.
//
// A block is multiplied in four phases, a quarter of the tile each:
//   (A0, B0)  (A0, B1)  (A1, B1)  (A1, B0)
// While a phase's 16 MFMAs run, its wave reads the next phase's new half into
// registers (B1, A1, the next block's A0, the next block's B0), and the
// workgroup starts the copy of the half that the phase before has finished
// with.  So each half is on its way for seven phases (96 KiB in flight per
// compute unit), every phase waits for all but the 12 newest copies and for
// its own reads, and one barrier a phase orders both.  8192 x 8192 x 4096
// bf16 with gelu and z kept: 400 to 420 us from box to box in a run of calls
// (1310 to 1370 TFLOP/s; 370 to 400 us without them, no more than the library's
// product of these sizes), 400 at best and 466 at the median under a profiler,
// where the clock has not settled; a wave's LDS reads take 75% of its MFMAs'
// time, and what is left is the clock that the matrix units hold at this load.
// The second block of a pair finds its first B half where the block before
// read it to, so the two B register sets change roles from block to block.
constexpr int kHalfBytes = 128 * 128;
constexpr int kBlockBytes = 4 * kHalfBytes;
constexpr int kBigLds = 2 * kBlockBytes;

struct BigArgs {
  Operand a, b;
  Epilogue e;
  uint64_t k;
  uint32_t tiles_m, tiles_n;
};

// 16 bytes a lane from memory to LDS, lane l's to lds + 16 l; past the
// resource's range zeros arrive.  All of the offset is in `voffset`: that is
// what the range check compares, while a scalar offset only lowers the range
// it is compared with, which has no defined meaning once that offset exceeds
// the range.  The wait is the caller's (vmcnt).  The compiler's own form of
// this instruction makes it wait for every copy under way at the next LDS
// read.  The instruction writes no register, so a copy under way cannot go
// over one, and nothing else in these kernels uses m0.
__device__ inline void copy_to_lds(__amdgpu_buffer_rsrc_t from, uint32_t lds, uint32_t voffset) {
  asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tbuffer_load_dwordx4 %1, %2, 0 offen lds" ::"s"(lds), "v"(voffset),
               "s"(from)
               : "memory");
}

// One operand's copies: half h of k block t of a 256-row (or -column) tile.
// Offsets from the tile's start (kAlong) or the block's first row (kDown) fit
// 31 bits, which the host has checked.  Rows and chunks that do not exist lie
// past the resource's range, so zeros take their place: rows past the
// matrix's end by themselves, and the chunks past k of a kAlong row by an
// offset out of any range.
template <class C, bool kAlong>
struct Copier {
  static constexpr int e = C::kElemBytes;
  const char* base;  // of the tile
  uint64_t left;     // bytes from there to the matrix's end
  uint32_t stride;   // bytes
  uint32_t blocks;
  uint32_t voffset;
  uint32_t last;     // kAlong: voffset in the last block

  __device__ inline void init(const Operand& o, uint64_t first, uint64_t k, uint32_t blocks_, int wave) {
    const int lane = threadIdx.x & 63;
    stride = static_cast<uint32_t>(o.stride * e);
    blocks = blocks_;
    const uint64_t at = kAlong ? first * stride : first * e;
    base = o.base + at;
    left = (o.rows - 1) * o.stride * e + o.cols * e - at;
    if constexpr (kAlong) {
      const int chunk = (lane & 7) ^ (lane >> 3);
      voffset = (wave * 8 + (lane >> 3)) * stride + chunk * 16;
      last = static_cast<uint64_t>(blocks - 1) * 64 + chunk * C::V < k ? voffset : kNowhere;
    } else {
      const int row = wave * 4 + (lane >> 4);
      voffset = row * stride + Stage<C, false, 128, 512>::swizzle(row, lane & 15) * 16;
      last = voffset;
    }
  }

  // past any range, and with any offset added still below 2^32
  static constexpr uint32_t kNowhere = 0x80000000u;

  static __device__ inline __amdgpu_buffer_rsrc_t range(const char* from, uint64_t bytes) {
    const uint32_t n = bytes >> 31 ? 0x7fffffffu : static_cast<uint32_t>(bytes);
    return __builtin_amdgcn_make_buffer_rsrc(const_cast<char*>(from), 0, static_cast<int>(n), kRawBufferWord3);
  }

  __device__ inline void copy(uint32_t lds, int h, uint32_t t, int wave) const {
    if constexpr (kAlong) {
      const __amdgpu_buffer_rsrc_t from = range(base, left);
      const uint32_t v = t + 1 < blocks ? voffset : (t + 1 == blocks ? last : kNowhere);
      const uint32_t k = t < blocks ? t * 128 : 0;
#pragma unroll
      for (int q = 0; q < 2; ++q) copy_to_lds(from, lds + (q * 8 + wave) * 1024, v + (h * 128 + q * 64) * stride + k);
    } else {
      const uint64_t at = static_cast<uint64_t>(t) * (64 * stride);
      const __amdgpu_buffer_rsrc_t from = range(base + at, t < blocks ? left - at : 0);
#pragma unroll
      for (int q = 0; q < 2; ++q)
        copy_to_lds(from, lds + (q * 8 + wave) * 1024, voffset + q * 32 * stride + h * 128 * e);
    }
  }
};

template <class C, bool kAAlong, bool kBAlong>
__global__ __launch_bounds__(512, 2) void linear_big(const BigArgs args) {
  using SA = Stage<C, kAAlong, 128, 512>;
  using SB = Stage<C, kBAlong, 128, 512>;
  extern __shared__ __align__(16) char lds[];
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int wm = wave >> 2, wn = wave & 3;
  const uint32_t lds0 = static_cast<uint32_t>(reinterpret_cast<uintptr_t>((__attribute__((address_space(3))) char*)lds));

  const TileAt at(xcd_run(blockIdx.x, args.tiles_m * args.tiles_n), args.tiles_m, args.tiles_n);
  const uint64_t m0 = static_cast<uint64_t>(at.m) * 256, n0 = static_cast<uint64_t>(at.n) * 256;

  Copier<C, kAAlong> ca;
  Copier<C, kBAlong> cb;
  const uint32_t blocks = static_cast<uint32_t>((args.k + 63) / 64);
  ca.init(args.a, m0, args.k, blocks, wave);
  cb.init(args.b, n0, args.k, blocks, wave);

  // Halves of block t: A0, A1, B0, B1.  Both blocks' A halves come first, so
  // that one address register and the instruction's offset reach them all.
  auto region = [](uint32_t t, int which) { return (which >> 1) * (4 * kHalfBytes) + (t & 1) * (2 * kHalfBytes) + (which & 1) * kHalfBytes; };

  f32x4 acc[4][4][2];  // quarter (i, j) is 2 i + j
#pragma unroll
  for (int p = 0; p < 4; ++p)
#pragma unroll
    for (int x = 0; x < 4; ++x)
#pragma unroll
      for (int y = 0; y < 2; ++y) acc[p][x][y] = f32x4{0.f, 0.f, 0.f, 0.f};
  u32x4 fa[2][2][4], fb[2][2][2];  // [set][step][tile]

  ca.copy(lds0 + region(0, 0), 0, 0, wave);
  cb.copy(lds0 + region(0, 2), 0, 0, wave);
  cb.copy(lds0 + region(0, 3), 1, 0, wave);
  ca.copy(lds0 + region(0, 1), 1, 0, wave);
  ca.copy(lds0 + region(1, 0), 0, 1, wave);
  cb.copy(lds0 + region(1, 2), 0, 1, wave);
  cb.copy(lds0 + region(1, 3), 1, 1, wave);
  ca.copy(lds0 + region(1, 1), 1, 1, wave);
  asm volatile("s_waitcnt vmcnt(12)\n\ts_barrier" ::: "memory");
#pragma unroll
  for (int s = 0; s < 2; ++s) {
#pragma unroll
    for (int x = 0; x < 4; ++x) fa[0][s][x] = SA::fragment(lds + region(0, 0), wm * 64 + 16 * x, s);
#pragma unroll
    for (int y = 0; y < 2; ++y) fb[0][s][y] = SB::fragment(lds + region(0, 2), wn * 32 + 16 * y, s);
  }
  asm volatile("s_waitcnt lgkmcnt(0)\n\ts_barrier" ::: "memory");
  ca.copy(lds0 + region(0, 0), 0, 2, wave);
  asm volatile("s_waitcnt vmcnt(12)\n\ts_barrier" ::: "memory");

  // One phase: the products of A set `i` and B set `b` into quarter (i, j);
  // `read` takes the slots 0..7 and reads a part of the next half in each.
  auto phase = [&](auto i_, auto j_, auto b_, auto&& read, auto&& copy) {
    constexpr int i = decltype(i_)::value, j = decltype(j_)::value, b = decltype(b_)::value;
#pragma unroll
    for (int slot = 0; slot < 8; ++slot) {
      const int s = slot >> 2, x = slot & 3;
      read(slot);
#pragma unroll
      for (int y = 0; y < 2; ++y)
        acc[2 * i + j][x][y] = multiply<C>(fb[b][s][y], fa[i][s][x], acc[2 * i + j][x][y]);
      if (slot == 3) copy();
      __builtin_amdgcn_sched_barrier(0);
    }
    asm volatile("s_waitcnt vmcnt(12) lgkmcnt(0)\n\ts_barrier" ::: "memory");
    __builtin_amdgcn_sched_barrier(0);
  };
  using Zero = std::integral_constant<int, 0>;
  using One = std::integral_constant<int, 1>;
  // One block whose first B half is in set `b`.
  auto block = [&](uint32_t t, auto b_, auto c_) {
    constexpr int b = decltype(b_)::value, c = decltype(c_)::value;
    phase(Zero{}, Zero{}, b_,
          [&](int slot) {
            if (slot < 4) fb[c][slot >> 1][slot & 1] = SB::fragment(lds + region(b, 3), wn * 32 + 16 * (slot & 1), slot >> 1);
          },
          [&] { cb.copy(lds0 + region(b, 2), 0, t + 2, wave); });
    phase(Zero{}, One{}, c_,
          [&](int slot) { fa[1][slot >> 2][slot & 3] = SA::fragment(lds + region(b, 1), wm * 64 + 16 * (slot & 3), slot >> 2); },
          [&] { cb.copy(lds0 + region(b, 3), 1, t + 2, wave); });
    phase(One{}, One{}, c_,
          [&](int slot) { fa[0][slot >> 2][slot & 3] = SA::fragment(lds + region(c, 0), wm * 64 + 16 * (slot & 3), slot >> 2); },
          [&] { ca.copy(lds0 + region(b, 1), 1, t + 2, wave); });
    phase(One{}, Zero{}, b_,
          [&](int slot) {
            if (slot < 4) fb[c][slot >> 1][slot & 1] = SB::fragment(lds + region(c, 2), wn * 32 + 16 * (slot & 1), slot >> 1);
          },
          [&] { ca.copy(lds0 + region(c, 0), 0, t + 3, wave); });
  };
  uint32_t t = 0;
  for (; t + 2 <= blocks; t += 2) {
    block(t, Zero{}, One{});
    block(t + 1, One{}, Zero{});
  }
  if (t < blocks) block(t, Zero{}, One{});
  // zeros that copies past the last block still bring must not meet the next
  // workgroup's LDS
  asm volatile("s_waitcnt vmcnt(0)" ::: "memory");

  finish_all<C, !(kAAlong && kBAlong)>(args.e, acc, [&](int p) {
    return Corner{m0 + (p >> 1) * 128 + wm * 64, n0 + (p & 1) * 128 + wn * 32};
  });
}

// ------------------------------------------------------------------ binary32 products

// A binary32 value is the sum of three bfloat16 values: its nearest, the
// nearest to what is left (at most 2^-8 of the value's leading power of two),
// and what is left then (at most 2^-17).  They hold all 24 bits as long as the
// last of them is no smaller than bfloat16's smallest values, so every operand
// is multiplied by 2^24 first: the last bit of any binary32 value, 2^-149 at
// least, is then 2^-125, a normal bfloat16.  (Unscaled, a value of 2^-120 kept
// 14 bits.)  Of the nine products of two such sums the six largest are taken,
// on the bfloat16 matrix units; the others are at most 2 * 2^-8 * 2^-17 + 2^-34
// of the product, what rounding it to binary32 costs.  Six bfloat16 MFMAs take
// 96 cycles where the binary32 MFMAs of the same 16 x 16 x 32 take 256.
// Infinities and NaN have no such parts (inf - inf), nor have values from
// 2^104 on after their scaling: they make the tile's sums non-finite, as do
// sums from 2^80 on, and a tile with a non-finite sum is summed again in
// binary32, unscaled.
struct Parts {
  u32x4 part[3];  // of eight values
};

constexpr float kSplitScale = 0x1p24f;  // of each operand
constexpr float kSplitBack = 0x1p-48f;  // of their product

__device__ inline Parts split(const u32x4& lo, const u32x4& hi) {
  float v[8];
  F32::unpack(lo, v);
  F32::unpack(hi, v + 4);
#pragma unroll
  for (int i = 0; i < 8; ++i) v[i] *= kSplitScale;
  Parts o;
#pragma unroll
  for (int p = 0; p < 3; ++p) {
    o.part[p] = BF16::pack(v);
    if (p == 2) break;
    float t[8];
    BF16::unpack(o.part[p], t);
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] -= t[i];
  }
  return o;
}

// One operand's kT x 64 block of k: binary32 from memory, three planes of
// bfloat16 in LDS, each in Stage<BF16>'s layout.
template <bool kAlong, int kT>
struct SplitStage {
  using S = Stage<BF16, kAlong, kT, 256>;
  static constexpr int kChunks = S::kChunks, kPerRow = S::kPerRow;
  static constexpr int kBytes = 3 * S::kBytes;
  u32x4 held[kChunks][2];

  __device__ inline void load(Feed<F32, kAlong, kT, 256, 2>& f) {
    f.next([&](int i, int q, const char* p, int valid) { held[i][q] = load_upto<F32>(p, valid); });
  }
  __device__ inline void load_edge(Feed<F32, kAlong, kT, 256, 2>& f, const Operand& o, uint64_t first, uint64_t k,
                                   uint64_t k_end) {
    f.edge(o, first, k, k_end, [&](int i, int q, const char* p, int valid) { held[i][q] = load_upto<F32>(p, valid); });
  }
  __device__ inline void store(char* lds) const {
#pragma unroll
    for (int i = 0; i < kChunks; ++i) {
      const int id = i * 256 + threadIdx.x;
      const int r = id / kPerRow, c = id % kPerRow;
      const Parts o = split(held[i][0], held[i][1]);
#pragma unroll
      for (int p = 0; p < 3; ++p)
        *reinterpret_cast<u32x4*>(lds + p * S::kBytes + (r * kPerRow + S::swizzle(r, c)) * 16) = o.part[p];
    }
  }
  static __device__ inline u32x4 fragment(const char* lds, int plane, int p, int s) {
    return S::fragment(lds + plane * S::kBytes, p, s);
  }
};

// One value of an operand, 0 outside of it.
template <bool kAlong>
__device__ inline float value_at(const Operand& o, uint64_t i, uint64_t k, uint64_t k_end) {
  const uint64_t row = kAlong ? i : k, col = kAlong ? k : i;
  if (row >= o.rows || col >= o.cols || k >= k_end) return 0.0f;
  return *reinterpret_cast<const float*>(o.base + (row * o.stride + col) * 4);
}

// kBM x kBN tiles by 4 waves in a square, 64 k at a time.  One LDS buffer, as
// three planes of it let two workgroups share a compute unit: one splits and
// stores while the other multiplies.  kDeep blocks' loads are in flight, as in
// linear_tile.
template <bool kAAlong, bool kBAlong, int kBM, int kBN, int kDeep>
__device__ inline void split_body(const TileArgs& t, uint32_t tile, uint32_t share, char* lds) {
  using SA = SplitStage<kAAlong, kBM>;
  using SB = SplitStage<kBAlong, kBN>;
  constexpr int kWM = kBM / 2 / 16, kWN = kBN / 2 / 16;
  const TileAt at(tile, t.tiles_m, t.tiles_n);
  const uint64_t m0 = static_cast<uint64_t>(at.m) * kBM, n0 = static_cast<uint64_t>(at.n) * kBN;
  const int wave = threadIdx.x >> 6;
  const int wm = (wave & 1) * (kBM / 2), wn = (wave >> 1) * (kBN / 2);
  const uint64_t k_first = static_cast<uint64_t>(share) * t.blocks_per_share * 64;
  uint64_t k_end = k_first + static_cast<uint64_t>(t.blocks_per_share) * 64;
  if (k_end > t.k) k_end = t.k;

  f32x4 acc[1][kWM][kWN];
#pragma unroll
  for (int i = 0; i < kWM; ++i)
#pragma unroll
    for (int j = 0; j < kWN; ++j) acc[0][i][j] = f32x4{0.f, 0.f, 0.f, 0.f};

  SA sa[kDeep];
  SB sb[kDeep];
  Feed<F32, kAAlong, kBM, 256, 2> feed_a;
  Feed<F32, kBAlong, kBN, 256, 2> feed_b;
  walk<kDeep, 1>(
      t, m0, n0, k_first, k_end, feed_a, feed_b, sa, sb,
      [&](int d, uint32_t) {
        sa[d].store(lds);
        sb[d].store(lds + SA::kBytes);
      },
      [&](uint32_t) {
#pragma unroll
        for (int s = 0; s < 2; ++s) {
          u32x4 fb[3][kWN];
#pragma unroll
          for (int p = 0; p < 3; ++p)
#pragma unroll
            for (int j = 0; j < kWN; ++j) fb[p][j] = SB::fragment(lds + SA::kBytes, p, wn + 16 * j, s);
#pragma unroll
          for (int i = 0; i < kWM; ++i) {
            u32x4 fa[3];
#pragma unroll
            for (int p = 0; p < 3; ++p) fa[p] = SA::fragment(lds, p, wm + 16 * i, s);
            // the smaller products first
#pragma unroll
            for (int sum = 2; sum >= 0; --sum)
#pragma unroll
              for (int p = 0; p <= sum; ++p)
#pragma unroll
                for (int j = 0; j < kWN; ++j) acc[0][i][j] = multiply<BF16>(fb[sum - p][j], fa[p], acc[0][i][j]);
          }
        }
      });

  bool odd = false;
#pragma unroll
  for (int i = 0; i < kWM; ++i)
#pragma unroll
    for (int j = 0; j < kWN; ++j)
#pragma unroll
      for (int c = 0; c < 4; ++c) odd |= !(fabsf(acc[0][i][j][c]) < INFINITY);
  if (__any(odd)) {
    const int lane = threadIdx.x & 63, r = lane & 15, g = lane >> 4;
#pragma unroll
    for (int i = 0; i < kWM; ++i)
#pragma unroll
      for (int j = 0; j < kWN; ++j) acc[0][i][j] = f32x4{0.f, 0.f, 0.f, 0.f};
    for (uint64_t k = k_first; k < k_end; k += 4) {
      float a[kWM], b[kWN];
#pragma unroll
      for (int i = 0; i < kWM; ++i) a[i] = value_at<kAAlong>(t.a, m0 + wm + 16 * i + r, k + g, k_end);
#pragma unroll
      for (int j = 0; j < kWN; ++j) b[j] = value_at<kBAlong>(t.b, n0 + wn + 16 * j + r, k + g, k_end);
#pragma unroll
      for (int i = 0; i < kWM; ++i)
#pragma unroll
        for (int j = 0; j < kWN; ++j)
          acc[0][i][j] = __builtin_amdgcn_mfma_f32_16x16x4f32(b[j], a[i], acc[0][i][j], 0, 0, 0);
    }
  } else {
#pragma unroll
    for (int i = 0; i < kWM; ++i)
#pragma unroll
      for (int j = 0; j < kWN; ++j) acc[0][i][j] *= kSplitBack;
  }
  if (t.e.partial) {
    using G = Groups<F32, kWM, kWN>;
#pragma unroll
    for (int q = 0; q < G::kCount; ++q) {
      float v[4];
      G::sums(acc[0], q, v);
      keep_partial<F32>(t.e, share, G::row(m0 + wm, q), G::column(n0 + wn, q), v);
    }
  } else {
    finish_all<F32, !(kAAlong && kBAlong)>(t.e, acc, [&](int) { return Corner{m0 + wm, n0 + wn}; });
  }
}

// ------------------------------------------------------------------ launches of tiles

// LDS of one tile's workgroup.
template <class C, bool kAAlong, bool kBAlong, int kBM, int kBN>
constexpr int tile_lds() {
  if constexpr (C::kElemBytes == 4)
    return SplitStage<kAAlong, kBM>::kBytes + SplitStage<kBAlong, kBN>::kBytes;
  else
    return 2 * (Stage<C, kAAlong, kBM, 256>::kBytes + Stage<C, kBAlong, kBN, 256>::kBytes);
}

template <class C, bool kAAlong, bool kBAlong, int kBM, int kBN>
__device__ inline void any_tile(const TileArgs& t, uint32_t tile, uint32_t share, char* lds) {
  if constexpr (C::kElemBytes == 4)
    split_body<kAAlong, kBAlong, kBM, kBN, 1>(t, tile, share, lds);
  else
    // what the registers hold: 256 a lane, of which the larger tile's sums are 64
    tile_body<C, kAAlong, kBAlong, kBM, kBN, kBM == 64 ? 4 : (kAAlong && kBAlong ? 2 : 1)>(t, tile, share, lds);
}

// One product: all tiles of the first share of k, then of the next one.
template <class C, bool kAAlong, bool kBAlong, int kBM, int kBN>
__global__ __launch_bounds__(256, 2) void linear_tile(const TileArgs t) {
  extern __shared__ __align__(16) char lds[];
  const uint32_t id = xcd_run(blockIdx.x, gridDim.x), tiles = t.tiles_m * t.tiles_n;
  any_tile<C, kAAlong, kBAlong, kBM, kBN>(t, id % tiles, id / tiles, lds);
}

// Both gradients' products and the bias gradient's last sums in one launch:
// small products leave the device half empty, and each launch costs about 2 us
// on the host.
struct PairArgs {
  TileArgs dx, dw;
  JoinArgs db;
  uint32_t dx_tiles, dw_tiles, dx_groups, dw_groups;  // groups: tiles x shares
};

template <class C, int kBM, int kBN>
__global__ __launch_bounds__(256, 2) void linear_pair(const PairArgs p) {
  extern __shared__ __align__(16) char lds[];
  uint32_t id = blockIdx.x;
  if (id < p.dx_groups) {
    id = xcd_run(id, p.dx_groups);
    any_tile<C, true, false, kBM, kBN>(p.dx, id % p.dx_tiles, id / p.dx_tiles, lds);
    return;
  }
  id -= p.dx_groups;
  if (id < p.dw_groups) {
    id = xcd_run(id, p.dw_groups);
    any_tile<C, false, false, kBM, kBN>(p.dw, id % p.dw_tiles, id / p.dw_tiles, lds);
    return;
  }
  join_block<C>(p.db, id - p.dw_groups, 0);
}

// Adds the shares of k in their order and finishes the sums of one group of V.
template <class C>
__device__ inline void join_shares(const Epilogue& e, int shares, uint64_t id) {
  constexpr int V = C::V;
  const uint64_t per_row = (e.n + V - 1) / V;
  if (id >= per_row * e.m) return;
  const uint64_t m = id / per_row, n = id % per_row * V;
  float v[V];
#pragma unroll
  for (int i = 0; i < V; ++i) v[i] = 0.0f;
  for (int s = 0; s < shares; ++s) {
    const float* p = e.partial + (static_cast<uint64_t>(s) * e.m + m) * e.partial_stride + n;
#pragma unroll
    for (int i = 0; i < V; i += 4) {
      const f32x4 q = *reinterpret_cast<const f32x4*>(p + i);
#pragma unroll
      for (int c = 0; c < 4; ++c) v[i + c] += q[c];
    }
  }
  finish<C>(e, m, n, v);
}

// Up to two products' shares: the first `groups` workgroups join a's.
template <class C>
__global__ __launch_bounds__(256) void linear_join(const Epilogue a, int a_shares, const Epilogue b, int b_shares,
                                                   uint32_t groups) {
  if (blockIdx.x < groups)
    join_shares<C>(a, a_shares, static_cast<uint64_t>(blockIdx.x) * 256 + threadIdx.x);
  else
    join_shares<C>(b, b_shares, static_cast<uint64_t>(blockIdx.x - groups) * 256 + threadIdx.x);
}

// ------------------------------------------------------------------ few rows

// Products of up to 32 rows, where the pass over w bounds: 8 waves share
// 16 kN rows of w (columns of y) and split k between them, each streams its
// part of w straight into the MFMA operand registers (no LDS on the way,
// every byte of w is used once), and the 8 waves' sums meet in LDS.  x is
// small and comes from the caches; its rows past the end repeat the last one,
// as do w's, and their results are not stored.  A step is 128 bytes of k;
// the loads of the next kDeep steps are in flight while kDeep are multiplied.
// 1 x 8192 x 4096 bf16: 12.6 us (5.3 TB/s); 32 x 4096 x 8192: 18.8 us, where
// reading x, as many bytes a workgroup as its part of w, takes the rest.
template <class C, int kM, int kN, int kDeep>
__global__ __launch_bounds__(512) void linear_few(const TileArgs t) {
  constexpr int V = C::V;
  constexpr int kStep = 8 * V;
  constexpr int kPitch = 16 * kN + 4;  // floats; rows 16 apart lie 4 banks apart
  __shared__ __align__(16) float sums[4][16 * kM * kPitch];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int r = lane & 15, g = lane >> 4;
  const uint64_t n0 = static_cast<uint64_t>(blockIdx.x) * (16 * kN);
  const char* w[kN];
  const char* x[kM];
#pragma unroll
  for (int j = 0; j < kN; ++j) {
    const uint64_t n = n0 + 16 * j + r;
    w[j] = t.b.base + ((n < t.b.rows ? n : t.b.rows - 1) * t.b.stride + g * V) * C::kElemBytes;
  }
#pragma unroll
  for (int i = 0; i < kM; ++i) {
    const uint64_t m = 16 * i + r;
    x[i] = t.a.base + ((m < t.a.rows ? m : t.a.rows - 1) * t.a.stride + g * V) * C::kElemBytes;
  }
  f32x4 acc[kM][kN];
#pragma unroll
  for (int i = 0; i < kM; ++i)
#pragma unroll
    for (int j = 0; j < kN; ++j) acc[i][j] = f32x4{0.f, 0.f, 0.f, 0.f};

  // this wave's whole steps of this share of k: [step, end)
  const uint64_t whole = t.k / kStep;
  const uint64_t share_first = static_cast<uint64_t>(blockIdx.y) * t.blocks_per_share;
  const uint64_t share_end = share_first + t.blocks_per_share < whole ? share_first + t.blocks_per_share : whole;
  const uint64_t per = (t.blocks_per_share + 7) / 8;
  uint64_t step = share_first + wave * per;
  uint64_t end = step + per < share_end ? step + per : share_end;
  if (step > end) step = end;

  u32x4 wq[2][kDeep][kN][2], xq[2][kDeep][kM][2];
  auto load = [&](int set, uint64_t from) {
#pragma unroll
    for (int d = 0; d < kDeep; ++d) {
      const uint64_t at = (from + d) * 128;
#pragma unroll
      for (int h = 0; h < 2; ++h) {
#pragma unroll
        for (int j = 0; j < kN; ++j) wq[set][d][j][h] = load_loose<C>(w[j] + at + 64 * h);
#pragma unroll
        for (int i = 0; i < kM; ++i) xq[set][d][i][h] = load_loose<C>(x[i] + at + 64 * h);
      }
    }
  };
  auto compute = [&](int set) {
#pragma unroll
    for (int d = 0; d < kDeep; ++d)
#pragma unroll
      for (int h = 0; h < 2; ++h)
#pragma unroll
        for (int i = 0; i < kM; ++i)
#pragma unroll
          for (int j = 0; j < kN; ++j) acc[i][j] = multiply<C>(wq[set][d][j][h], xq[set][d][i][h], acc[i][j]);
  };
  // The multiplication stands in the branch with the loads it overlaps: behind
  // a join of paths with and without them the compiler waits for all.
  if (step + kDeep <= end) {
    load(0, step);
    for (;;) {
      if (step + 2 * kDeep > end) {
        compute(0);
        step += kDeep;
        break;
      }
      load(1, step + kDeep);
      compute(0);
      step += kDeep;
      if (step + 2 * kDeep > end) {
        compute(1);
        step += kDeep;
        break;
      }
      load(0, step + kDeep);
      compute(1);
      step += kDeep;
    }
  }
  auto single = [&](uint64_t at, bool whole_step) {
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      u32x4 a[kM], b[kN];
      const uint64_t k = at * kStep + h * (kStep / 2) + g * V;
      const int valid = whole_step ? V : (k >= t.k ? 0 : (t.k - k < V ? static_cast<int>(t.k - k) : V));
#pragma unroll
      for (int j = 0; j < kN; ++j) b[j] = load_upto<C>(w[j] + at * 128 + 64 * h, valid);
#pragma unroll
      for (int i = 0; i < kM; ++i) a[i] = load_upto<C>(x[i] + at * 128 + 64 * h, valid);
#pragma unroll
      for (int i = 0; i < kM; ++i)
#pragma unroll
        for (int j = 0; j < kN; ++j) acc[i][j] = multiply<C>(b[j], a[i], acc[i][j]);
    }
  };
  for (; step < end; ++step) single(step, true);
  // k past the last whole step: the last share's last wave
  if (t.k % kStep && blockIdx.y == gridDim.y - 1 && wave == 7) single(whole, false);

  // waves 4..7 hand their sums to waves 0..3
#pragma unroll
  for (int turn = 1; turn >= 0; --turn) {
    if (wave >> 2 == turn)
#pragma unroll
      for (int i = 0; i < kM; ++i)
#pragma unroll
        for (int j = 0; j < kN; ++j) {
          f32x4& at = *reinterpret_cast<f32x4*>(&sums[wave & 3][(16 * i + r) * kPitch + 16 * j + 4 * g]);
          at = turn ? acc[i][j] : at + acc[i][j];
        }
    __syncthreads();
  }
  constexpr int kGroups = 16 * kM * 16 * kN / V;
  for (int id = threadIdx.x; id < kGroups; id += 512) {
    const int m = id / (16 * kN / V), n = id % (16 * kN / V) * V;
    float v[V];
#pragma unroll
    for (int c = 0; c < V; ++c) v[c] = 0.0f;
#pragma unroll
    for (int q = 0; q < 4; ++q)
#pragma unroll
      for (int c = 0; c < V; ++c) v[c] += sums[q][m * kPitch + n + c];
    if (t.e.partial)
      keep_partial<C>(t.e, blockIdx.y, m, n0 + n, v);
    else
      finish<C>(t.e, m, n0 + n, v);
  }
}

// ------------------------------------------------------------------ operands laid out anew

struct PackArgs {
  const char* from;
  char* to;
  uint64_t from_stride, to_stride, rows, cols;
};

// A copy of a matrix with rows at 16-byte boundaries, each padded with zeros
// to whole vectors.  linear_big takes only such operands.
template <class C>
__global__ __launch_bounds__(256) void linear_pack(const PackArgs a) {
  constexpr int V = C::V;
  const uint64_t per_row = (a.cols + V - 1) / V;
  const uint64_t total = per_row * a.rows;
  for (uint64_t id = static_cast<uint64_t>(blockIdx.x) * 256 + threadIdx.x; id < total;
       id += static_cast<uint64_t>(gridDim.x) * 256) {
    const uint64_t row = id / per_row, col = id % per_row * V;
    const int valid = a.cols - col < V ? static_cast<int>(a.cols - col) : V;
    *reinterpret_cast<u32x4*>(a.to + (row * a.to_stride + col) * C::kElemBytes) =
        load_upto<C>(a.from + (row * a.from_stride + col) * C::kElemBytes, valid);
  }
}

// ------------------------------------------------------------------ dz and the bias gradient

struct SlopeArgs {
  const char* dy;
  const char* z;   // null: no activation
  char* dz;        // null: not wanted (dy itself is dz)
  float* sums;     // null: no bias gradient; else [gridDim.y][sums_stride]
  uint64_t dy_stride, z_stride, dz_stride, sums_stride;
  uint64_t rows, cols;
  uint32_t rows_per_group;
  int act;
};

// dz = dy act'(z), and each column's sum of dz over this workgroup's rows,
// in binary32 from the unrounded products.  A pass over memory: 64 lanes
// cover 64 V columns, the 4 waves take the rows in turn.
// dz is rounded to the element type because the matrix units multiply that
// type (its two halves would take two products each): up to 2^-8 (bf16) of
// each term, independent from term to term, which adds to a product's error no
// more than the rounding of its result (2.4e-3 of dx and dw against 64 bits,
// with the result's rounding alone 1.7e-3).
template <class C>
__global__ __launch_bounds__(256) void linear_slope(const SlopeArgs a) {
  constexpr int V = C::V;
  constexpr bool kFast = C::kElemBytes == 2;
  __shared__ float part[4][64 * V];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const uint64_t n = (static_cast<uint64_t>(blockIdx.x) * 64 + lane) * V;
  const uint64_t first = static_cast<uint64_t>(blockIdx.y) * a.rows_per_group;
  uint64_t end = first + a.rows_per_group;
  if (end > a.rows) end = a.rows;
  const int valid = n >= a.cols ? 0 : (a.cols - n < V ? static_cast<int>(a.cols - n) : V);
  float sum[V];
#pragma unroll
  for (int i = 0; i < V; ++i) sum[i] = 0.0f;
  with_activation(a.z ? a.act : MSCL_ACT_NONE, [&](auto act) {
   with_edges(n - lane * V + 64 * V <= a.cols, [&](auto full) {
    constexpr int kAct = decltype(act)::value;
    constexpr bool kFull = decltype(full)::value;
    constexpr int kRows = 4;  // in flight
    for (uint64_t m0 = first + wave; m0 < end; m0 += 4 * kRows) {
      u32x4 dy[kRows], z[kRows];
#pragma unroll
      for (int q = 0; q < kRows; ++q) {
        const uint64_t m = m0 + 4 * q < end ? m0 + 4 * q : end - 1;
        const int there = kFull ? V : valid;
        dy[q] = load_upto<C>(a.dy + (m * a.dy_stride + n) * C::kElemBytes, there);
        if constexpr (kAct != MSCL_ACT_NONE) z[q] = load_upto<C>(a.z + (m * a.z_stride + n) * C::kElemBytes, there);
      }
#pragma unroll
      for (int q = 0; q < kRows; ++q) {
        if (m0 + 4 * q >= end) continue;
        float g[V];
        C::unpack(dy[q], g);
        if constexpr (kAct != MSCL_ACT_NONE) {
          float t[V];
          C::unpack(z[q], t);
#pragma unroll
          for (int i = 0; i < V; ++i) g[i] *= slope<kAct, kFast>(t[i]);
        }
#pragma unroll
        for (int i = 0; i < V; ++i) sum[i] += g[i];
        // rows of dz are padded to whole vectors, and the padding is 0: that
        // is what dy reads as there
        if (a.dz && (kFull || valid > 0))
          *reinterpret_cast<u32x4*>(a.dz + ((m0 + 4 * q) * a.dz_stride + n) * C::kElemBytes) = C::pack(g);
      }
    }
   });
  });
  if (!a.sums) return;
#pragma unroll
  for (int i = 0; i < V; ++i) part[wave][lane * V + i] = sum[i];
  __syncthreads();
  float* out = a.sums + blockIdx.y * a.sums_stride;
  for (int c = threadIdx.x; c < 64 * V; c += 256) {
    const uint64_t col = static_cast<uint64_t>(blockIdx.x) * 64 * V + c;
    if (col < a.cols) out[col] = (part[0][c] + part[1][c]) + (part[2][c] + part[3][c]);
  }
}

}  // namespace mscl
