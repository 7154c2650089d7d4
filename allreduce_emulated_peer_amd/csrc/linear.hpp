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
// the 16-bit types and v_mfma_f32_16x16x4_f32 for binary32.  The B tile is
// given as the instruction's first operand, so a lane ends up with four
// neighbouring columns n of one row m; v_permlane16_swap of two
// neighbouring tiles makes eight, one 16-byte store of a 16-bit type.
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

// ------------------------------------------------------------------ activations

// Activations and their slopes in binary32.  kFast is taken where the result
// is rounded to 16 bits: the hardware's exp2 and reciprocal (1 ulp each), and
// erfc by Abramowitz & Stegun 7.1.26 (absolute error 1.5e-7), against
// roundings of 2^-9 and 2^-12.  binary32 results use the math library.
// The Gaussian tail is computed as erfc(|z|), never as 1 + erf(z), so small
// values at negative z keep their relative accuracy.
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
    const float u = fabsf(z) * 0.70710678118654752440f;
    const float t = __builtin_amdgcn_rcpf(fmaf(0.3275911f, u, 1.0f));
    float p = fmaf(1.061405429f, t, -1.453152027f);
    p = fmaf(p, t, 1.421413741f);
    p = fmaf(p, t, -0.284496736f);
    p = fmaf(p, t, 0.254829592f);
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

// Finishes V neighbouring sums of row m from column n on, and stores them.
template <class C, int kAct>
__device__ inline void finish(const Epilogue& e, uint64_t m, uint64_t n, float* v) {
  constexpr int V = C::V;
  constexpr bool kFast = C::kElemBytes == 2;
  if (m >= e.m || n >= e.n) return;
  const int valid = e.n - n < V ? static_cast<int>(e.n - n) : V;
  const bool full = valid == V;
  float t[V];
  if (e.bias) {
    C::unpack(load_upto<C>(e.bias + n * C::kElemBytes, valid), t);
#pragma unroll
    for (int i = 0; i < V; ++i) v[i] += t[i];
  }
  if (e.z) {
    char* p = e.z + (m * e.z_stride + n) * C::kElemBytes;
    const u32x4 b = C::pack(v);
    if (full)
      store_loose<C>(p, b);
    else
      store_partial<C>(p, 0, b, valid);
  }
  if constexpr (kAct != MSCL_ACT_NONE) {
#pragma unroll
    for (int i = 0; i < V; ++i) v[i] = activate<kAct, kFast>(v[i]);
  }
  if (e.residual) {
    C::unpack(load_upto<C>(e.residual + (m * e.residual_stride + n) * C::kElemBytes, valid), t);
#pragma unroll
    for (int i = 0; i < V; ++i) v[i] += t[i];
  }
  char* p = e.y + (m * e.y_stride + n) * C::kElemBytes;
  const u32x4 b = C::pack(v);
  if (full)
    store_loose<C>(p, b);
  else
    store_partial<C>(p, 0, b, valid);
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

// The sums of a wave's kM x kN tiles of 16 x 16 (tile (i, j) at row
// m0 + 16 i, column n0 + 16 j), given to fn(m, n, V values).  In tile (i, j)
// lane l holds row l % 16, columns 4 (l / 16) .. + 3; for a 16-bit type two
// neighbouring tiles trade halves, so that each lane holds eight columns.
template <class C, int kM, int kN, class Fn>
__device__ inline void each_group(f32x4 (&acc)[kM][kN], uint64_t m0, uint64_t n0, Fn&& fn) {
  const int lane = threadIdx.x & 63;
  const int r = lane & 15, g = lane >> 4;
#pragma unroll
  for (int i = 0; i < kM; ++i) {
    const uint64_t m = m0 + 16 * i + r;
    if constexpr (C::V == 4) {
#pragma unroll
      for (int j = 0; j < kN; ++j) {
        float v[4] = {acc[i][j][0], acc[i][j][1], acc[i][j][2], acc[i][j][3]};
        fn(m, n0 + 16 * j + 4 * g, v);
      }
    } else {
      static_assert(kN % 2 == 0, "16-bit tiles come in pairs");
#pragma unroll
      for (int j = 0; j < kN; j += 2) {
        float v[8];
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          float a = acc[i][j][q], b = acc[i][j + 1][q];
          swap_rows16(a, b);
          v[q] = a;
          v[4 + q] = b;
        }
        fn(m, n0 + 16 * (j + (g & 1)) + 8 * (g >> 1), v);
      }
    }
  }
}

// ------------------------------------------------------------------ general tile kernel

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
  uint32_t blocks_per_share;  // blocks of k that one share (blockIdx.y) sums
};

// One operand's kT x (128-byte block of k) tile, from memory through
// registers into LDS.  kAlong: kT rows of 128 bytes, 16-byte chunk c of row r
// at chunk c ^ (r % 8), so that eight neighbouring rows' equal chunks lie in
// different banks.  kDown: one row of kT elements for each k; 32-byte (16-bit
// types, read transposed) or 64-byte (binary32) segments are xored with bits
// of k so that the rows that one instruction reads lie in different banks.
template <class C, bool kAlong, int kT, int kThreads>
struct Stage {
  static constexpr int V = C::V;
  static constexpr int kBlock = 8 * V;  // k per block
  static constexpr int kChunks = kT * 8 / kThreads;  // 16-byte chunks per thread
  static constexpr int kBytes = kT * 128;
  static constexpr int kPerRow = kAlong ? 8 : kT / V;  // chunks per LDS row
  u32x4 held[kChunks];

  static __device__ inline int swizzle(int row, int chunk) {
    if constexpr (kAlong) return chunk ^ (row & 7);
    if constexpr (V == 8) {  // segments of 2 chunks; rows k .. k + 3 and k + 8 .. k + 11 are read at once
      constexpr int kSegs = kT / 16;
      const int key = kSegs >= 8 ? ((row & 3) | ((row >> 3 & 1) << 2)) : ((row >> 1 & 1) | ((row >> 3 & 1) << 1));
      return chunk ^ ((key & (kSegs - 1)) << 1);
    }
    return chunk ^ ((row >> 2 & 3) << 2);  // binary32: rows 4 apart are read at once
  }

  __device__ inline void load(const Operand& o, uint64_t first, uint64_t k0, uint64_t k_end) {
#pragma unroll
    for (int i = 0; i < kChunks; ++i) {
      const int id = i * kThreads + threadIdx.x;
      const int r = id / kPerRow, c = id % kPerRow;
      const uint64_t row = (kAlong ? first : k0) + r;
      const uint64_t col = (kAlong ? k0 : first) + static_cast<uint64_t>(c) * V;
      const uint64_t rows = kAlong ? o.rows : k_end;
      const uint64_t cols = kAlong ? k_end : o.cols;
      int valid = 0;
      if (row < rows && col < cols) valid = cols - col < V ? static_cast<int>(cols - col) : V;
      held[i] = load_upto<C>(o.base + (row * o.stride + col) * C::kElemBytes, valid);
    }
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
    } else if constexpr (V == 8) {
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
    } else {
      u32x4 out;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int k = 16 * s + 4 * g + j;
        const int col = p + r;
        out[j] = *reinterpret_cast<const uint32_t*>(lds + (k * kPerRow + swizzle(k, col >> 2)) * 16 + (col & 3) * 4);
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

// Any sizes, strides and alignments: kBM x kBN tiles by 4 waves in a square,
// 128 bytes of k at a time, the next block's loads in flight while the
// present one is multiplied, two LDS buffers.  blockIdx.y is the share of k.
template <class C, bool kAAlong, bool kBAlong, int kBM, int kBN>
__global__ __launch_bounds__(256) void linear_tile(const TileArgs t) {
  using SA = Stage<C, kAAlong, kBM, 256>;
  using SB = Stage<C, kBAlong, kBN, 256>;
  constexpr int kWM = kBM / 2 / 16, kWN = kBN / 2 / 16;
  __shared__ __align__(16) char lds[2 * (SA::kBytes + SB::kBytes)];
  const uint32_t tm = blockIdx.x % t.tiles_m, tn = blockIdx.x / t.tiles_m;
  const uint64_t m0 = static_cast<uint64_t>(tm) * kBM, n0 = static_cast<uint64_t>(tn) * kBN;
  const int wave = threadIdx.x >> 6;
  const int wm = (wave & 1) * (kBM / 2), wn = (wave >> 1) * (kBN / 2);
  const uint64_t k_first = static_cast<uint64_t>(blockIdx.y) * t.blocks_per_share * SA::kBlock;
  uint64_t k_end = k_first + static_cast<uint64_t>(t.blocks_per_share) * SA::kBlock;
  if (k_end > t.k) k_end = t.k;

  f32x4 acc[kWM][kWN];
#pragma unroll
  for (int i = 0; i < kWM; ++i)
#pragma unroll
    for (int j = 0; j < kWN; ++j) acc[i][j] = f32x4{0.f, 0.f, 0.f, 0.f};

  SA sa;
  SB sb;
  int buf = 0;
  if (k_first < k_end) {
    sa.load(t.a, m0, k_first, k_end);
    sb.load(t.b, n0, k_first, k_end);
    sa.store(lds);
    sb.store(lds + SA::kBytes);
  }
  __syncthreads();
  for (uint64_t k0 = k_first; k0 < k_end; k0 += SA::kBlock) {
    const bool more = k0 + SA::kBlock < k_end;
    if (more) {
      sa.load(t.a, m0, k0 + SA::kBlock, k_end);
      sb.load(t.b, n0, k0 + SA::kBlock, k_end);
    }
    const char* la = lds + buf * (SA::kBytes + SB::kBytes);
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
        for (int j = 0; j < kWN; ++j) acc[i][j] = multiply<C>(fb[j], fa[i], acc[i][j]);
    }
    if (more) {
      buf ^= 1;
      sa.store(lds + buf * (SA::kBytes + SB::kBytes));
      sb.store(lds + buf * (SA::kBytes + SB::kBytes) + SA::kBytes);
    }
    __syncthreads();
  }
  if (t.e.partial) {
    each_group<C>(acc, m0 + wm, n0 + wn,
                  [&](uint64_t m, uint64_t n, float* v) { keep_partial<C>(t.e, blockIdx.y, m, n, v); });
  } else {
    with_activation(t.e.act, [&](auto act) {
      each_group<C>(acc, m0 + wm, n0 + wn,
                    [&](uint64_t m, uint64_t n, float* v) { finish<C, decltype(act)::value>(t.e, m, n, v); });
    });
  }
}

// Adds the shares of k in their order and finishes the sums.
template <class C>
__global__ __launch_bounds__(256) void linear_join(const Epilogue e, int shares) {
  constexpr int V = C::V;
  const uint64_t per_row = (e.n + V - 1) / V;
  const uint64_t id = static_cast<uint64_t>(blockIdx.x) * 256 + threadIdx.x;
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
  with_activation(e.act, [&](auto act) { finish<C, decltype(act)::value>(e, m, n, v); });
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
// type: 2^-9 (bf16) of each term, independent from term to term, which adds
// to a product's error no more than the rounding of its result.
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
    constexpr int kAct = decltype(act)::value;
#pragma unroll 2
    for (uint64_t m = first + wave; m < end; m += 4) {
      float g[V];
      C::unpack(load_upto<C>(a.dy + (m * a.dy_stride + n) * C::kElemBytes, valid), g);
      if constexpr (kAct != MSCL_ACT_NONE) {
        float z[V];
        C::unpack(load_upto<C>(a.z + (m * a.z_stride + n) * C::kElemBytes, valid), z);
#pragma unroll
        for (int i = 0; i < V; ++i) g[i] *= slope<kAct, kFast>(z[i]);
      }
#pragma unroll
      for (int i = 0; i < V; ++i) sum[i] += g[i];
      if (a.dz) {
        char* p = a.dz + (m * a.dz_stride + n) * C::kElemBytes;
        const u32x4 b = C::pack(g);
        if (valid == V)
          store_loose<C>(p, b);
        else if (valid > 0)
          store_partial<C>(p, 0, b, valid);
      }
    }
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
