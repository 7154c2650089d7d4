// Layer norm over the rows of a matrix, and its backward pass, on gfx950.
//
//   mean = sum(x) / W,  rstd = 1 / sqrt(sum((x - mean)^2) / W + eps)
//   y = (x - mean) rstd w + b
// and, with h = (x - mean) rstd and g = dy w,
//   dx = rstd (g - mean(g) - h mean(g h)),  dw = sum_rows dy h,  db = sum_rows dy.
// All sums, statistics and products are binary32; each result is rounded once.
//
// These are passes over memory (8 and 16 operations an element), so a row is
// read once and held in registers between its reductions and its results:
// the variance is the second pass over the held values, not E[x^2] - mean^2.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "../../include/mscl.h"
#include "codec.hpp"
#include "linear.hpp"

namespace mscl {

// Sum over `kThreads` threads (whole waves), the same value in all of them.
// `slot` alternates between two LDS arrays, so one barrier a call is enough.
template <int kThreads, int kN>
__device__ inline void block_sums(float (&v)[kN], float (*lds)[kThreads / 64][kN], int slot) {
#pragma unroll
  for (int i = 0; i < kN; ++i)
#pragma unroll
    for (int d = 32; d > 0; d >>= 1) v[i] += __shfl_xor(v[i], d, 64);
  if constexpr (kThreads > 64) {
    const int wave = threadIdx.x >> 6;
    if ((threadIdx.x & 63) == 0)
#pragma unroll
      for (int i = 0; i < kN; ++i) lds[slot][wave][i] = v[i];
    __syncthreads();
#pragma unroll
    for (int i = 0; i < kN; ++i) {
      float s = 0.0f;
#pragma unroll
      for (int w = 0; w < kThreads / 64; ++w) s += lds[slot][w][i];
      v[i] = s;
    }
  }
}

// kV values of parameter type P from element n on (`valid` of them exist).
template <class P, int kV>
__device__ inline void load_params(const char* base, uint64_t n, int valid, float fill, float* out) {
  if (!base) {
#pragma unroll
    for (int i = 0; i < kV; ++i) out[i] = fill;
    return;
  }
  static_assert(kV % P::V == 0, "parameters have the input's type or binary32");
#pragma unroll
  for (int i = 0; i < kV; i += P::V) {
    float t[P::V];
    P::unpack(load_upto<P>(base + (n + i) * P::kElemBytes, valid - i), t);
#pragma unroll
    for (int c = 0; c < P::V; ++c) out[i + c] = t[c];
  }
}

template <class C>
__device__ inline void store_upto(char* p, const float* v, int valid) {
  const u32x4 b = C::pack(v);
  if (valid >= C::V)
    store_loose<C>(p, b);
  else if (valid > 0)
    store_partial<C>(p, 0, b, valid);
}

struct NormArgs {
  const char* x;
  const char* w;  // null: 1
  const char* b;  // null: 0
  char* y;
  float* mean;    // null: not wanted
  float* rstd;
  uint64_t x_stride, y_stride, rows, width;
  float eps;
};

// kThreads threads and kVecs 16-byte vectors each hold one row; a workgroup
// has 256 / kThreads rows when kThreads is one wave.
template <class C, class P, int kThreads, int kVecs>
__global__ __launch_bounds__(kThreads < 256 ? 256 : kThreads) void norm_rows(const NormArgs a) {
  constexpr int V = C::V;
  constexpr int kRows = kThreads < 256 ? 256 / kThreads : 1;
  static_assert(kThreads == 64 || kThreads >= 256, "a row is one wave's or one workgroup's");
  __shared__ float lds[2][kThreads / 64][1];
  const int tid = kThreads < 256 ? threadIdx.x & (kThreads - 1) : threadIdx.x;
  const uint64_t row = static_cast<uint64_t>(blockIdx.x) * kRows + (kThreads < 256 ? threadIdx.x / kThreads : 0);
  if (row >= a.rows) return;  // a whole wave's row, or never
  const char* x = a.x + row * a.x_stride * C::kElemBytes;
  float v[kVecs][V];
  float s[1] = {0.0f};
#pragma unroll
  for (int k = 0; k < kVecs; ++k) {
    const uint64_t n = (static_cast<uint64_t>(k) * kThreads + tid) * V;
    const int valid = n >= a.width ? 0 : (a.width - n < V ? static_cast<int>(a.width - n) : V);
    C::unpack(load_upto<C>(x + n * C::kElemBytes, valid), v[k]);
  }
#pragma unroll
  for (int k = 0; k < kVecs; ++k)
#pragma unroll
    for (int i = 0; i < V; ++i) s[0] += v[k][i];
  block_sums<kThreads, 1>(s, lds, 0);
  const float inv = 1.0f / static_cast<float>(a.width);
  const float mean = s[0] * inv;
  s[0] = 0.0f;
#pragma unroll
  for (int k = 0; k < kVecs; ++k)
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const uint64_t n = (static_cast<uint64_t>(k) * kThreads + tid) * V + i;
      const float d = v[k][i] - mean;
      v[k][i] = d;
      s[0] += n < a.width ? d * d : 0.0f;
    }
  block_sums<kThreads, 1>(s, lds, 1);
  const float rstd = 1.0f / sqrtf(s[0] * inv + a.eps);
  if (tid == 0) {
    if (a.mean) a.mean[row] = mean;
    if (a.rstd) a.rstd[row] = rstd;
  }
  char* y = a.y + row * a.y_stride * C::kElemBytes;
#pragma unroll
  for (int k = 0; k < kVecs; ++k) {
    const uint64_t n = (static_cast<uint64_t>(k) * kThreads + tid) * V;
    const int valid = n >= a.width ? 0 : (a.width - n < V ? static_cast<int>(a.width - n) : V);
    if (valid <= 0) continue;
    float w[V], b[V];
    load_params<P, V>(a.w, n, valid, 1.0f, w);
    load_params<P, V>(a.b, n, valid, 0.0f, b);
#pragma unroll
    for (int i = 0; i < V; ++i) w[i] = fmaf(v[k][i] * rstd, w[i], b[i]);
    store_upto<C>(y + n * C::kElemBytes, w, valid);
  }
}

// Rows too wide for registers: the row is read three times (twice from cache).
template <class C, class P>
__global__ __launch_bounds__(1024) void norm_rows_wide(const NormArgs a) {
  constexpr int V = C::V;
  __shared__ float lds[2][16][1];
  const uint64_t row = blockIdx.x;
  const char* x = a.x + row * a.x_stride * C::kElemBytes;
  char* y = a.y + row * a.y_stride * C::kElemBytes;
  const float inv = 1.0f / static_cast<float>(a.width);
  float s[1] = {0.0f};
  auto each = [&](auto&& fn) {
    for (uint64_t n = static_cast<uint64_t>(threadIdx.x) * V; n < a.width; n += 1024 * V) {
      const int valid = a.width - n < V ? static_cast<int>(a.width - n) : V;
      float v[V];
      C::unpack(load_upto<C>(x + n * C::kElemBytes, valid), v);
      fn(n, valid, v);
    }
  };
  each([&](uint64_t, int, float* v) {
    float t = 0.0f;
#pragma unroll
    for (int i = 0; i < V; ++i) t += v[i];
    s[0] += t;
  });
  block_sums<1024, 1>(s, lds, 0);
  const float mean = s[0] * inv;
  s[0] = 0.0f;
  each([&](uint64_t, int valid, float* v) {
    float t = 0.0f;
#pragma unroll
    for (int i = 0; i < V; ++i) t += i < valid ? (v[i] - mean) * (v[i] - mean) : 0.0f;
    s[0] += t;
  });
  block_sums<1024, 1>(s, lds, 1);
  const float rstd = 1.0f / sqrtf(s[0] * inv + a.eps);
  if (threadIdx.x == 0) {
    if (a.mean) a.mean[row] = mean;
    if (a.rstd) a.rstd[row] = rstd;
  }
  each([&](uint64_t n, int valid, float* v) {
    float w[V], b[V];
    load_params<P, V>(a.w, n, valid, 1.0f, w);
    load_params<P, V>(a.b, n, valid, 0.0f, b);
#pragma unroll
    for (int i = 0; i < V; ++i) w[i] = fmaf((v[i] - mean) * rstd, w[i], b[i]);
    store_upto<C>(y + n * C::kElemBytes, w, valid);
  });
}

// ------------------------------------------------------------------ backward

struct NormBackArgs {
  const char* dy;
  const char* x;
  const float* mean;
  const float* rstd;
  const char* w;  // null: 1
  char* dx;       // null: not wanted
  float* sums;    // [groups][2][sums_stride]: dw then db; null: not wanted
  uint64_t dy_stride, x_stride, dx_stride, sums_stride, rows, width;
  uint32_t rows_per_group;
};

// dx alone, a row per workgroup (or per wave), held in registers.
template <class C, class P, int kThreads, int kVecs>
__global__ __launch_bounds__(kThreads < 256 ? 256 : kThreads) void norm_back_rows(const NormBackArgs a) {
  constexpr int V = C::V;
  constexpr int kRows = kThreads < 256 ? 256 / kThreads : 1;
  __shared__ float lds[1][kThreads / 64][2];
  const int tid = kThreads < 256 ? threadIdx.x & (kThreads - 1) : threadIdx.x;
  const uint64_t row = static_cast<uint64_t>(blockIdx.x) * kRows + (kThreads < 256 ? threadIdx.x / kThreads : 0);
  if (row >= a.rows) return;
  const char* x = a.x + row * a.x_stride * C::kElemBytes;
  const char* dy = a.dy + row * a.dy_stride * C::kElemBytes;
  const float mean = a.mean[row], rstd = a.rstd[row];
  u32x4 xb[kVecs], gb[kVecs];
#pragma unroll
  for (int k = 0; k < kVecs; ++k) {
    const uint64_t n = (static_cast<uint64_t>(k) * kThreads + tid) * V;
    const int valid = n >= a.width ? 0 : (a.width - n < V ? static_cast<int>(a.width - n) : V);
    xb[k] = load_upto<C>(x + n * C::kElemBytes, valid);
    gb[k] = load_upto<C>(dy + n * C::kElemBytes, valid);
  }
  float g[kVecs][V], h[kVecs][V];
  float s[2] = {0.0f, 0.0f};
#pragma unroll
  for (int k = 0; k < kVecs; ++k) {
    const uint64_t n = (static_cast<uint64_t>(k) * kThreads + tid) * V;
    const int valid = n >= a.width ? 0 : (a.width - n < V ? static_cast<int>(a.width - n) : V);
    float w[V];
    load_params<P, V>(a.w, n, valid, 1.0f, w);
    C::unpack(xb[k], h[k]);
    C::unpack(gb[k], g[k]);
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const bool in = i < valid;
      h[k][i] = in ? (h[k][i] - mean) * rstd : 0.0f;
      g[k][i] = in ? g[k][i] * w[i] : 0.0f;
      s[0] += g[k][i];
      s[1] = fmaf(g[k][i], h[k][i], s[1]);
    }
  }
  block_sums<kThreads, 2>(s, lds, 0);
  const float inv = 1.0f / static_cast<float>(a.width);
  const float c0 = s[0] * inv, c1 = s[1] * inv;
  char* dx = a.dx + row * a.dx_stride * C::kElemBytes;
#pragma unroll
  for (int k = 0; k < kVecs; ++k) {
    const uint64_t n = (static_cast<uint64_t>(k) * kThreads + tid) * V;
    const int valid = n >= a.width ? 0 : (a.width - n < V ? static_cast<int>(a.width - n) : V);
    float d[V];
#pragma unroll
    for (int i = 0; i < V; ++i) d[i] = rstd * (g[k][i] - c0 - h[k][i] * c1);
    store_upto<C>(dx + n * C::kElemBytes, d, valid);
  }
}

// dx of rows too wide for registers: two passes over the row.
template <class C, class P>
__global__ __launch_bounds__(1024) void norm_back_rows_wide(const NormBackArgs a) {
  constexpr int V = C::V;
  __shared__ float lds[1][16][2];
  const uint64_t row = blockIdx.x;
  const char* x = a.x + row * a.x_stride * C::kElemBytes;
  const char* dy = a.dy + row * a.dy_stride * C::kElemBytes;
  char* dx = a.dx + row * a.dx_stride * C::kElemBytes;
  const float mean = a.mean[row], rstd = a.rstd[row];
  float s[2] = {0.0f, 0.0f};
  auto each = [&](auto&& fn) {
    for (uint64_t n = static_cast<uint64_t>(threadIdx.x) * V; n < a.width; n += 1024 * V) {
      const int valid = a.width - n < V ? static_cast<int>(a.width - n) : V;
      float h[V], g[V], w[V];
      C::unpack(load_upto<C>(x + n * C::kElemBytes, valid), h);
      C::unpack(load_upto<C>(dy + n * C::kElemBytes, valid), g);
      load_params<P, V>(a.w, n, valid, 1.0f, w);
#pragma unroll
      for (int i = 0; i < V; ++i) {
        h[i] = i < valid ? (h[i] - mean) * rstd : 0.0f;
        g[i] = i < valid ? g[i] * w[i] : 0.0f;
      }
      fn(n, valid, h, g);
    }
  };
  each([&](uint64_t, int, float* h, float* g) {
#pragma unroll
    for (int i = 0; i < V; ++i) {
      s[0] += g[i];
      s[1] = fmaf(g[i], h[i], s[1]);
    }
  });
  block_sums<1024, 2>(s, lds, 0);
  const float inv = 1.0f / static_cast<float>(a.width);
  const float c0 = s[0] * inv, c1 = s[1] * inv;
  each([&](uint64_t n, int valid, float* h, float* g) {
    float d[V];
#pragma unroll
    for (int i = 0; i < V; ++i) d[i] = rstd * (g[i] - c0 - h[i] * c1);
    store_upto<C>(dx + n * C::kElemBytes, d, valid);
  });
}

// dw and db over a group of rows: 64 lanes cover 64 V columns, the 4 waves
// take the group's rows in turn.
template <class C>
__global__ __launch_bounds__(256) void norm_back_columns(const NormBackArgs a) {
  constexpr int V = C::V;
  __shared__ float part[4][64 * V];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const uint64_t n = (static_cast<uint64_t>(blockIdx.x) * 64 + lane) * V;
  const int valid = n >= a.width ? 0 : (a.width - n < V ? static_cast<int>(a.width - n) : V);
  const uint64_t first = static_cast<uint64_t>(blockIdx.y) * a.rows_per_group;
  uint64_t end = first + a.rows_per_group;
  if (end > a.rows) end = a.rows;
  float dw[V], db[V];
#pragma unroll
  for (int i = 0; i < V; ++i) dw[i] = db[i] = 0.0f;
#pragma unroll 2
  for (uint64_t row = first + wave; row < end; row += 4) {
    const float mean = a.mean[row], rstd = a.rstd[row];
    float h[V], g[V];
    C::unpack(load_upto<C>(a.x + (row * a.x_stride + n) * C::kElemBytes, valid), h);
    C::unpack(load_upto<C>(a.dy + (row * a.dy_stride + n) * C::kElemBytes, valid), g);
#pragma unroll
    for (int i = 0; i < V; ++i) {
      dw[i] = fmaf(g[i], (h[i] - mean) * rstd, dw[i]);
      db[i] += g[i];
    }
  }
  for (int which = 0; which < 2; ++which) {
    if (which) __syncthreads();
#pragma unroll
    for (int i = 0; i < V; ++i) part[wave][lane * V + i] = which ? db[i] : dw[i];
    __syncthreads();
    float* out = a.sums + (2 * static_cast<uint64_t>(blockIdx.y) + which) * a.sums_stride;
    for (int c = threadIdx.x; c < 64 * V; c += 256) {
      const uint64_t col = static_cast<uint64_t>(blockIdx.x) * 64 * V + c;
      if (col < a.width) out[col] = (part[0][c] + part[1][c]) + (part[2][c] + part[3][c]);
    }
  }
}

// ------------------------------------------------------------------ column sums

struct JoinArgs {
  const float* sums;  // [groups][kinds][stride]
  char* out[2];       // null: not wanted
  uint64_t stride, width;
  uint32_t groups, kinds;
};

// Adds the groups' column sums (blockIdx.y: the kind) in a fixed order and
// rounds them: 32 columns a workgroup, 8 threads a column.
template <class P>
__global__ __launch_bounds__(256) void column_join(const JoinArgs a) {
  __shared__ float part[8][33];
  const int c = threadIdx.x & 31, q = threadIdx.x >> 5;
  const uint64_t col = static_cast<uint64_t>(blockIdx.x) * 32 + c;
  const uint32_t kind = blockIdx.y;
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

}  // namespace mscl
