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

// A thread's vectors of a row start at 16-byte boundaries of memory, whatever
// the row's own start: the row is taken as beginning `shift` elements before
// its first one.  16 bytes off such a boundary take two cache requests (4099
// rows of 5001 fp16: 23 us, of 5000 19 us).  Vector k of thread t holds the
// columns from n on, of which lo .. hi - 1 exist.
template <class C, int kThreads>
struct Span16 {
  int64_t n;
  int lo, hi;
  __device__ inline Span16(uint64_t width, int shift, int k, int tid) {
    n = (static_cast<int64_t>(k) * kThreads + tid) * C::V - shift;
    const int64_t left = static_cast<int64_t>(width) - n;
    lo = n < 0 ? static_cast<int>(-n) : 0;
    hi = left <= 0 ? 0 : (left < C::V ? static_cast<int>(left) : C::V);
  }
  __device__ inline bool whole() const { return lo == 0 && hi == C::V; }
  __device__ inline bool none() const { return lo >= hi; }
};

template <class C>
__device__ inline int shift_of(const char* row) {
  return static_cast<int>(reinterpret_cast<uintptr_t>(row) & 15) / C::kElemBytes;
}

// Elements lo .. hi - 1 of the V at p; the others read as 0.
template <class C>
__device__ inline u32x4 load_between(const char* p, int lo, int hi) {
  if (lo == 0) return load_upto<C>(p, hi);
  u32x4 v = {0u, 0u, 0u, 0u};
#pragma unroll
  for (int i = 0; i < C::V; ++i)
    if (i >= lo && i < hi) {
      const uint32_t bits = reinterpret_cast<const typename C::Bits*>(p)[i];
      if constexpr (C::kElemBytes == 4)
        v[i] = bits;
      else
        v[i >> 1] |= bits << (16 * (i & 1));
    }
  return v;
}
template <class C>
__device__ inline void store_between(char* p, const float* v, int lo, int hi) {
  if (lo == 0) return store_upto<C>(p, v, hi);
  const u32x4 b = C::pack(v);
#pragma unroll
  for (int i = 0; i < C::V; ++i)
    if (i >= lo && i < hi) {
      if constexpr (C::kElemBytes == 4)
        reinterpret_cast<uint32_t*>(p)[i] = b[i];
      else
        reinterpret_cast<uint16_t*>(p)[i] = static_cast<uint16_t>(b[i >> 1] >> (16 * (i & 1)));
    }
}

// load_params for a vector whose first elements may not exist.
template <class P, int kV>
__device__ inline void load_params_between(const char* base, int64_t n, int lo, int hi, float fill, float* out) {
  if (!base || lo == 0) return load_params<P, kV>(base, n, hi, fill, out);
#pragma unroll
  for (int i = 0; i < kV; i += P::V)
    P::unpack(load_between<P>(base + (n + i) * P::kElemBytes, lo - i < 0 ? 0 : lo - i, hi - i), out + i);
}

// kThreads threads and kVecs 16-byte vectors each hold one row; a workgroup
// has 256 / kThreads rows when kThreads is one wave.  A row per workgroup and
// many workgroups a compute unit: workgroups that stay, keep the parameters
// and fetch the next row ahead were slower (8192 x 8192 bf16 56 against 52 us,
// 4099 x 5001 fp16 25 against 21.5), as they need twice the registers.
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
  const int shift = shift_of<C>(x);
  u32x4 held[kVecs];
#pragma unroll
  for (int k = 0; k < kVecs; ++k) {
    const Span16<C, kThreads> s(a.width, shift, k, tid);
    held[k] = load_between<C>(x + s.n * C::kElemBytes, s.lo, s.hi);
  }
  const float inv = 1.0f / static_cast<float>(a.width);
  float v[kVecs][V];
  float s[1] = {0.0f};
#pragma unroll
  for (int k = 0; k < kVecs; ++k) {
    C::unpack(held[k], v[k]);
#pragma unroll
    for (int i = 0; i < V; ++i) s[0] += v[k][i];
  }
  block_sums<kThreads, 1>(s, lds, 0);
  const float mean = s[0] * inv;
  s[0] = 0.0f;
#pragma unroll
  for (int k = 0; k < kVecs; ++k) {
    const Span16<C, kThreads> sp(a.width, shift, k, tid);
    const bool whole = sp.whole();
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const float d = v[k][i] - mean;
      v[k][i] = d;
      s[0] += whole || (i >= sp.lo && i < sp.hi) ? d * d : 0.0f;
    }
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
    const Span16<C, kThreads> sp(a.width, shift, k, tid);
    if (sp.none()) continue;
    float w[V], b[V];
    load_params_between<P, V>(a.w, sp.n, sp.lo, sp.hi, 1.0f, w);
    load_params_between<P, V>(a.b, sp.n, sp.lo, sp.hi, 0.0f, b);
#pragma unroll
    for (int i = 0; i < V; ++i) w[i] = fmaf(v[k][i] * rstd, w[i], b[i]);
    store_between<C>(y + sp.n * C::kElemBytes, w, sp.lo, sp.hi);
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

// Takes from the compiler what it knows of a held vector, so that values
// derived from it are derived again after a reduction and not kept through it
// (two rows of 8192 16-bit elements: 64 registers less, and no spills).
__device__ inline void forget(u32x4& v) { asm volatile("" : "+v"(v)); }

struct NormBackArgs {
  const char* dy;
  const char* x;
  const float* mean;
  const float* rstd;
  const char* w;  // null: 1
  char* dx;       // null: not wanted
  float* sums;    // [groups][2][sums_stride]: dw then db; null: not wanted
  float* along;   // [rows][column blocks][2]: a block's sums of g and of g h
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
  // (g, h) of one vector, derived before and after the reduction
  auto derive = [&](int k, float* g, float* h) {
    const uint64_t n = (static_cast<uint64_t>(k) * kThreads + tid) * V;
    const int valid = n >= a.width ? 0 : (a.width - n < V ? static_cast<int>(a.width - n) : V);
    float w[V];
    load_params<P, V>(a.w, n, valid, 1.0f, w);
    C::unpack(xb[k], h);
    C::unpack(gb[k], g);
#pragma unroll
    for (int i = 0; i < V; ++i) {
      h[i] = i < valid ? (h[i] - mean) * rstd : 0.0f;
      g[i] = i < valid ? g[i] * w[i] : 0.0f;
    }
  };
  float s[2] = {0.0f, 0.0f};
#pragma unroll
  for (int k = 0; k < kVecs; ++k) {
    float g[V], h[V];
    derive(k, g, h);
#pragma unroll
    for (int i = 0; i < V; ++i) {
      s[0] += g[i];
      s[1] = fmaf(g[i], h[i], s[1]);
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
    float g[V], h[V];
    forget(xb[k]);
    forget(gb[k]);
    derive(k, g, h);
#pragma unroll
    for (int i = 0; i < V; ++i) g[i] = rstd * (g[i] - c0 - h[i] * c1);
    store_upto<C>(dx + n * C::kElemBytes, g, valid);
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

// The rows that a wave of the two kernels below has in flight, 4 apart.  Rows
// past `end` are read as the last one and count as 0.  kFull: all of the
// wave's vectors are whole, so that no load hangs on a lane's branch.
constexpr int kTileRows = 4;
template <class C, bool kFull>
struct TileRows {
  u32x4 x[kTileRows], dy[kTileRows];
  float mean[kTileRows], rstd[kTileRows];
  __device__ inline void load(const NormBackArgs& a, uint64_t row0, uint64_t end, uint64_t n, int valid) {
#pragma unroll
    for (int q = 0; q < kTileRows; ++q) {
      const uint64_t row = row0 + 4 * q < end ? row0 + 4 * q : end - 1;
      mean[q] = a.mean[row];
      rstd[q] = a.rstd[row];
      x[q] = load_upto<C>(a.x + (row * a.x_stride + n) * C::kElemBytes, kFull ? C::V : valid);
      dy[q] = load_upto<C>(a.dy + (row * a.dy_stride + n) * C::kElemBytes, kFull ? C::V : valid);
    }
#pragma unroll
    for (int q = 0; q < kTileRows; ++q)
      if (row0 + 4 * q >= end) {
        mean[q] = rstd[q] = 0.0f;
        x[q] = dy[q] = u32x4{0u, 0u, 0u, 0u};  // x too: 0 times an infinity there would be NaN
      }
  }
};

// Few rows: two launches.  The first reads x and dy by tiles (a group of rows
// by 64 V columns; the 4 waves take the group's rows in turn) and sums both
// ways: down its columns for dw and db, along its part of each row for dx's
// two means.
template <class C, class P>
__global__ __launch_bounds__(256) void norm_back_tiles(const NormBackArgs a) {
  constexpr int V = C::V;
  __shared__ float part[4][64 * V];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const uint64_t n = (static_cast<uint64_t>(blockIdx.x) * 64 + lane) * V;
  const int valid = n >= a.width ? 0 : (a.width - n < V ? static_cast<int>(a.width - n) : V);
  const uint64_t first = static_cast<uint64_t>(blockIdx.y) * a.rows_per_group;
  uint64_t end = first + a.rows_per_group;
  if (end > a.rows) end = a.rows;
  float dw[V], db[V], w[V];
  load_params<P, V>(a.w, n, valid, 1.0f, w);
#pragma unroll
  for (int i = 0; i < V; ++i) dw[i] = db[i] = 0.0f;
  with_edges(n - lane * V + 64 * V <= a.width, [&](auto full) {
    constexpr bool kFull = decltype(full)::value;
    for (uint64_t row0 = first + wave; row0 < end; row0 += 4 * kTileRows) {
      TileRows<C, kFull> rows;
      rows.load(a, row0, end, n, valid);
      float s[kTileRows][2];
#pragma unroll
      for (int q = 0; q < kTileRows; ++q) {
        float h[V], g[V];
        C::unpack(rows.x[q], h);
        C::unpack(rows.dy[q], g);
        s[q][0] = s[q][1] = 0.0f;
#pragma unroll
        for (int i = 0; i < V; ++i) {
          h[i] = kFull || i < valid ? (h[i] - rows.mean[q]) * rows.rstd[q] : 0.0f;
          dw[i] = fmaf(g[i], h[i], dw[i]);
          db[i] += g[i];
          const float gw = kFull || i < valid ? g[i] * w[i] : 0.0f;
          s[q][0] += gw;
          s[q][1] = fmaf(gw, h[i], s[q][1]);
        }
      }
      if (a.dx) {
#pragma unroll
        for (int d = 32; d > 0; d >>= 1)
#pragma unroll
          for (int q = 0; q < kTileRows; ++q) {
            s[q][0] += __shfl_xor(s[q][0], d, 64);
            s[q][1] += __shfl_xor(s[q][1], d, 64);
          }
#pragma unroll
        for (int q = 0; q < kTileRows; ++q)
          if (lane == 0 && row0 + 4 * q < end)
            *reinterpret_cast<f32x2*>(a.along + ((row0 + 4 * q) * gridDim.x + blockIdx.x) * 2) = f32x2{s[q][0], s[q][1]};
      }
    }
  });
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

// dx, dw and db in one pass over x and dy, for many rows.  A workgroup of
// 512 threads stays and walks over the rows: kThreads of them hold a row
// (so 512 / kThreads rows side by side), kRows rows in turn go through one
// reduction, and each thread keeps its columns' weights and its columns' sums
// of dw and db in registers.  The next rows are on their way while the present
// ones are reduced.  At the end each workgroup writes one row of partial sums
// of dw and of db, which column_join adds: 256 workgroups' partial sums are
// 4 KiB a column, a second read of x and dy 4 or 8 bytes a row and column.
template <class C, class P, int kThreads, int kVecs, int kRows>
__global__ __launch_bounds__(512) void norm_back_fused(const NormBackArgs a) {
  constexpr int V = C::V;
  constexpr int kSlots = 512 / kThreads, kWaves = kThreads / 64;
  __shared__ float lds[2][8][2 * kRows];
  const int tid = threadIdx.x % kThreads;
  const int slot = __builtin_amdgcn_readfirstlane(threadIdx.x / kThreads);
  int valid[kVecs];
  float w[kVecs][V], dw[kVecs][V], db[kVecs][V];
#pragma unroll
  for (int k = 0; k < kVecs; ++k) {
    const uint64_t n = (static_cast<uint64_t>(k) * kThreads + tid) * V;
    valid[k] = n >= a.width ? 0 : (a.width - n < V ? static_cast<int>(a.width - n) : V);
    load_params<P, V>(a.w, n, valid[k], 1.0f, w[k]);
#pragma unroll
    for (int i = 0; i < V; ++i) dw[k][i] = db[k][i] = 0.0f;
  }
  const uint64_t round = static_cast<uint64_t>(gridDim.x) * kSlots * kRows;
  uint64_t row0 = (static_cast<uint64_t>(blockIdx.x) * kSlots + slot) * kRows;
  struct Held {
    u32x4 x[kVecs], dy[kVecs];
    float mean, rstd;
  };
  Held now[kRows], next[kRows];
  auto load = [&](Held* to, uint64_t first) {
#pragma unroll
    for (int q = 0; q < kRows; ++q) {
      const uint64_t row = first + q;
      const bool in = row < a.rows;  // a row that is not there adds 0 to every sum
      to[q].mean = in ? a.mean[row] : 0.0f;
      to[q].rstd = in ? a.rstd[row] : 0.0f;
#pragma unroll
      for (int k = 0; k < kVecs; ++k) {
        const uint64_t n = (static_cast<uint64_t>(k) * kThreads + tid) * V;
        to[q].x[k] = load_upto<C>(a.x + (row * a.x_stride + n) * C::kElemBytes, in ? valid[k] : 0);
        to[q].dy[k] = load_upto<C>(a.dy + (row * a.dy_stride + n) * C::kElemBytes, in ? valid[k] : 0);
      }
    }
  };
  const float inv = 1.0f / static_cast<float>(a.width);
  int turn = 0;
  load(now, row0);
  // every wave of the workgroup runs the same number of rounds
  for (uint64_t first = static_cast<uint64_t>(blockIdx.x) * kSlots * kRows; first < a.rows; first += round) {
    load(next, row0 + round);
    float s[2 * kRows];
#pragma unroll
    for (int q = 0; q < kRows; ++q) {
      s[2 * q] = s[2 * q + 1] = 0.0f;
#pragma unroll
      for (int k = 0; k < kVecs; ++k) {
        float h[V], g[V];
        C::unpack(now[q].x[k], h);
        C::unpack(now[q].dy[k], g);
#pragma unroll
        for (int i = 0; i < V; ++i) {
          h[i] = i < valid[k] ? (h[i] - now[q].mean) * now[q].rstd : 0.0f;
          dw[k][i] = fmaf(g[i], h[i], dw[k][i]);
          db[k][i] += g[i];
          const float gw = i < valid[k] ? g[i] * w[k][i] : 0.0f;
          s[2 * q] += gw;
          s[2 * q + 1] = fmaf(gw, h[i], s[2 * q + 1]);
        }
      }
    }
#pragma unroll
    for (int i = 0; i < 2 * kRows; ++i)
#pragma unroll
      for (int d = 32; d > 0; d >>= 1) s[i] += __shfl_xor(s[i], d, 64);
    if constexpr (kWaves > 1) {
      if ((threadIdx.x & 63) == 0)
#pragma unroll
        for (int i = 0; i < 2 * kRows; ++i) lds[turn][threadIdx.x >> 6][i] = s[i];
      __syncthreads();
#pragma unroll
      for (int i = 0; i < 2 * kRows; ++i) {
        s[i] = 0.0f;
#pragma unroll
        for (int v = 0; v < kWaves; ++v) s[i] += lds[turn][slot * kWaves + v][i];
      }
      turn ^= 1;
    }
    if (a.dx) {
#pragma unroll
      for (int q = 0; q < kRows; ++q) {
        if (row0 + q >= a.rows) continue;
        const float c0 = s[2 * q] * inv, c1 = s[2 * q + 1] * inv;
#pragma unroll
        for (int k = 0; k < kVecs; ++k) {
          const uint64_t n = (static_cast<uint64_t>(k) * kThreads + tid) * V;
          float h[V], g[V];
          forget(now[q].x[k]);
          forget(now[q].dy[k]);
          C::unpack(now[q].x[k], h);
          C::unpack(now[q].dy[k], g);
#pragma unroll
          for (int i = 0; i < V; ++i)
            g[i] = now[q].rstd * (g[i] * w[k][i] - c0 - (h[i] - now[q].mean) * now[q].rstd * c1);
          store_upto<C>(a.dx + ((row0 + q) * a.dx_stride + n) * C::kElemBytes, g, valid[k]);
        }
      }
    }
#pragma unroll
    for (int q = 0; q < kRows; ++q) now[q] = next[q];
    row0 += round;
  }
  if constexpr (kSlots == 1) {
#pragma unroll
    for (int which = 0; which < 2; ++which) {
      float* out = a.sums + (2 * static_cast<uint64_t>(blockIdx.x) + which) * a.sums_stride;
#pragma unroll
      for (int k = 0; k < kVecs; ++k) {
        const uint64_t n = (static_cast<uint64_t>(k) * kThreads + tid) * V;
#pragma unroll
        for (int i = 0; i < V; i += 4) {  // rows of the partial sums are padded to whole vectors
          const float* v = which ? &db[k][i] : &dw[k][i];
          if (n + i < a.width) *reinterpret_cast<f32x4*>(out + n + i) = f32x4{v[0], v[1], v[2], v[3]};
        }
      }
    }
  } else {
    static_assert(kSlots == 1 || kVecs == 1, "several rows side by side hold one vector a thread");
    __shared__ float part[kSlots][kThreads * V + 1];
#pragma unroll
    for (int which = 0; which < 2; ++which) {
      __syncthreads();
#pragma unroll
      for (int i = 0; i < V; ++i) part[slot][tid * V + i] = which ? db[0][i] : dw[0][i];
      __syncthreads();
      float* out = a.sums + (2 * static_cast<uint64_t>(blockIdx.x) + which) * a.sums_stride;
      for (uint64_t c = threadIdx.x; c < a.width; c += 512) {
        float t = 0.0f;
#pragma unroll
        for (int v = 0; v < kSlots; ++v) t += part[v][c];
        out[c] = t;
      }
    }
  }
}

// The second launch for few rows: the first `tiles` workgroups turn
// norm_back_tiles' row sums into dx, tile by tile (x and dy come from the
// caches by then), the others join its column sums.
template <class C, class P>
__global__ __launch_bounds__(256) void norm_back_apply(const NormBackArgs a, const JoinArgs join, uint32_t blocks,
                                                       uint32_t tiles, uint32_t joins) {
  constexpr int V = C::V;
  if (blockIdx.x >= tiles) {
    const uint32_t id = blockIdx.x - tiles;
    join_block<P>(join, id % joins, id / joins);
    return;
  }
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const uint64_t n = (static_cast<uint64_t>(blockIdx.x % blocks) * 64 + lane) * V;
  const int valid = n >= a.width ? 0 : (a.width - n < V ? static_cast<int>(a.width - n) : V);
  const uint64_t first = static_cast<uint64_t>(blockIdx.x / blocks) * a.rows_per_group;
  uint64_t end = first + a.rows_per_group;
  if (end > a.rows) end = a.rows;
  float w[V];
  load_params<P, V>(a.w, n, valid, 1.0f, w);
  const float inv = 1.0f / static_cast<float>(a.width);
  with_edges(n - lane * V + 64 * V <= a.width, [&](auto full) {
    constexpr bool kFull = decltype(full)::value;
    for (uint64_t row0 = first + wave; row0 < end; row0 += 4 * kTileRows) {
      TileRows<C, kFull> rows;
      rows.load(a, row0, end, n, valid);
      float s[kTileRows][2];
#pragma unroll
      for (int q = 0; q < kTileRows; ++q) s[q][0] = s[q][1] = 0.0f;
      for (uint32_t b = lane; b < blocks; b += 64)
#pragma unroll
        for (int q = 0; q < kTileRows; ++q)
          if (row0 + 4 * q < end) {
            const f32x2 p = *reinterpret_cast<const f32x2*>(a.along + ((row0 + 4 * q) * blocks + b) * 2);
            s[q][0] += p[0];
            s[q][1] += p[1];
          }
#pragma unroll
      for (int d = 32; d > 0; d >>= 1)
#pragma unroll
        for (int q = 0; q < kTileRows; ++q) {
          s[q][0] += __shfl_xor(s[q][0], d, 64);
          s[q][1] += __shfl_xor(s[q][1], d, 64);
        }
#pragma unroll
      for (int q = 0; q < kTileRows; ++q) {
        if (row0 + 4 * q >= end) continue;
        const float c0 = s[q][0] * inv, c1 = s[q][1] * inv;
        float h[V], g[V];
        C::unpack(rows.x[q], h);
        C::unpack(rows.dy[q], g);
#pragma unroll
        for (int i = 0; i < V; ++i)
          g[i] = rows.rstd[q] * (g[i] * w[i] - c0 - (h[i] - rows.mean[q]) * rows.rstd[q] * c1);
        store_upto<C>(a.dx + ((row0 + 4 * q) * a.dx_stride + n) * C::kElemBytes, g, kFull ? V : valid);
      }
    }
  });
}

}  // namespace mscl
