// Rows to 8-bit integers with a scale for each, on gfx950: a pass over memory
// that holds a row in registers between finding its largest size and rounding.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "../../include/mscl.h"
#include "codec.hpp"
#include "linear.hpp"

namespace mscl {

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
// Memory bounds it: 8192 x 8192 bf16 36.8 us (5.5 TB/s); 32 x 8192 3.1 us, one
// way through a row.
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
