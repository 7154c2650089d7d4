// Host side that the operators' translation units share: argument checks, the
// choice of kernel, tile and split, and launches of more than one operator.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>
#include <stdio.h>
#include <string.h>

#include <algorithm>
#include <atomic>

#include "../../include/mscl.h"
#include "failure.hpp"
#include "linear.hpp"

namespace mscl {
namespace __attribute__((visibility("hidden"))) launch {

// ------------------------------------------------------------------ checks

inline mscl_status_t bad(const char* msg) { return record_failure(MSCL_ERR_INVALID_ARGUMENT, msg); }

inline mscl_status_t failed_hip(hipError_t e, const char* what) {
  char text[160];
  snprintf(text, sizeof text, "%s: %s", what, hipGetErrorString(e));
  return record_failure(MSCL_ERR_HIP, text);
}

inline size_t bytes_of(int dtype) { return dtype == MSCL_FLOAT32 ? 4 : 2; }
inline bool known_dtype(int d) { return d == MSCL_FLOAT32 || d == MSCL_FLOAT16 || d == MSCL_BFLOAT16; }

// A buffer of a call: its name for messages, where it lies, whether the call
// writes it, and the buffer that it may be exactly the same as.
struct Span {
  const char* name;
  uintptr_t first, bytes;       // from its first byte to its last one
  uintptr_t rows, pitch, width; // rows of `width` bytes, `pitch` bytes apart
  bool written;
  const char* may_be;
};

// Whether two buffers share a byte.  Column blocks of one larger matrix (rows
// equally far apart) and a single row between a matrix's rows are told apart
// exactly; matrices of different pitches share bytes if their extents do.
inline bool meet(const Span& p, const Span& q) {
  const Span &a = p.first <= q.first ? p : q, &b = p.first <= q.first ? q : p;
  const uintptr_t d = b.first - a.first;
  if (d >= a.bytes) return false;
  if (a.rows > 1 && b.rows > 1 && a.pitch != b.pitch) return true;
  if (a.rows == 1 && b.rows == 1) return true;
  // b's row 0 starts `r` bytes behind the start of a's row `row`, or where that
  // row would be; all of b's rows lie so to some row of a
  const uintptr_t pitch = a.rows > 1 ? a.pitch : b.pitch;
  const uintptr_t row = d / pitch, r = d % pitch;
  if (d - std::min(row, a.rows - 1) * pitch < a.width) return true;
  return row + 1 < a.rows && pitch - r < b.width;
}

struct Spans {
  Span s[12];
  int n = 0;
  mscl_status_t status = MSCL_SUCCESS;

  // rows x cols elements of `e` bytes, `stride` elements apart.  A null
  // pointer is refused if `needed` and the matrix has elements.
  void add(const char* name, const void* p, size_t rows, size_t cols, size_t stride, size_t e, bool written,
           bool needed, const char* may_be = nullptr) {
    if (status != MSCL_SUCCESS) return;
    char text[160];
    if (rows == 0 || cols == 0) return;
    if (!p) {
      if (!needed) return;
      snprintf(text, sizeof text, "%s is null", name);
      status = bad(text);
      return;
    }
    if (rows > 1 && stride < cols) {
      snprintf(text, sizeof text, "the row stride of %s is shorter than its rows", name);
      status = bad(text);
      return;
    }
    // 2^62 bytes bound every product below
    const size_t most = size_t(1) << 62;
    const size_t reach = rows > 1 ? rows - 1 : 0;
    if (cols > most / e || (reach && stride > (most / e - cols) / reach)) {
      snprintf(text, sizeof text, "the size of %s overflows", name);
      status = bad(text);
      return;
    }
    const uintptr_t a = reinterpret_cast<uintptr_t>(p);
    const uintptr_t bytes = (reach * stride + cols) * e;
    if (a % e) {
      snprintf(text, sizeof text, "%s is not aligned to its elements", name);
      status = record_failure(MSCL_ERR_MISALIGNED, text);
      return;
    }
    if (UINTPTR_MAX - a < bytes) {
      snprintf(text, sizeof text, "%s wraps the address space", name);
      status = bad(text);
      return;
    }
    s[n++] = Span{name, a, bytes, rows, stride * e, cols * e, written, may_be};
  }

  mscl_status_t check() const {
    mscl_status_t st = status;
    for (int i = 1; i < n && st == MSCL_SUCCESS; ++i) st = check_last(i);
    return st;
  }

  // Span `i` against those before it.
  mscl_status_t check_last(int i) const {
    for (int j = 0; j < i; ++j) {
      if (!s[i].written && !s[j].written) continue;
      if (!meet(s[i], s[j])) continue;
      const bool same = s[i].first == s[j].first && s[i].bytes == s[j].bytes;
      const bool allowed = (s[i].may_be && !strcmp(s[i].may_be, s[j].name)) ||
                           (s[j].may_be && !strcmp(s[j].may_be, s[i].name));
      if (same && allowed) continue;
      char text[160];
      snprintf(text, sizeof text, "%s and %s overlap", s[j].name, s[i].name);
      return bad(text);
    }
    return MSCL_SUCCESS;
  }

  // The workspace of a call whose other buffers have passed check().
  mscl_status_t check_workspace(const void* p, size_t have, size_t need) {
    if (need == 0) return MSCL_SUCCESS;
    char text[160];
    if (!p || have < need) {
      snprintf(text, sizeof text, "workspace of %zu bytes needed, %zu given", need, p ? have : size_t(0));
      return bad(text);
    }
    if (reinterpret_cast<uintptr_t>(p) % 16)
      return record_failure(MSCL_ERR_MISALIGNED, "workspace is not 16-byte aligned");
    add("workspace", p, 1, need, 0, 1, true, true);
    return status != MSCL_SUCCESS ? status : check_last(n - 1);
  }
};

// Compute units of the current device, looked up once per device; the
// library holds code for gfx950 alone.
inline mscl_status_t current_device(int* cus) {
  constexpr int kMost = 64;
  static std::atomic<int> known[kMost];
  int dev = 0;
  hipError_t e = hipGetDevice(&dev);
  if (e != hipSuccess) return failed_hip(e, "hipGetDevice");
  if (dev < 0 || dev >= kMost) return bad("device ordinal out of range");
  int n = known[dev].load(std::memory_order_relaxed);
  if (n == 0) {
    hipDeviceProp_t prop;
    e = hipGetDeviceProperties(&prop, dev);
    if (e != hipSuccess) return failed_hip(e, "hipGetDeviceProperties");
    if (strncmp(prop.gcnArchName, "gfx950", 6) != 0)
      return record_failure(MSCL_ERR_UNSUPPORTED, "this library is built for gfx950");
    n = std::max(1, prop.multiProcessorCount);
    known[dev].store(n, std::memory_order_relaxed);
  }
  *cus = n;
  return MSCL_SUCCESS;
}

inline mscl_status_t launched(const char* what) {
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess) return failed_hip(e, what);
  log_text(3, what);
  return MSCL_SUCCESS;
}

inline const char* bytes_at(const void* p) { return static_cast<const char*>(p); }
inline char* bytes_at(void* p) { return static_cast<char*>(p); }
inline uint64_t ceil_div(uint64_t a, uint64_t b) { return a / b + (a % b != 0); }
inline uint64_t round_up(uint64_t a, uint64_t b) { return ceil_div(a, b) * b; }

// Grids are 32-bit; sizes beyond them are refused, not cut.
constexpr uint64_t kMostGroups = 0x7fffffffu;

// Nor has a launch 2^32 threads or more.  The gated block and the 8-bit products
// refuse a plan that needs one where it is made, by the workspace query too (the
// linear layer and layer norm return HIP's error at the launch); `threads` (not
// always whole in 64 bits) are those of its largest launch.
inline mscl_status_t check_threads(double threads) {
  return threads < 4294967296.0 ? MSCL_SUCCESS : bad("the matrices have too many tiles for a launch");
}

// Runs fn(codec) for an element type.
template <class Fn>
mscl_status_t with_codec(int dtype, Fn&& fn) {
  switch (dtype) {
    case MSCL_FLOAT32: return fn(F32{});
    case MSCL_FLOAT16: return fn(F16{});
    default: return fn(BF16{});
  }
}
template <class Fn>
mscl_status_t with_codecs(int dtype, int param_dtype, Fn&& fn) {
  if (dtype == MSCL_FLOAT32) return fn(F32{}, F32{});
  if (dtype == MSCL_FLOAT16) return param_dtype == MSCL_FLOAT32 ? fn(F16{}, F32{}) : fn(F16{}, F16{});
  return param_dtype == MSCL_FLOAT32 ? fn(BF16{}, F32{}) : fn(BF16{}, BF16{});
}

// ------------------------------------------------------------------ column sums

inline JoinArgs join_args(const float* sums, uint64_t stride, uint64_t width, uint32_t groups, void* first, void* second,
                   uint32_t kinds) {
  JoinArgs j;
  j.sums = sums;
  j.out[0] = bytes_at(first);
  j.out[1] = bytes_at(second);
  j.stride = stride;
  j.width = width;
  j.groups = groups;
  j.kinds = kinds;
  return j;
}

// ------------------------------------------------------------------ matrix products

constexpr int kCus = 256;  // of an MI355X: the plans must not depend on a device, as workspaces are sized without one

// How one product m x n x k runs.
struct ProductPlan {
  enum { kTile, kBig, kFew } kind = kTile;
  int tile_m = 64, tile_n = 64;
  bool pack_a = false, pack_b = false;  // operands laid out anew for linear_big
  uint32_t shares = 1;   // of k
  uint32_t blocks_per_share = 1;
  uint64_t partial_stride = 0;
  size_t a_bytes = 0, b_bytes = 0, partial_bytes = 0;
  size_t bytes() const { return a_bytes + b_bytes + partial_bytes; }
};

// Whether linear_big can take an operand as it lies: 16-byte chunks that are
// aligned and whole, and offsets within a tile that fit 31 bits.
inline bool lies_well(const Operand& o) {
  return reinterpret_cast<uintptr_t>(o.base) % 16 == 0 && o.stride % 8 == 0 && o.cols % 8 == 0;
}
inline bool within_reach(uint64_t stride, uint64_t cols, bool along) {
  const uint64_t limit = uint64_t(1) << 30;  // elements of 2 bytes
  return stride < limit / 256 && (!along || cols < limit - 256 * stride);
}

inline uint64_t packed_stride(uint64_t cols) { return round_up(cols, 64); }
inline size_t packed_bytes(const Operand& o, size_t e = 2) {
  return round_up(o.rows * packed_stride(o.cols) * e, 256);
}

// linear_tile's tile for a launch of `large` tiles of 128 x 128.
inline void choose_tile(ProductPlan* p, uint64_t large, int dtype) {
  if (dtype == MSCL_FLOAT32) {
    p->tile_m = 2 * large >= kCus / 2 ? 128 : 64;  // by 64
  } else if (large >= kCus) {
    p->tile_m = p->tile_n = 128;
  }
}

// Shares of k for a product of m x n: no workgroup's run of blocks of 64 k is
// longer than the launch's blocks (of all of its tiles) divided over what the
// device holds at once, two workgroups a compute unit; 4 blocks at least.
// 512 x 512 fp32 with k = 2048: 1 share 53 us, 2 30, 4 20, 8 18; 300 x 700
// with k = 1024: 1 share 29 us, 4 14, 8 15.
inline void choose_shares(ProductPlan* p, uint64_t m, uint64_t n, uint64_t k, uint64_t launch_blocks) {
  const uint64_t steps = ceil_div(k, 64);
  const uint64_t run = std::max<uint64_t>(4, ceil_div(launch_blocks, 2 * kCus));
  const uint64_t shares = std::min<uint64_t>(32, std::max<uint64_t>(1, steps / run));
  p->blocks_per_share = static_cast<uint32_t>(std::max<uint64_t>(1, ceil_div(steps, shares)));
  p->shares = static_cast<uint32_t>(std::max<uint64_t>(1, ceil_div(steps, p->blocks_per_share)));
  p->partial_stride = round_up(n, 8);
  if (p->shares > 1) p->partial_bytes = round_up(p->shares * m * p->partial_stride * 4, 256);
}

// Whether a forward product leaves more than half of the rows or columns of
// its 256 x 256 tiles empty and is better off with other kernels.  What bounds
// it is the pass over the long operand, so 256 tiles, one on each compute unit,
// still do (k 8192, us: 17 x 65536 187 against 218 with few rows, 64 x 65536
// 194 against 200 by small tiles, 65536 x 64 190 against 199), 128 do not (1 x
// 32768 162 against 89, 32 x 49152 192 against 170, 64 x 32768 157 against 125,
// 32768 x 64 161 against 126), and up to 16 rows linear_few is faster still (1
// x 65536 189 against 173).  Input gradients gain nothing (64 x 32768 142
// against 126, 64 x 49152 153 against 163).
inline bool mostly_empty(bool forward, uint64_t m, uint64_t n, uint64_t tiles) {
  return forward && (m <= 16 || (std::min(m, n) <= 128 && tiles < kCus));
}

inline ProductPlan plan_product(const Operand& a, bool a_along, const Operand& b, bool b_along, uint64_t m, uint64_t n,
                         uint64_t k, int dtype) {
  ProductPlan p;
  const uint64_t block = 128 / bytes_of(dtype);
  const uint64_t blocks = ceil_div(k, block);
  const uint64_t big_m = ceil_div(m, 256), big_n = ceil_div(n, 256);
  if (dtype != MSCL_FLOAT32 && big_m * big_n >= kCus / 2 && blocks >= 4 && blocks < (1u << 24) &&
      !mostly_empty(a_along && b_along, m, n, big_m * big_n)) {
    p.pack_a = !lies_well(a);
    p.pack_b = !lies_well(b);
    // An operand is laid out anew only for enough rows (columns) of tiles that
    // use it; small tiles take it as it lies (32768 outputs, k 4096, w at odd
    // addresses, us: 512 rows 212 with the copy, 182 without; 600 267 and 219;
    // 1000 291 and 340; k 8192, 1 row: 398 against 164 with few rows).  Small
    // tiles read both operands of a weight gradient down their columns, whose
    // edges cost them more (16384 x 600, 8192 rows: 262 and 344).
    const uint64_t enough = a_along ? 4 : 3;
    if ((!p.pack_a || big_n >= enough) && (!p.pack_b || big_m >= enough) &&
        within_reach(p.pack_a ? packed_stride(a.cols) : a.stride, a.cols, a_along) &&
        within_reach(p.pack_b ? packed_stride(b.cols) : b.stride, b.cols, b_along)) {
      p.kind = ProductPlan::kBig;
      p.tile_m = p.tile_n = 256;
      if (p.pack_a) p.a_bytes = packed_bytes(a);
      if (p.pack_b) p.b_bytes = packed_bytes(b);
      return p;
    }
    p.pack_a = p.pack_b = false;
  }
  // Up to 32 rows (bf16, us: 32 x 4096 x 8192 19 against 21 by tiles, 64 x
  // 4096 x 8192 27 against 23).  Each wave reads all of x's part of k again,
  // so with more than 8 rows 32 rows of w share it where that still fills the
  // device (16 x 4096 x 8192: 17 against 20; 16 x 2048 x 2048: 8.0 against
  // 6.3), with more than 16 always (32 x 8192 x 4096: 24 against 26).
  if (a_along && b_along && m <= 32 && k > 0) {
    const uint64_t whole = std::max<uint64_t>(1, k / block);
    p.kind = ProductPlan::kFew;
    p.tile_m = 32;
    p.tile_n = m > 16 || (m > 8 && ceil_div(n, 32) >= kCus) ? 32 : 16;
    const uint64_t groups = ceil_div(n, p.tile_n);
    // 8 waves of a workgroup split k already; shares only where the
    // workgroups leave compute units idle, and of 4 steps a wave at least
    const uint64_t shares = groups < kCus ? std::max<uint64_t>(1, std::min(kCus / groups, whole / 32)) : 1;
    p.blocks_per_share = static_cast<uint32_t>(ceil_div(whole, shares));
    p.shares = static_cast<uint32_t>(ceil_div(whole, p.blocks_per_share));
    p.partial_stride = round_up(n, 8);
    if (p.shares > 1) p.partial_bytes = p.shares * m * p.partial_stride * 4;
    return p;
  }
  choose_tile(&p, ceil_div(m, 128) * ceil_div(n, 128), dtype);
  choose_shares(&p, m, n, k, ceil_div(m, p.tile_m) * ceil_div(n, p.tile_n) * ceil_div(k, 64));
  return p;
}

// More dynamic LDS than a kernel gets unasked, asked for once on each device.
template <auto kKernel>
hipError_t allow_lds(int bytes) {
  static std::atomic<uint64_t> done{0};
  int dev = 0;
  hipError_t e = hipGetDevice(&dev);
  if (e != hipSuccess) return e;
  const uint64_t bit = uint64_t(1) << dev;  // current_device() has bounded it
  if (done.load(std::memory_order_acquire) & bit) return hipSuccess;
  e = hipFuncSetAttribute(reinterpret_cast<const void*>(kKernel), hipFuncAttributeMaxDynamicSharedMemorySize, bytes);
  if (e == hipSuccess) done.fetch_or(bit, std::memory_order_release);
  return e;
}

inline TileArgs tile_args(const ProductPlan& p, const Operand& a, const Operand& b, uint64_t k, const Epilogue& e,
                   char* workspace) {
  TileArgs t;
  t.a = a;
  t.b = b;
  t.e = e;
  t.k = k;
  t.e.partial = p.shares > 1 ? reinterpret_cast<float*>(workspace) : nullptr;
  t.e.partial_stride = p.partial_stride;
  t.tiles_m = static_cast<uint32_t>(ceil_div(e.m, p.tile_m));
  t.tiles_n = static_cast<uint32_t>(ceil_div(e.n, p.tile_n));
  t.blocks_per_share = p.blocks_per_share;
  return t;
}

// A matrix as a product takes it.  The stride of a single row means nothing to
// the caller and anything may stand there, but the plans go by it and the
// kernels' loads of rows past the end are placed by it.
inline Operand operand(const void* p, uint64_t stride, uint64_t rows, uint64_t cols) {
  return Operand{bytes_at(p), rows > 1 ? stride : cols, rows, cols};
}

// Row groups of a pass that sums columns: enough workgroups for the device,
// but at least 16 rows each, so that the partial sums stay a small part of
// the traffic, and whole turns of 16 rows (4 waves with 4 rows in flight):
// 17 rows take as long as 32.
inline void plan_groups(uint64_t rows, uint64_t column_blocks, uint32_t* groups, uint32_t* rows_per_group) {
  const uint64_t want = std::max<uint64_t>(1, ceil_div(4 * kCus, std::max<uint64_t>(1, column_blocks)));
  uint64_t per = std::max<uint64_t>(16, ceil_div(rows, want) / 16 * 16);
  per = std::max(per, round_up(ceil_div(rows, 65535), 16));
  *rows_per_group = static_cast<uint32_t>(std::min<uint64_t>(per, 0xffffffffu));
  *groups = static_cast<uint32_t>(std::max<uint64_t>(1, ceil_div(rows, *rows_per_group)));
}

// ------------------------------------------------------------------ defined in operators.hip

// The last sums of a column sum's `kinds`.
mscl_status_t join_columns(int param_dtype, const JoinArgs& j, uint32_t kinds, hipStream_t stream);
// A 16-bit operand laid out anew at `to`.
mscl_status_t pack_operand(int dtype, Operand* o, char* to, hipStream_t stream);
// A product of two operands that both have k down their columns.
mscl_status_t weight_gradient(int dtype, const ProductPlan& p, const Operand& a, const Operand& b, uint64_t k,
                              const Epilogue& e, char* workspace, hipStream_t stream);

}  // namespace launch
}  // namespace mscl
