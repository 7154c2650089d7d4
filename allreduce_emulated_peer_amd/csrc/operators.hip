// Host side of the linear layer and of layer norm (include/mscl.h): argument
// checks, the choice of kernel, tile and split, and the launches of the
// kernels in linear.hpp and norm.hpp.  Every entry point returns a status
// code; nothing here aborts or allocates.

#include <hip/hip_runtime.h>
#include <stdint.h>
#include <stdio.h>
#include <string.h>

#include <algorithm>
#include <atomic>

#include "../../include/mscl.h"
#include "failure.hpp"
#include "linear.hpp"
#include "norm.hpp"

namespace {

using namespace mscl;

// ------------------------------------------------------------------ checks

mscl_status_t bad(const char* msg) { return record_failure(MSCL_ERR_INVALID_ARGUMENT, msg); }

mscl_status_t failed_hip(hipError_t e, const char* what) {
  char text[160];
  snprintf(text, sizeof text, "%s: %s", what, hipGetErrorString(e));
  return record_failure(MSCL_ERR_HIP, text);
}

size_t bytes_of(int dtype) { return dtype == MSCL_FLOAT32 ? 4 : 2; }
bool known_dtype(int d) { return d == MSCL_FLOAT32 || d == MSCL_FLOAT16 || d == MSCL_BFLOAT16; }

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
bool meet(const Span& p, const Span& q) {
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
mscl_status_t current_device(int* cus) {
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

mscl_status_t launched(const char* what) {
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess) return failed_hip(e, what);
  log_text(3, what);
  return MSCL_SUCCESS;
}

const char* bytes_at(const void* p) { return static_cast<const char*>(p); }
char* bytes_at(void* p) { return static_cast<char*>(p); }
uint64_t ceil_div(uint64_t a, uint64_t b) { return a / b + (a % b != 0); }
uint64_t round_up(uint64_t a, uint64_t b) { return ceil_div(a, b) * b; }

// Grids are 32-bit; sizes beyond them are refused, not cut.
constexpr uint64_t kMostGroups = 0x7fffffffu;

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

JoinArgs join_args(const float* sums, uint64_t stride, uint64_t width, uint32_t groups, void* first, void* second,
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

mscl_status_t join_columns(int param_dtype, const JoinArgs& j, uint32_t kinds, hipStream_t stream) {
  const uint64_t blocks = ceil_div(j.width, 32);
  if (blocks > kMostGroups) return bad("the rows are too wide");
  return with_codec(param_dtype, [&](auto p) {
    column_join<decltype(p)><<<dim3(static_cast<uint32_t>(blocks), kinds), 256, 0, stream>>>(j);
    return launched("column_join");
  });
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
bool lies_well(const Operand& o) {
  return reinterpret_cast<uintptr_t>(o.base) % 16 == 0 && o.stride % 8 == 0 && o.cols % 8 == 0;
}
bool within_reach(uint64_t stride, uint64_t cols, bool along) {
  const uint64_t limit = uint64_t(1) << 30;  // elements of 2 bytes
  return stride < limit / 256 && (!along || cols < limit - 256 * stride);
}

uint64_t packed_stride(uint64_t cols) { return round_up(cols, 64); }
size_t packed_bytes(const Operand& o) { return round_up(o.rows * packed_stride(o.cols) * 2, 256); }

// linear_tile's tile for a launch of `large` tiles of 128 x 128.
void choose_tile(ProductPlan* p, uint64_t large, int dtype) {
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
void choose_shares(ProductPlan* p, uint64_t m, uint64_t n, uint64_t k, uint64_t launch_blocks) {
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
bool mostly_empty(bool forward, uint64_t m, uint64_t n, uint64_t tiles) {
  return forward && (m <= 16 || (std::min(m, n) <= 128 && tiles < kCus));
}

ProductPlan plan_product(const Operand& a, bool a_along, const Operand& b, bool b_along, uint64_t m, uint64_t n,
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

template <class C>
mscl_status_t pack(Operand* o, char* to, hipStream_t stream) {
  PackArgs a{o->base, to, o->stride, packed_stride(o->cols), o->rows, o->cols};
  const uint64_t groups = std::min<uint64_t>(ceil_div(ceil_div(o->cols, C::V) * o->rows, 256), 16 * kCus);
  linear_pack<C><<<static_cast<uint32_t>(groups), 256, 0, stream>>>(a);
  *o = Operand{to, a.to_stride, o->rows, round_up(o->cols, C::V)};
  return launched("linear_pack");
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

TileArgs tile_args(const ProductPlan& p, const Operand& a, const Operand& b, uint64_t k, const Epilogue& e,
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

template <class C, bool kAAlong, bool kBAlong, int kBM, int kBN>
mscl_status_t launch_tile(const TileArgs& t, uint32_t shares, hipStream_t stream) {
  constexpr int kLds = tile_lds<C, kAAlong, kBAlong, kBM, kBN>();
  const hipError_t err = allow_lds<&linear_tile<C, kAAlong, kBAlong, kBM, kBN>>(kLds);
  if (err != hipSuccess) return failed_hip(err, "hipFuncSetAttribute");
  linear_tile<C, kAAlong, kBAlong, kBM, kBN><<<t.tiles_m * t.tiles_n * shares, 256, kLds, stream>>>(t);
  return launched("linear_tile");
}

// The joins of up to two products; a product of one share has none.
template <class C>
mscl_status_t launch_join(const Epilogue& a, uint32_t a_shares, const Epilogue& b, uint32_t b_shares, hipStream_t stream) {
  const uint64_t first = a_shares > 1 ? ceil_div(ceil_div(a.n, C::V) * a.m, 256) : 0;
  const uint64_t second = b_shares > 1 ? ceil_div(ceil_div(b.n, C::V) * b.m, 256) : 0;
  if (first + second == 0) return MSCL_SUCCESS;
  if (first + second > kMostGroups) return bad("the matrices have too many tiles");
  linear_join<C><<<static_cast<uint32_t>(first + second), 256, 0, stream>>>(
      a, static_cast<int>(a_shares), b, static_cast<int>(b_shares), static_cast<uint32_t>(first));
  return launched("linear_join");
}

template <class C>
void launch_few(int rows_of_w, const TileArgs& t, dim3 grid, hipStream_t stream) {
  if (t.e.m > 16)
    linear_few<C, 2, 2, 1><<<grid, 512, 0, stream>>>(t);
  else if (rows_of_w == 32)
    linear_few<C, 1, 2, 1><<<grid, 512, 0, stream>>>(t);
  else
    linear_few<C, 1, 1, 2><<<grid, 512, 0, stream>>>(t);
}

template <class C, bool kAAlong, bool kBAlong>
mscl_status_t product(const ProductPlan& p, Operand a, Operand b, uint64_t k, const Epilogue& e0, char* workspace,
                      hipStream_t stream) {
  const uint64_t tm = ceil_div(e0.m, p.tile_m), tn = ceil_div(e0.n, p.tile_n);
  if (tm > kMostGroups / tn / p.shares) return bad("the matrices have too many tiles");
  const uint32_t groups = static_cast<uint32_t>(tm * tn);
  if constexpr (C::kElemBytes == 2) {
    if (p.kind == ProductPlan::kBig) {
      mscl_status_t st = MSCL_SUCCESS;
      if (p.pack_a) st = pack<C>(&a, workspace, stream);
      if (st == MSCL_SUCCESS && p.pack_b) st = pack<C>(&b, workspace + p.a_bytes, stream);
      if (st != MSCL_SUCCESS) return st;
      const hipError_t err = allow_lds<&linear_big<C, kAAlong, kBAlong>>(kBigLds);
      if (err != hipSuccess) return failed_hip(err, "hipFuncSetAttribute");
      BigArgs t{a, b, e0, round_up(k, C::V), static_cast<uint32_t>(tm), static_cast<uint32_t>(tn)};
      linear_big<C, kAAlong, kBAlong><<<groups, 512, kBigLds, stream>>>(t);
      return launched("linear_big");
    }
  }
  const TileArgs t = tile_args(p, a, b, k, e0, workspace);
  mscl_status_t st = MSCL_SUCCESS;
  if (p.kind == ProductPlan::kFew) {
    if constexpr (kAAlong && kBAlong) launch_few<C>(p.tile_n, t, dim3(groups, p.shares), stream);
    st = launched("linear_few");
  } else if (p.tile_m == 128) {
    st = launch_tile<C, kAAlong, kBAlong, 128, C::kElemBytes == 4 ? 64 : 128>(t, p.shares, stream);
  } else {
    st = launch_tile<C, kAAlong, kBAlong, 64, 64>(t, p.shares, stream);
  }
  if (st != MSCL_SUCCESS) return st;
  return launch_join<C>(t.e, p.shares, t.e, 1, stream);
}

// dx and dw in one launch, and db's last sums with them (groups 0: no db).
template <class C, int kBM, int kBN>
mscl_status_t launch_pair(const PairArgs& a, uint32_t db_groups, hipStream_t stream) {
  constexpr int kLds = std::max(tile_lds<C, true, false, kBM, kBN>(), tile_lds<C, false, false, kBM, kBN>());
  const hipError_t err = allow_lds<&linear_pair<C, kBM, kBN>>(kLds);
  if (err != hipSuccess) return failed_hip(err, "hipFuncSetAttribute");
  linear_pair<C, kBM, kBN><<<a.dx_groups + a.dw_groups + db_groups, 256, kLds, stream>>>(a);
  return launched("linear_pair");
}

template <class C>
mscl_status_t pair(const ProductPlan& dx, bool want_dx, const ProductPlan& dw, bool want_dw, PairArgs& a,
                   uint32_t db_groups, hipStream_t stream) {
  const uint64_t dx_tiles = uint64_t(a.dx.tiles_m) * a.dx.tiles_n, dw_tiles = uint64_t(a.dw.tiles_m) * a.dw.tiles_n;
  if (dx_tiles * dx.shares + dw_tiles * dw.shares > kMostGroups / 2) return bad("the matrices have too many tiles");
  a.dx_tiles = static_cast<uint32_t>(dx_tiles);
  a.dw_tiles = static_cast<uint32_t>(dw_tiles);
  a.dx_groups = want_dx ? a.dx_tiles * dx.shares : 0;
  a.dw_groups = want_dw ? a.dw_tiles * dw.shares : 0;
  if (a.dx_groups + a.dw_groups + db_groups == 0) return MSCL_SUCCESS;
  const mscl_status_t st = dx.tile_m == 128 ? launch_pair<C, 128, C::kElemBytes == 4 ? 64 : 128>(a, db_groups, stream)
                                            : launch_pair<C, 64, 64>(a, db_groups, stream);
  if (st != MSCL_SUCCESS) return st;
  return launch_join<C>(a.dx.e, want_dx ? dx.shares : 1, a.dw.e, want_dw ? dw.shares : 1, stream);
}

mscl_status_t check_linear(const mscl_linear_t* c, Spans& s) {
  if (!c) return bad("call is null");
  if (!known_dtype(c->dtype)) return bad("unknown dtype");
  if (c->activation < MSCL_ACT_NONE || c->activation > MSCL_ACT_SILU) return bad("unknown activation");
  const size_t e = bytes_of(c->dtype);
  s.add("x", c->x, c->rows, c->in_features, c->x_stride, e, false, c->out_features != 0);
  s.add("w", c->w, c->out_features, c->in_features, c->w_stride, e, false, c->rows != 0);
  s.add("bias", c->bias, 1, c->out_features, 0, e, false, false);
  s.add("residual", c->residual, c->rows, c->out_features, c->residual_stride, e, false, false);
  s.add("y", c->y, c->rows, c->out_features, c->y_stride, e, true, true, "residual");
  s.add("preact", c->preact, c->rows, c->out_features, c->preact_stride, e, true, false);
  return s.check();
}

// A matrix as a product takes it.  The stride of a single row means nothing to
// the caller and anything may stand there, but the plans go by it and the
// kernels' loads of rows past the end are placed by it.
Operand operand(const void* p, uint64_t stride, uint64_t rows, uint64_t cols) {
  return Operand{bytes_at(p), rows > 1 ? stride : cols, rows, cols};
}

Operand x_of(const mscl_linear_t& c) { return operand(c.x, c.x_stride, c.rows, c.in_features); }
Operand w_of(const mscl_linear_t& c) { return operand(c.w, c.w_stride, c.out_features, c.in_features); }

ProductPlan plan_linear(const mscl_linear_t& c) {
  return plan_product(x_of(c), true, w_of(c), true, c.rows, c.out_features, c.in_features, c.dtype);
}

// Parts of a backward call's workspace, each from a 256-byte boundary.
struct BackwardPlan {
  ProductPlan dx, dw;
  bool slope = false;  // dz is computed into the workspace
  bool pair = false;   // dx and dw in one launch
  Operand dz, x, w;    // dz without its address where it is computed
  uint32_t groups = 0, rows_per_group = 0;  // of the bias gradient's partial sums
  size_t dz_at = 0, sums_at = 0, partial_at = 0, bytes = 0;
};

// Row groups of a pass that sums columns: enough workgroups for the device,
// but at least 16 rows each, so that the partial sums stay a small part of
// the traffic, and whole turns of 16 rows (4 waves with 4 rows in flight):
// 17 rows take as long as 32.
void plan_groups(uint64_t rows, uint64_t column_blocks, uint32_t* groups, uint32_t* rows_per_group) {
  const uint64_t want = std::max<uint64_t>(1, ceil_div(4 * kCus, std::max<uint64_t>(1, column_blocks)));
  uint64_t per = std::max<uint64_t>(16, ceil_div(rows, want) / 16 * 16);
  per = std::max(per, round_up(ceil_div(rows, 65535), 16));
  *rows_per_group = static_cast<uint32_t>(std::min<uint64_t>(per, 0xffffffffu));
  *groups = static_cast<uint32_t>(std::max<uint64_t>(1, ceil_div(rows, *rows_per_group)));
}

BackwardPlan plan_linear_backward(const mscl_linear_backward_t& c) {
  BackwardPlan p;
  const size_t e = bytes_of(c.dtype);
  p.slope = c.activation != MSCL_ACT_NONE && (c.dx || c.dw);
  size_t at = 0;
  p.dz = operand(c.dy, c.dy_stride, c.rows, c.out_features);
  p.x = operand(c.x, c.x_stride, c.rows, c.in_features);
  p.w = operand(c.w, c.w_stride, c.out_features, c.in_features);
  if (p.slope) {
    p.dz = Operand{nullptr, packed_stride(c.out_features), c.rows, round_up(c.out_features, 16 / e)};
    p.dz_at = at;
    at = round_up(at + c.rows * p.dz.stride * e, 256);
  }
  if (c.dbias) {
    plan_groups(c.rows, ceil_div(c.out_features, 64 * (16 / e)), &p.groups, &p.rows_per_group);
    p.sums_at = at;
    at = round_up(at + size_t(p.groups) * c.out_features * 4, 256);
  }
  p.partial_at = at;
  size_t partial = 0;
  // The plans go by sizes and layouts, not by which gradients are wanted: a
  // gradient has the same bits alone.
  if (!c.dx) p.w = Operand{nullptr, c.in_features, c.out_features, c.in_features};
  if (!c.dw) p.x = Operand{nullptr, c.in_features, c.rows, c.in_features};
  if (c.rows && c.out_features && c.in_features) {
    p.dx = plan_product(p.dz, true, p.w, false, c.rows, c.in_features, c.out_features, c.dtype);
    p.dw = plan_product(p.dz, false, p.x, false, c.out_features, c.in_features, c.rows, c.dtype);
    p.pair = p.dx.kind == ProductPlan::kTile && p.dw.kind == ProductPlan::kTile;
  }
  if (p.pair) {
    const uint64_t k = ceil_div(c.in_features, 128);
    p.dx = p.dw = ProductPlan();
    choose_tile(&p.dx, (ceil_div(c.rows, 128) + ceil_div(c.out_features, 128)) * k, c.dtype);
    choose_tile(&p.dw, (ceil_div(c.rows, 128) + ceil_div(c.out_features, 128)) * k, c.dtype);
    const uint64_t launch = (ceil_div(c.rows, p.dx.tile_m) * ceil_div(c.out_features, 64) +
                             ceil_div(c.out_features, p.dw.tile_m) * ceil_div(c.rows, 64)) *
                            ceil_div(c.in_features, p.dx.tile_n);
    choose_shares(&p.dx, c.rows, c.in_features, c.out_features, launch);
    choose_shares(&p.dw, c.out_features, c.in_features, c.rows, launch);
    partial = (c.dx ? p.dx.partial_bytes : 0) + (c.dw ? p.dw.partial_bytes : 0);
  } else {
    if (c.dx) partial = std::max(partial, p.dx.bytes());
    if (c.dw) partial = std::max(partial, p.dw.bytes());
  }
  p.bytes = at + partial;
  return p;
}

mscl_status_t check_linear_backward(const mscl_linear_backward_t* c, Spans& s) {
  if (!c) return bad("call is null");
  if (!known_dtype(c->dtype)) return bad("unknown dtype");
  if (c->activation < MSCL_ACT_NONE || c->activation > MSCL_ACT_SILU) return bad("unknown activation");
  const size_t e = bytes_of(c->dtype);
  const bool some = c->dx || c->dw || c->dbias;
  s.add("dy", c->dy, c->rows, c->out_features, c->dy_stride, e, false, some);
  if (c->dw) s.add("x", c->x, c->rows, c->in_features, c->x_stride, e, false, c->out_features != 0);
  if (c->dx) s.add("w", c->w, c->out_features, c->in_features, c->w_stride, e, false, c->rows != 0);
  if (c->activation != MSCL_ACT_NONE)
    s.add("preact", c->preact, c->rows, c->out_features, c->preact_stride, e, false, some);
  s.add("dx", c->dx, c->rows, c->in_features, c->dx_stride, e, true, false);
  s.add("dw", c->dw, c->out_features, c->in_features, c->dw_stride, e, true, false);
  s.add("dbias", c->dbias, 1, c->out_features, 0, e, true, false);
  return s.check();
}

// ------------------------------------------------------------------ layer norm

mscl_status_t check_params(int dtype, int param_dtype, size_t width) {
  if (!known_dtype(dtype) || !known_dtype(param_dtype)) return bad("unknown dtype");
  if (param_dtype != dtype && param_dtype != MSCL_FLOAT32) return bad("param_dtype must be dtype or MSCL_FLOAT32");
  if (width == 0) return bad("width must be at least 1");
  return MSCL_SUCCESS;
}

mscl_status_t check_layer_norm(const mscl_layer_norm_t* c, Spans& s) {
  if (!c) return bad("call is null");
  mscl_status_t st = check_params(c->dtype, c->param_dtype, c->width);
  if (st != MSCL_SUCCESS) return st;
  if (!(c->eps >= 0.0)) return bad("eps must be at least 0");
  const size_t e = bytes_of(c->dtype), pe = bytes_of(c->param_dtype);
  s.add("x", c->x, c->rows, c->width, c->x_stride, e, false, true);
  s.add("weight", c->weight, 1, c->width, 0, pe, false, false);
  s.add("bias", c->bias, 1, c->width, 0, pe, false, false);
  s.add("y", c->y, c->rows, c->width, c->y_stride, e, true, true, "x");
  s.add("mean", c->mean, 1, c->rows, 0, 4, true, false);
  s.add("rstd", c->rstd, 1, c->rows, 0, 4, true, false);
  return s.check();
}

mscl_status_t check_layer_norm_backward(const mscl_layer_norm_backward_t* c, Spans& s) {
  if (!c) return bad("call is null");
  mscl_status_t st = check_params(c->dtype, c->param_dtype, c->width);
  if (st != MSCL_SUCCESS) return st;
  const size_t e = bytes_of(c->dtype), pe = bytes_of(c->param_dtype);
  const bool some = c->dx || c->dweight || c->dbias;
  s.add("dy", c->dy, c->rows, c->width, c->dy_stride, e, false, some);
  s.add("x", c->x, c->rows, c->width, c->x_stride, e, false, some);
  s.add("mean", c->mean, 1, c->rows, 0, 4, false, some);
  s.add("rstd", c->rstd, 1, c->rows, 0, 4, false, some);
  s.add("weight", c->weight, 1, c->width, 0, pe, false, false);
  s.add("dx", c->dx, c->rows, c->width, c->dx_stride, e, true, false, "dy");
  s.add("dweight", c->dweight, 1, c->width, 0, pe, true, false);
  s.add("dbias", c->dbias, 1, c->width, 0, pe, true, false);
  return s.check();
}

struct NormBackPlan {
  bool sums = false;
  bool fused = false;  // norm_back_fused, with `groups` workgroups
  uint32_t groups = 0, rows_per_group = 0;
  uint64_t blocks = 0;  // of columns, in norm_back_tiles
  uint64_t sums_stride = 0;
  size_t along_at = 0, bytes = 0;
};

// Threads that hold a row of `vecs` vectors in norm_back_fused.
int fused_threads(uint64_t vecs) { return vecs <= 64 ? 64 : vecs <= 128 ? 128 : vecs <= 256 ? 256 : 512; }

NormBackPlan plan_layer_norm_backward(const mscl_layer_norm_backward_t& c) {
  NormBackPlan p;
  p.sums = c.dweight || c.dbias;
  if (!p.sums) return p;
  p.sums_stride = round_up(c.width, 8);
  const uint64_t e = bytes_of(c.dtype), vecs = ceil_div(c.width, 16 / e);
  // Partial sums written and read (16 bytes a column and workgroup) against a
  // second read of x and dy (2 e bytes a row and column).
  if (c.dx && vecs <= (e == 4 ? 2048 : 1024) && c.rows * 2 * e >= 16 * kCus) {
    p.fused = true;
    const uint64_t at_once = vecs > 1024 ? 1 : 2 * (512 / fused_threads(vecs));
    p.groups = static_cast<uint32_t>(std::min<uint64_t>(kCus, ceil_div(c.rows, at_once)));
  } else {
    p.blocks = ceil_div(c.width, 64 * (16 / e));
    plan_groups(c.rows, p.blocks, &p.groups, &p.rows_per_group);
  }
  p.along_at = round_up(size_t(p.groups) * 2 * p.sums_stride * 4, 256);
  p.bytes = p.along_at + (c.dx ? c.rows * p.blocks * 8 : 0);
  return p;
}

template <class C, class P>
void launch_norm_back_fused(const NormBackArgs& a, uint32_t groups, hipStream_t s) {
  const uint64_t vecs = ceil_div(a.width, C::V);
  if (C::V == 4 && vecs > 1024)
    norm_back_fused<C, P, 512, C::V == 4 ? 4 : 2, C::V == 4 ? 1 : 2><<<groups, 512, 0, s>>>(a);
  else if (vecs > 512)
    norm_back_fused<C, P, 512, 2, 2><<<groups, 512, 0, s>>>(a);
  else switch (fused_threads(vecs)) {
    case 64: norm_back_fused<C, P, 64, 1, 2><<<groups, 512, 0, s>>>(a); break;
    case 128: norm_back_fused<C, P, 128, 1, 2><<<groups, 512, 0, s>>>(a); break;
    case 256: norm_back_fused<C, P, 256, 1, 2><<<groups, 512, 0, s>>>(a); break;
    default: norm_back_fused<C, P, 512, 1, 2><<<groups, 512, 0, s>>>(a);
  }
}

template <class C, class P, int kThreads, int kVecs>
void launch_norm_rows(const NormArgs& a, hipStream_t s) {
  const uint64_t groups = kThreads < 256 ? ceil_div(a.rows, 256 / kThreads) : a.rows;
  norm_rows<C, P, kThreads, kVecs><<<static_cast<uint32_t>(groups), kThreads < 256 ? 256 : kThreads, 0, s>>>(a);
}

// A row's 16-byte vectors -> threads and vectors per thread that hold it.  Few
// rows want the shortest way through a row, one vector a thread (32 x 8192
// bf16: 1024 threads 3.9 us, 256 threads 5.1); many rows want few threads
// with several vectors in flight each (8192 x 8192 bf16: 1024 threads 68 us,
// 512 53, 256 48; 8192 x 2048: 256 threads 17.0 us, 64 threads 15.4).
template <class C, class P>
void launch_norm(const NormArgs& a, hipStream_t s) {
  const bool aligned = reinterpret_cast<uintptr_t>(a.x) % 16 == 0 && (a.rows == 1 || a.x_stride % C::V == 0);
  const uint64_t vecs = ceil_div(a.width, C::V) + (aligned ? 0 : 1);
  if (vecs <= 64) return launch_norm_rows<C, P, 64, 1>(a, s);
  if (a.rows <= 2 * kCus) {
    if (vecs <= 256) return launch_norm_rows<C, P, 256, 1>(a, s);
    if (vecs <= 512) return launch_norm_rows<C, P, 512, 1>(a, s);
    if (vecs <= 1024) return launch_norm_rows<C, P, 1024, 1>(a, s);
  }
  if (vecs <= 128) return launch_norm_rows<C, P, 64, 2>(a, s);
  if (vecs <= 256) return launch_norm_rows<C, P, 64, 4>(a, s);
  if (vecs <= 512) return launch_norm_rows<C, P, 256, 2>(a, s);
  if (vecs <= 768) return launch_norm_rows<C, P, 256, 3>(a, s);
  if (vecs <= 1024) return launch_norm_rows<C, P, 256, 4>(a, s);
  if (vecs <= 2048) return launch_norm_rows<C, P, 512, 4>(a, s);
  if (vecs <= 4096) return launch_norm_rows<C, P, 1024, 4>(a, s);
  norm_rows_wide<C, P><<<static_cast<uint32_t>(a.rows), 1024, 0, s>>>(a);
}

template <class C, class P>
void launch_norm_back(const NormBackArgs& a, hipStream_t s) {
  const uint64_t vecs = ceil_div(a.width, C::V);
  const uint32_t rows = static_cast<uint32_t>(a.rows), quads = static_cast<uint32_t>(ceil_div(a.rows, 4));
  if (vecs <= 64)
    norm_back_rows<C, P, 64, 1><<<quads, 256, 0, s>>>(a);
  else if (vecs <= 128)
    norm_back_rows<C, P, 64, 2><<<quads, 256, 0, s>>>(a);
  else if (vecs <= 256)
    norm_back_rows<C, P, 256, 1><<<rows, 256, 0, s>>>(a);
  else if (vecs <= 512)
    norm_back_rows<C, P, 256, 2><<<rows, 256, 0, s>>>(a);
  else if (vecs <= 1024)
    norm_back_rows<C, P, 256, 4><<<rows, 256, 0, s>>>(a);
  else if (vecs <= 2048)
    norm_back_rows<C, P, 1024, 2><<<rows, 1024, 0, s>>>(a);
  else if (vecs <= 4096 && C::V == 4)
    norm_back_rows<C, P, 1024, C::V == 4 ? 4 : 2><<<rows, 1024, 0, s>>>(a);
  else
    norm_back_rows_wide<C, P><<<rows, 1024, 0, s>>>(a);
}

}  // namespace

extern "C" {

mscl_status_t mscl_linear_workspace(const mscl_linear_t* call, size_t* bytes) {
  if (!bytes) return bad("bytes is null");
  Spans spans;
  const mscl_status_t st = check_linear(call, spans);
  if (st != MSCL_SUCCESS) return st;
  *bytes = call->rows && call->out_features ? plan_linear(*call).bytes() : 0;
  return MSCL_SUCCESS;
}

mscl_status_t mscl_linear(const mscl_linear_t* call, void* workspace, size_t workspace_bytes, void* stream) {
  Spans spans;
  mscl_status_t st = check_linear(call, spans);
  if (st != MSCL_SUCCESS) return st;
  const mscl_linear_t& c = *call;
  if (c.rows == 0 || c.out_features == 0) return MSCL_SUCCESS;
  const ProductPlan p = plan_linear(c);
  if ((st = spans.check_workspace(workspace, workspace_bytes, p.bytes())) != MSCL_SUCCESS) return st;
  int cus = 0;
  if ((st = current_device(&cus)) != MSCL_SUCCESS) return st;
  Epilogue e;
  memset(&e, 0, sizeof e);
  e.bias = bytes_at(c.bias);
  e.residual = bytes_at(c.residual);
  e.residual_stride = c.residual_stride;
  e.y = bytes_at(c.y);
  e.y_stride = c.y_stride;
  e.z = bytes_at(c.preact);
  e.z_stride = c.preact_stride;
  e.m = c.rows;
  e.n = c.out_features;
  e.act = c.activation;
  return with_codec(c.dtype, [&](auto t) {
    return product<decltype(t), true, true>(p, x_of(c), w_of(c), c.in_features, e, bytes_at(workspace),
                                            static_cast<hipStream_t>(stream));
  });
}

mscl_status_t mscl_linear_backward_workspace(const mscl_linear_backward_t* call, size_t* bytes) {
  if (!bytes) return bad("bytes is null");
  Spans spans;
  const mscl_status_t st = check_linear_backward(call, spans);
  if (st != MSCL_SUCCESS) return st;
  *bytes = plan_linear_backward(*call).bytes;
  return MSCL_SUCCESS;
}

mscl_status_t mscl_linear_backward(const mscl_linear_backward_t* call, void* workspace, size_t workspace_bytes,
                                   void* stream) {
  Spans spans;
  mscl_status_t st = check_linear_backward(call, spans);
  if (st != MSCL_SUCCESS) return st;
  const mscl_linear_backward_t& c = *call;
  const BackwardPlan p = plan_linear_backward(c);
  if ((st = spans.check_workspace(workspace, workspace_bytes, p.bytes)) != MSCL_SUCCESS) return st;
  const bool dx = c.dx && c.rows && c.in_features;
  const bool dw = c.dw && c.out_features && c.in_features;
  const bool db = c.dbias && c.out_features;
  if (!dx && !dw && !db) return MSCL_SUCCESS;
  int cus = 0;
  if ((st = current_device(&cus)) != MSCL_SUCCESS) return st;
  const hipStream_t s = static_cast<hipStream_t>(stream);
  char* ws = bytes_at(workspace);
  Operand dz = p.dz;
  if (p.slope) dz.base = ws + p.dz_at;
  JoinArgs db_join;
  memset(&db_join, 0, sizeof db_join);
  if (db || (p.slope && (dx || dw))) {
    SlopeArgs a;
    memset(&a, 0, sizeof a);
    a.dy = bytes_at(c.dy);
    a.dy_stride = c.dy_stride;
    a.z = c.activation != MSCL_ACT_NONE ? bytes_at(c.preact) : nullptr;
    a.z_stride = c.preact_stride;
    a.act = c.activation;
    a.rows = c.rows;
    a.cols = c.out_features;
    if (p.slope) {
      a.dz = ws + p.dz_at;
      a.dz_stride = p.dz.stride;
    }
    uint32_t groups = p.groups;
    a.rows_per_group = p.rows_per_group;
    if (db) {
      a.sums = reinterpret_cast<float*>(ws + p.sums_at);
      a.sums_stride = c.out_features;
    } else {
      plan_groups(c.rows, ceil_div(c.out_features, 64 * (16 / bytes_of(c.dtype))), &groups, &a.rows_per_group);
    }
    const uint64_t blocks = ceil_div(c.out_features, 64 * (16 / bytes_of(c.dtype)));
    if (blocks > kMostGroups) return bad("the matrices have too many tiles");
    if (blocks) {
      st = with_codec(c.dtype, [&](auto t) {
        linear_slope<decltype(t)><<<dim3(static_cast<uint32_t>(blocks), groups), 256, 0, s>>>(a);
        return launched("linear_slope");
      });
      if (st != MSCL_SUCCESS) return st;
    }
    db_join = join_args(a.sums, c.out_features, c.out_features, groups, c.dbias, nullptr, 1);
  }
  Epilogue ex, ew;
  memset(&ex, 0, sizeof ex);
  ex.y = bytes_at(c.dx);
  ex.y_stride = c.dx_stride;
  ex.m = c.rows;
  ex.n = c.in_features;
  memset(&ew, 0, sizeof ew);
  ew.y = bytes_at(c.dw);
  ew.y_stride = c.dw_stride;
  ew.m = c.out_features;
  ew.n = c.in_features;
  char* partial = ws + p.partial_at;
  if (p.pair) {
    return with_codec(c.dtype, [&](auto t) {
      PairArgs a;
      a.dx = tile_args(p.dx, dz, p.w, c.out_features, ex, partial);
      a.dw = tile_args(p.dw, dz, p.x, c.rows, ew, partial + (dx ? p.dx.partial_bytes : 0));
      a.db = db_join;
      const uint64_t db_groups = db ? ceil_div(c.out_features, 32) : 0;
      if (db_groups > kMostGroups / 2) return bad("the matrices have too many tiles");
      return pair<decltype(t)>(p.dx, dx, p.dw, dw, a, static_cast<uint32_t>(db_groups), s);
    });
  }
  if (db && (st = join_columns(c.dtype, db_join, 1, s)) != MSCL_SUCCESS) return st;
  if (dx) {
    st = with_codec(c.dtype, [&](auto t) {
      return product<decltype(t), true, false>(p.dx, dz, p.w, c.out_features, ex, partial, s);
    });
    if (st != MSCL_SUCCESS) return st;
  }
  if (dw) {
    st = with_codec(c.dtype, [&](auto t) {
      return product<decltype(t), false, false>(p.dw, dz, p.x, c.rows, ew, partial, s);
    });
  }
  return st;
}

mscl_status_t mscl_layer_norm(const mscl_layer_norm_t* call, void* stream) {
  Spans spans;
  mscl_status_t st = check_layer_norm(call, spans);
  if (st != MSCL_SUCCESS) return st;
  const mscl_layer_norm_t& c = *call;
  if (c.rows == 0) return MSCL_SUCCESS;
  if (c.rows > kMostGroups) return bad("too many rows");
  int cus = 0;
  if ((st = current_device(&cus)) != MSCL_SUCCESS) return st;
  NormArgs a;
  a.x = bytes_at(c.x);
  a.x_stride = c.x_stride;
  a.w = bytes_at(c.weight);
  a.b = bytes_at(c.bias);
  a.y = bytes_at(c.y);
  a.y_stride = c.y_stride;
  a.mean = c.mean;
  a.rstd = c.rstd;
  a.rows = c.rows;
  a.width = c.width;
  a.eps = static_cast<float>(c.eps);
  return with_codecs(c.dtype, c.param_dtype, [&](auto t, auto p) {
    launch_norm<decltype(t), decltype(p)>(a, static_cast<hipStream_t>(stream));
    return launched("norm_rows");
  });
}

mscl_status_t mscl_layer_norm_backward_workspace(const mscl_layer_norm_backward_t* call, size_t* bytes) {
  if (!bytes) return bad("bytes is null");
  Spans spans;
  const mscl_status_t st = check_layer_norm_backward(call, spans);
  if (st != MSCL_SUCCESS) return st;
  *bytes = plan_layer_norm_backward(*call).bytes;
  return MSCL_SUCCESS;
}

mscl_status_t mscl_layer_norm_backward(const mscl_layer_norm_backward_t* call, void* workspace,
                                       size_t workspace_bytes, void* stream) {
  Spans spans;
  mscl_status_t st = check_layer_norm_backward(call, spans);
  if (st != MSCL_SUCCESS) return st;
  const mscl_layer_norm_backward_t& c = *call;
  const NormBackPlan p = plan_layer_norm_backward(c);
  if ((st = spans.check_workspace(workspace, workspace_bytes, p.bytes)) != MSCL_SUCCESS) return st;
  if (c.rows > kMostGroups) return bad("too many rows");
  if (!p.sums && (!c.dx || c.rows == 0)) return MSCL_SUCCESS;
  int cus = 0;
  if ((st = current_device(&cus)) != MSCL_SUCCESS) return st;
  const hipStream_t s = static_cast<hipStream_t>(stream);
  NormBackArgs a;
  a.dy = bytes_at(c.dy);
  a.dy_stride = c.dy_stride;
  a.x = bytes_at(c.x);
  a.x_stride = c.x_stride;
  a.mean = c.mean;
  a.rstd = c.rstd;
  a.w = bytes_at(c.weight);
  a.dx = bytes_at(c.dx);
  a.dx_stride = c.dx_stride;
  a.sums = reinterpret_cast<float*>(workspace);
  a.along = nullptr;
  a.sums_stride = p.sums_stride;
  a.rows = c.rows;
  a.width = c.width;
  a.rows_per_group = p.rows_per_group;
  if (p.fused) {
    st = with_codecs(c.dtype, c.param_dtype, [&](auto t, auto q) {
      launch_norm_back_fused<decltype(t), decltype(q)>(a, p.groups, s);
      return launched("norm_back_fused");
    });
    if (st != MSCL_SUCCESS) return st;
    const JoinArgs j = join_args(a.sums, a.sums_stride, c.width, p.groups, c.dweight, c.dbias, 2);
    return join_columns(c.param_dtype, j, 2, s);
  }
  if (p.sums) {
    a.along = reinterpret_cast<float*>(bytes_at(workspace) + p.along_at);
    const uint64_t tiles = c.dx ? p.blocks * ceil_div(c.rows, p.rows_per_group) : 0, joins = ceil_div(c.width, 32);
    if (joins > kMostGroups / 4 || tiles > kMostGroups / 2) return bad("the matrices have too many tiles");
    return with_codecs(c.dtype, c.param_dtype, [&](auto t, auto q) {
      using T = decltype(t);
      using Q = decltype(q);
      norm_back_tiles<T, Q><<<dim3(static_cast<uint32_t>(p.blocks), p.groups), 256, 0, s>>>(a);
      const mscl_status_t done = launched("norm_back_tiles");
      if (done != MSCL_SUCCESS) return done;
      const JoinArgs j = join_args(a.sums, a.sums_stride, c.width, p.groups, c.dweight, c.dbias, 2);
      norm_back_apply<T, Q><<<static_cast<uint32_t>(tiles + 2 * joins), 256, 0, s>>>(
          a, j, static_cast<uint32_t>(p.blocks), static_cast<uint32_t>(tiles), static_cast<uint32_t>(joins));
      return launched("norm_back_apply");
    });
  }
  if (!c.dx || c.rows == 0) return MSCL_SUCCESS;
  return with_codecs(c.dtype, c.param_dtype, [&](auto t, auto q) {
    launch_norm_back<decltype(t), decltype(q)>(a, s);
    return launched("norm_back_rows");
  });
}

}  // extern "C"
