// What the block-scaled products (fp8.hip, mx.hip) share: operands' rows and tiles, copies to LDS,
// conversions and stores of outputs.
#pragma once

#include <algorithm>

#include "common.h"

namespace gptq {
namespace {

typedef int i32x8 __attribute__((ext_vector_type(8)));
typedef int i32x4 __attribute__((ext_vector_type(4)));
typedef unsigned u32x4 __attribute__((ext_vector_type(4)));

template <typename T>
__device__ __forceinline__ T from_f32(float v);
template <>
__device__ __forceinline__ float from_f32<float>(float v) { return v; }
template <>
__device__ __forceinline__ BF16 from_f32<BF16>(float v) {
  return BF16{__builtin_bit_cast(uint16_t, static_cast<__bf16>(v))};
}
template <>
__device__ __forceinline__ F16 from_f32<F16>(float v) {
  return F16{__builtin_bit_cast(uint16_t, static_cast<_Float16>(v))};
}

template <typename T, int V>
struct alignas(sizeof(T) * V) Vec {
  T v[V];
};

// N consecutive elements as fp32, in 16-byte loads, which the chip takes at any address.
template <typename T, int N>
__device__ __forceinline__ void load_row(const T* p, float* x) {
  T w[N];
  __builtin_memcpy(w, p, sizeof(w));
#pragma unroll
  for (int i = 0; i < N; ++i) x[i] = load_as_f32(&w[i]);
}

// The larger of |x| as bits: orders all finite values, infinity and NaN above them.
template <int N>
__device__ __forceinline__ uint32_t top_bits(const float* x) {
  uint32_t t = 0;
#pragma unroll
  for (int i = 0; i < N; ++i) t = max(t, __float_as_uint(x[i]) & 0x7FFFFFFFu);
  return t;
}

// Which tile a workgroup takes.  Workgroups go to the 8 XCDs in turn, 32 CUs each; tiles are
// numbered in bands of 4 tile rows, column by column, and an XCD takes runs of 32 consecutive ones:
// the 32 tiles it works on at once are then 4 x 8 and read 12 operand panels through its L2 instead
// of the 18 of a row-by-row grid.  What is left of whole rounds of 256 is shared out evenly (in
// runs of 32 some XCDs had 32 tiles more than others: 5000 x 5000 x 4096 116 us, 108 so; runs of 8
// throughout: 111 there, but 8192 x 4096 x 14336 413 instead of 405).
struct TileOrder {
  int tiles_n;
  int64_t tiles_m;
};
inline int64_t order_grid(const TileOrder& o) { return (o.tiles_m * o.tiles_n + 7) / 8 * 8; }
// (tile row, tile column) of workgroup b; false for none
__device__ __forceinline__ bool ordered_tile(const TileOrder& o, uint32_t b, int64_t* mt, int* nt) {
  const uint32_t total = static_cast<uint32_t>(o.tiles_m) * static_cast<uint32_t>(o.tiles_n);   // at most 2^22
  const uint32_t whole = total & ~255u, run = b < whole ? 32 : (total - whole + 7) / 8;
  const uint32_t first = b < whole ? b & ~255u : whole, slot = b - first;
  const uint32_t p = first + slot % 8 * run + slot / 8;
  if (slot / 8 >= run || p >= total) return false;
  const uint32_t per = 4u * static_cast<uint32_t>(o.tiles_n);
  const uint32_t band = p / per, r = p % per;
  const uint32_t rows = min(4u, static_cast<uint32_t>(o.tiles_m) - 4 * band);
  *mt = 4 * band + r % rows;
  *nt = static_cast<int>(r / rows);
  return true;
}

struct MmArgs {
  int64_t m;             // output rows
  int n, k, kb, nb;      // outputs, inputs and their blocks
  const uint8_t* X;      // e4m3 rows
  int64_t ldx, x_rows;
  const void* xs;        // their scales
  int64_t xsr, xsb;
  const uint8_t* W;
  const void* ws;
  void* Y;
  int64_t ldy;
  int y_dtype;
  bool e8;               // scales are E8M0
  const int64_t* off;    // grouped: the experts' ranges
  const int32_t* rows;   // grouped: rows of X, or null
  int experts;
  int tiles_n;
  TileOrder order;
};

__device__ const u32x4 zero16 = {0, 0, 0, 0};

// One tile of output rows: rows p0 .. p0 + count - 1 of expert e (count <= 0: no tile).
struct Tile {
  int e;
  int64_t p0;
  int count;
};
// A value that is the same in every lane, in a scalar register.
__device__ __forceinline__ int uniform(int v) { return __builtin_amdgcn_readfirstlane(v); }
__device__ __forceinline__ int64_t uniform(int64_t v) {
  const uint32_t lo = uniform(static_cast<int>(v)), hi = uniform(static_cast<int>(v >> 32));
  return static_cast<int64_t>((static_cast<uint64_t>(hi) << 32) | lo);
}

// The mt-th tile of TM rows: of the one problem, or counting tiles expert by expert.  Every wave
// finds it for itself, 64 experts at a time.
__device__ __forceinline__ Tile find_tile(const MmArgs& a, int64_t mt, int TM) {
  if (a.off == nullptr) {
    const int64_t p0 = mt * TM;
    return {0, p0, static_cast<int>(min(static_cast<int64_t>(TM), a.m - p0))};
  }
  const int lane = threadIdx.x & 63;
  int before = 0;   // tiles of earlier experts; the launch bounds their number
  for (int e0 = 0; e0 < a.experts; e0 += 64) {
    int64_t lo = 0, n = 0;
    if (e0 + lane < a.experts) {
      lo = min(max(a.off[e0 + lane], static_cast<int64_t>(0)), a.m);
      n = min(max(a.off[e0 + lane + 1], lo), a.m) - lo;
    }
    const int own = static_cast<int>((n + TM - 1) / TM);
    int inc = own;
    for (int d = 1; d < 64; d <<= 1) {
      const int o = __shfl_up(inc, d);
      if (lane >= d) inc += o;
    }
    const uint64_t past = __ballot(before + inc > mt);
    if (past) {
      const int l = __builtin_ctzll(past);
      const int64_t r0 = (mt - (before + __shfl(inc - own, l))) * TM;
      const int64_t lo_l = __shfl(lo, l), n_l = __shfl(n, l);
      return {uniform(e0 + l), uniform(lo_l + r0),
              uniform(static_cast<int>(min(static_cast<int64_t>(TM), n_l - r0)))};
    }
    before += __shfl(inc, 63);
  }
  return {0, 0, 0};
}
template <int TM>
__device__ __forceinline__ Tile find_tile(const MmArgs& a, int64_t mt) { return find_tile(a, mt, TM); }

// The row of X behind output row p, -1 for none.
__device__ __forceinline__ int64_t source_row(const MmArgs& a, int64_t p) {
  if (a.rows == nullptr) return p < a.x_rows ? p : -1;
  const int64_t r = a.rows[p];
  return r >= 0 && r < a.x_rows ? r : -1;
}

// An E8M0 code as fp32 (2^-127 is subnormal there).
__device__ __forceinline__ float e8m0_f32(int code) {
  return code == 255 ? __uint_as_float(0x7FC00000u) : code == 0 ? __uint_as_float(0x00400000u)
                                                                 : __uint_as_float(static_cast<uint32_t>(code) << 23);
}

// Rows of Y may start at any element: the chip takes 16-byte stores at any address (2443 x 6075 x
// 5664, whose rows are of odd length: 98 us, 119 by single values).
template <typename T>
__device__ __forceinline__ void store4(T* p, const float* v, int n) {
  if (n >= 4) {
    Vec<T, 4> o;
#pragma unroll
    for (int i = 0; i < 4; ++i) o.v[i] = from_f32<T>(v[i]);
    __builtin_memcpy(p, &o, sizeof(o));
  } else {
    for (int i = 0; i < n; ++i) p[i] = from_f32<T>(v[i]);
  }
}
// four values as bf16 or fp16
template <bool kBf16>
__device__ __forceinline__ uint2 pack16(f32x4 v) {
  uint16_t u[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) u[i] = kBf16 ? from_f32<BF16>(v[i]).bits : from_f32<F16>(v[i]).bits;
  return make_uint2(u[0] | static_cast<uint32_t>(u[1]) << 16, u[2] | static_cast<uint32_t>(u[3]) << 16);
}
// eight 16-bit outputs o .. o + 7, those below n
__device__ __forceinline__ void store_narrow(const MmArgs& a, uint16_t* p, int o, uint4 v) {
  if (o + 8 <= a.n) {
    __builtin_memcpy(p, &v, sizeof(v));
    return;
  }
  uint64_t lo = static_cast<uint64_t>(v.y) << 32 | v.x, hi = static_cast<uint64_t>(v.w) << 32 | v.z;
#pragma unroll 1
  for (int i = 0; i < 8 && o + i < a.n; ++i) {
    p[i] = static_cast<uint16_t>(lo);
    lo = lo >> 16 | hi << 48;
    hi >>= 16;
  }
}
// outputs o .. o + 3 of output row p
__device__ __forceinline__ void store_y(const MmArgs& a, int64_t p, int o, const float* v) {
  const int n = a.n - o;
  if (n <= 0) return;
  const int64_t i = p * a.ldy + o;
  if (a.y_dtype == GPTQ_F32) store4(static_cast<float*>(a.Y) + i, v, n);
  else if (a.y_dtype == GPTQ_BF16) store4(static_cast<BF16*>(a.Y) + i, v, n);
  else store4(static_cast<F16*>(a.Y) + i, v, n);
}

// One wave copies 64 16-byte pieces to LDS: lane l's bytes land at base + 16 l (base uniform).
// Issued from inline assembly, which has no register result; the caller waits with wait_copies.
__device__ __forceinline__ void copy16(const void* src, unsigned base) {
  unsigned saved;
  asm volatile(
      "s_mov_b32 %0, m0\n\t"
      "s_mov_b32 m0, %2\n\t"
      "global_load_lds_dwordx4 %1, off\n\t"
      "s_mov_b32 m0, %0"
      : "=&s"(saved)
      : "v"(src), "s"(base)
      : "memory");
}
// 64 4-byte pieces, lane l's to base + 4 l.
__device__ __forceinline__ void copy4(const void* src, unsigned base) {
  unsigned saved;
  asm volatile(
      "s_mov_b32 %0, m0\n\t"
      "s_mov_b32 m0, %2\n\t"
      "global_load_lds_dword %1, off\n\t"
      "s_mov_b32 m0, %0"
      : "=&s"(saved)
      : "v"(src), "s"(base)
      : "memory");
}
// The same from a scalar base and 32-bit offsets.
__device__ __forceinline__ void copy16_at(const void* from, uint32_t off, unsigned base) {
  unsigned saved;
  asm volatile(
      "s_mov_b32 %0, m0\n\t"
      "s_mov_b32 m0, %3\n\t"
      "global_load_lds_dwordx4 %1, %2\n\t"
      "s_mov_b32 m0, %0"
      : "=&s"(saved)
      : "v"(off), "s"(from), "s"(base)
      : "memory");
}
// s_waitcnt vmcnt(N): all but the last N copies and loads are done.
template <int N>
__device__ __forceinline__ void wait_vmcnt() {
  static_assert(N >= 0 && N < 64, "vmcnt field");
  __builtin_amdgcn_s_waitcnt(0xF70 | (N & 15) | ((N >> 4) << 14));
}
__device__ __forceinline__ void wait_copies() { __builtin_amdgcn_s_waitcnt(0xF70); }   // vmcnt(0)

// Tiles of tm rows that a launch has workgroups for: grouped, as many as any ranges can make.
int64_t tile_rows(const MmArgs& a, int tm) {
  return a.off == nullptr ? (a.m + tm - 1) / tm : a.m / tm + std::min<int64_t>(a.experts, a.m);
}

}  // namespace
}  // namespace gptq
