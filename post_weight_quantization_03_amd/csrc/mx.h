// The 4-bit microscaled form: e2m1 codes, two to a byte (the first in the low half), with one E8M0
// scale per 32 inputs of a row.  Shared by mx.hip and mx_moe.hip.
#pragma once

#include <type_traits>

#include "product.h"

namespace gptq {
namespace {

constexpr int MXB = 32;   // inputs per scale

// What the second operand of a product holds: 4-bit codes and scales, or 16-bit values; fp16 ones beside
// weights whose scales fp16 can take.
enum MxKind { kMx4 = 0, kMxBf16 = 1, kMxF16 = 2, kMxF16Direct = 3 };
template <int KIND>
using MxConst = std::integral_constant<int, KIND>;

typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
typedef _Float16 f16x2 __attribute__((ext_vector_type(2)));
typedef float f32x2 __attribute__((ext_vector_type(2)));

// Eight codes as bf16 values times their scale: e2m1's 2 significant bits fit bf16's 8, so nothing
// is rounded (below 2^-133 excepted).  The conversion takes the scale as the exponent field of an
// fp32 number, that is the E8M0 code itself: 0 stands for 2^-127, 255 for NaN.
__device__ __forceinline__ bf16x8 mx_bf16(uint32_t codes, uint32_t scale) {
  const float s = __uint_as_float(scale << 23);
  const bf16x2 a = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(codes, s, 0);
  const bf16x2 b = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(codes, s, 1);
  const bf16x2 c = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(codes, s, 2);
  const bf16x2 d = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(codes, s, 3);
  return bf16x8{a[0], a[1], b[0], b[1], c[0], c[1], d[0], d[1]};
}

// The same as fp16 values: exact for scales of 2^-23 to 2^13, where 0.5 becomes fp16's least value and 6
// stays below its largest.
__device__ __forceinline__ f16x8 mx_f16(uint32_t codes, uint32_t scale) {
  const float s = __uint_as_float(scale << 23);
  const f16x2 a = __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(codes, s, 0);
  const f16x2 b = __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(codes, s, 1);
  const f16x2 c = __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(codes, s, 2);
  const f16x2 d = __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(codes, s, 3);
  return f16x8{a[0], a[1], b[0], b[1], c[0], c[1], d[0], d[1]};
}
template <int KIND>
__device__ __forceinline__ auto mx_weights16(uint32_t codes, uint32_t scale) {
  if constexpr (KIND == kMxF16Direct) return mx_f16(codes, scale);
  else return mx_bf16(codes, scale);
}

// Scale codes seen, four at a time: whether mx_f16 takes all of them.
struct ScaleRange {
  typedef uint16_t u16x2 __attribute__((ext_vector_type(2)));
  u16x2 least = {127, 127}, most = {127, 127};
  __device__ __forceinline__ void add(uint32_t codes) {
    const u16x2 even = __builtin_bit_cast(u16x2, codes & 0x00FF00FFu);
    const u16x2 odd = __builtin_bit_cast(u16x2, codes >> 8 & 0x00FF00FFu);
    least = __builtin_elementwise_min(least, __builtin_elementwise_min(even, odd));
    most = __builtin_elementwise_max(most, __builtin_elementwise_max(even, odd));
  }
  __device__ __forceinline__ bool f16() const {
    return least[0] >= 104 && least[1] >= 104 && most[0] <= 140 && most[1] <= 140;
  }
};

// Eight 16-bit values of X for the matrix instructions.  Where the weights' scales are none that fp16
// takes, fp16's 11 significant bits go as two bf16 numbers, the upper 8 bits and the rest, both exact: two
// products.  An infinity has no rest.
template <int KIND>
struct XValues {
  std::conditional_t<KIND == kMxF16Direct, f16x8, bf16x8> hi;
  bf16x8 lo;   // kMxF16
  XValues() = default;
  __device__ __forceinline__ explicit XValues(i32x4 v) {
    if constexpr (KIND == kMxF16) {
      const f16x8 h = __builtin_bit_cast(f16x8, v);
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const float f = static_cast<float>(h[i]);
        const float up = __uint_as_float(__float_as_uint(f) & 0xFFFF0000u);
        hi[i] = static_cast<__bf16>(up);
        lo[i] = static_cast<__bf16>(f == up ? 0.0f : f - up);
      }
    } else {
      hi = __builtin_bit_cast(decltype(hi), v);
    }
  }
};
template <int KIND, typename W>
__device__ __forceinline__ f32x4 mx_mma16(W w, const XValues<KIND>& x, f32x4 acc) {
  if constexpr (KIND == kMxF16Direct) {
    return __builtin_amdgcn_mfma_f32_16x16x32_f16(w, x.hi, acc, 0, 0, 0);
  } else {
    if constexpr (KIND == kMxF16) acc = __builtin_amdgcn_mfma_f32_16x16x32_bf16(w, x.lo, acc, 0, 0, 0);
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(w, x.hi, acc, 0, 0, 0);
  }
}

// A barrier for LDS alone, which loads and copies cross.
__device__ __forceinline__ void lds_barrier() {
  asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
  __builtin_amdgcn_s_barrier();
  asm volatile("" ::: "memory");
}

__device__ __forceinline__ i32x8 widen(i32x4 v) { return i32x8{v[0], v[1], v[2], v[3], 0, 0, 0, 0}; }

}  // namespace
}  // namespace gptq
