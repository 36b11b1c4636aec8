// The 4-bit microscaled form: e2m1 codes, two to a byte (the first in the low half), with one E8M0
// scale per 32 inputs of a row.  Shared by mx.hip and mx_moe.hip.
#pragma once

#include "product.h"

namespace gptq {
namespace {

constexpr int MXB = 32;   // inputs per scale

// What the second operand of a product holds: 4-bit codes and scales, or 16-bit values.
enum MxKind { kMx4 = 0, kMxBf16 = 1, kMxF16 = 2 };

typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
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

// Eight 16-bit values of X for the bf16 instructions.  fp16's 11 significant bits are two bf16
// numbers, the upper 8 bits and the rest, both exact: two products, but weights of any scale (as
// fp16 a weight below 2^-24 or above 65504 would be lost).  An infinity has no rest.
template <int KIND>
struct XValues {
  bf16x8 hi, lo;
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
      hi = __builtin_bit_cast(bf16x8, v);
    }
  }
};
template <int KIND>
__device__ __forceinline__ f32x4 mx_mma16(bf16x8 w, const XValues<KIND>& x, f32x4 acc) {
  if constexpr (KIND == kMxF16) acc = __builtin_amdgcn_mfma_f32_16x16x32_bf16(w, x.lo, acc, 0, 0, 0);
  return __builtin_amdgcn_mfma_f32_16x16x32_bf16(w, x.hi, acc, 0, 0, 0);
}

__device__ __forceinline__ i32x8 widen(i32x4 v) { return i32x8{v[0], v[1], v[2], v[3], 0, 0, 0, 0}; }

}  // namespace
}  // namespace gptq
