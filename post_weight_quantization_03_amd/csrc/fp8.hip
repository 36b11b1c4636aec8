// Block-scaled 8-bit linear layers on gfx950: rounding to e4m3 with a scale per block of 128
// inputs, and the product of such activations and weights, dense or grouped by expert.
//
//   scale_b = max |x| / 448 (or the power of two at or above it),  q = rne_e4m3(x / scale_b)
//   Y[r, o] = sum_b xs[r, b] ws[o / 128, b] sum_{c in b} xq[r, c] q[o, c]
//
// For 16-bit Y the inner sums are v_mfma_f32_16x16x128_f8f6f4: one instruction's K is one block
// of 128, so its 16x16 result takes one scale per row and 128 outputs.  Weights are the first
// operand and activations the second: a lane then holds one activation row and 4 consecutive
// outputs, its scale is one register, and its outputs are stored together.  fp32 scales
// multiply each block's result in fp32; E8M0 scales are operands of the instruction itself.
// The 8-bit matrix instructions of this chip (all shapes alike, by experiment) add 8
// consecutive products at the scale of the largest and cut what lies 2^-13 below it: at most
// 7 * 2^-13 of sum |x q|.  For 16-bit Y that is taken: it is under bf16's half step of 2^-8 (of the same
// sum) though not under fp16's 2^-11, and small beside the codes' own 2^-4.  Errors relative to the
// result's norm (512 x 2048 x 4096, E8M0): 1.5e-5 on normal inputs, 5e-5 with channels 20 times as
// large, 9e-5 with one 1000 times as large; with fp16's rounding 2.08, 2.13 and 2.26e-4 where fp32 sums
// rounded to fp16 have 2.07e-4, with bf16's 1.66e-3 either way.
// fp32 Y is for those who want fp32 sums: the codes are turned into bf16, which holds them exactly, and
// multiplied by v_mfma_f32_16x16x32_bf16 (4096 x 4096 x 4096 59 us to fp16, 147 to fp32).
#include <algorithm>
#include <cfloat>

#include "product.h"

namespace gptq {
namespace {

constexpr int FB = 128;   // inputs per scale

// ---------------------------------------------------------------------------- rounding

__device__ __forceinline__ uint32_t eight_lanes_max(uint32_t t) {
  for (int d = 1; d < 8; d <<= 1) t = max(t, static_cast<uint32_t>(__shfl_xor(static_cast<int>(t), d)));
  return t;
}

struct Scale {
  float s;        // the scale
  uint8_t code;   // its E8M0 code
};
template <bool E8>
__device__ __forceinline__ Scale block_scale(uint32_t top) {
  if (top >= 0x7F800000u) return {__uint_as_float(0x7FC00000u), 255};
  if constexpr (E8) {
    // 448 = 1.75 * 2^8
    int e = static_cast<int>(top >> 23) - 127 - 8 + ((top & 0x7FFFFFu) > 0x600000u);
    e = max(e, -126);
    return {__uint_as_float(static_cast<uint32_t>(e + 127) << 23), static_cast<uint8_t>(e + 127)};
  } else {
    return {fmaxf(__uint_as_float(top) / 448.0f, __uint_as_float(0x00800000u)), 0};
  }
}

// fp32 toward which the exact quotient lies, last bit set where it is inexact (rounding to odd):
// rounding that to e4m3 is rounding the quotient itself, since e4m3's values and midpoints have
// that bit clear.
__device__ __forceinline__ float odd_quotient(float x, float s, float r) {
  const float q0 = x * r;
  const float q = fmaf(fmaf(-q0, s, x), r, q0);
  const float e = fmaf(-q, s, x);   // exact sign of the true quotient less q
  const uint32_t u = __float_as_uint(q);
  const uint32_t down = (u ^ __float_as_uint(e)) >> 31;
  return e == 0.0f ? q : __uint_as_float((u - down) | 1u);
}

// N values of a block as e4m3 bytes, 4 to a word.
template <bool E8, int N>
__device__ __forceinline__ void round_values(const float* x, Scale sc, uint32_t* w) {
  float v[N];
  if (!(sc.s == sc.s)) {
#pragma unroll
    for (int i = 0; i < N; ++i) v[i] = 0.0f;
  } else if constexpr (E8) {
    const float r = __uint_as_float((254u - sc.code) << 23);
#pragma unroll
    for (int i = 0; i < N; ++i) v[i] = x[i] * r;   // exact
  } else {
    // both sides by 2^64 where the residual of a tiny quotient would leave fp32's range
    const float up = sc.s < 0x1p-60f ? 0x1p64f : 1.0f;
    const float s = sc.s * up, r = 1.0f / s;
#pragma unroll
    for (int i = 0; i < N; ++i) v[i] = odd_quotient(x[i] * up, s, r);
  }
#pragma unroll
  for (int i = 0; i < N; i += 4) {
    int p = __builtin_amdgcn_cvt_pk_fp8_f32(v[i], v[i + 1], 0, false);
    p = __builtin_amdgcn_cvt_pk_fp8_f32(v[i + 2], v[i + 3], p, true);
    w[i / 4] = static_cast<uint32_t>(p);
  }
}

struct QuantArgs {
  int64_t rows;
  int cols;
  const void* X;
  int64_t ldx, bsx;
  uint8_t* Q;
  void* S;
  int64_t lsr, lsb, bss;
};

template <bool E8>
__device__ __forceinline__ void store_scale(const QuantArgs& a, int64_t i, Scale sc) {
  if constexpr (E8) static_cast<uint8_t*>(a.S)[i] = sc.code;
  else static_cast<float*>(a.S)[i] = sc.s;
}

// 1 x 128 blocks: 8 lanes per block, 16 values each; a workgroup takes QB blocks of 32 / QB rows.
// Bound by memory.  32 blocks of one row are 8 KB in one piece (8192 x 4096 in bf16: 20.2 us, 5.0
// TB/s, a copy's rate here; one block of 32 rows 25.9 us although its scales leave in one
// piece); rows of fewer than 16 blocks take 4.
template <typename T, bool E8, int QB>
__global__ __launch_bounds__(256) void quant_rows_kernel(QuantArgs a) {
  const int u = threadIdx.x / 8, b = blockIdx.y * QB + u % QB;
  const int64_t row = static_cast<int64_t>(blockIdx.x) * (32 / QB) + u / QB;
  const int col = b * FB + (threadIdx.x & 7) * 16;
  const bool live = row < a.rows && col < a.cols;
  float x[16];
#pragma unroll
  for (int i = 0; i < 16; ++i) x[i] = 0.0f;
  if (live) load_row<T, 16>(static_cast<const T*>(a.X) + blockIdx.z * a.bsx + row * a.ldx + col, x);
  const uint32_t top = eight_lanes_max(top_bits<16>(x));
  if (!live) return;
  const Scale sc = block_scale<E8>(top);
  uint32_t w[4];
  round_values<E8, 16>(x, sc, w);
  *reinterpret_cast<uint4*>(a.Q + (blockIdx.z * a.rows + row) * a.cols + col) = make_uint4(w[0], w[1], w[2], w[3]);
  if ((threadIdx.x & 7) == 0) store_scale<E8>(a, blockIdx.z * a.bss + row * a.lsr + b * a.lsb, sc);
}

// 128 x 128 blocks: one workgroup per block, 64 values per thread (4 rows of 16) in registers.
// Bound by memory (64 x 1408 x 2048 in bf16: 108 us, 5.1 TB/s).
template <typename T, bool E8>
__global__ __launch_bounds__(256) void quant_tile_kernel(QuantArgs a) {
  __shared__ uint32_t tops[4];
  const int b = blockIdx.y;
  const int64_t row0 = static_cast<int64_t>(blockIdx.x) * FB + threadIdx.x / 8;
  const int col = b * FB + (threadIdx.x & 7) * 16;
  float x[4][16];
  uint32_t top = 0;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
#pragma unroll
    for (int j = 0; j < 16; ++j) x[i][j] = 0.0f;
    if (row0 + 32 * i < a.rows && col < a.cols)
      load_row<T, 16>(static_cast<const T*>(a.X) + blockIdx.z * a.bsx + (row0 + 32 * i) * a.ldx + col, x[i]);
  }
#pragma unroll
  for (int i = 0; i < 4; ++i) top = max(top, top_bits<16>(x[i]));
  for (int d = 1; d < 64; d <<= 1) top = max(top, static_cast<uint32_t>(__shfl_xor(static_cast<int>(top), d)));
  if ((threadIdx.x & 63) == 0) tops[threadIdx.x >> 6] = top;
  __syncthreads();
  top = max(max(tops[0], tops[1]), max(tops[2], tops[3]));
  const Scale sc = block_scale<E8>(top);
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if (row0 + 32 * i >= a.rows || col >= a.cols) continue;
    uint32_t w[4];
    round_values<E8, 16>(x[i], sc, w);
    *reinterpret_cast<uint4*>(a.Q + (blockIdx.z * a.rows + row0 + 32 * i) * a.cols + col) =
        make_uint4(w[0], w[1], w[2], w[3]);
  }
  if (threadIdx.x == 0) store_scale<E8>(a, blockIdx.z * a.bss + blockIdx.x * a.lsr + b * a.lsb, sc);
}

template <typename T, bool E8>
gptq_status launch_quant(const QuantArgs& a, int batch, int block_rows, hipStream_t stream) {
  const int64_t kb = (a.cols + FB - 1) / FB;
  const int qb = block_rows == FB ? 1 : kb >= 16 ? 32 : 4, qr = block_rows == FB ? FB : 32 / qb;
  const int64_t gx = (a.rows + qr - 1) / qr, gy = (kb + qb - 1) / qb;
  if (gx > (1 << 24) - 1 || gy > 65535 || batch > 65535) return GPTQ_ERR_UNSUPPORTED;
  const dim3 grid(static_cast<unsigned>(gx), static_cast<unsigned>(gy), batch), block(256);
  if (block_rows == FB) GPTQ_LAUNCH((quant_tile_kernel<T, E8>), grid, block, 0, stream, a);
  else if (qb == 32) GPTQ_LAUNCH((quant_rows_kernel<T, E8, 32>), grid, block, 0, stream, a);
  else GPTQ_LAUNCH((quant_rows_kernel<T, E8, 4>), grid, block, 0, stream, a);
  return GPTQ_OK;
}

template <typename T>
gptq_status launch_quant_t(const QuantArgs& a, int batch, int block_rows, bool e8, hipStream_t stream) {
  return e8 ? launch_quant<T, true>(a, batch, block_rows, stream) : launch_quant<T, false>(a, batch, block_rows, stream);
}

// ---------------------------------------------------------------------------- product

// Output rows without a row of X are zeros, also where a weight or its scale is NaN: the kernels
// mark them in LDS before their first stage (a load of row_index between the stores of Y would
// wait for the stores before it: 49152 rows of 64 experts of 1408 x 2048 238 us, 229 so).

// How a kernel multiplies: 8-bit instructions with fp32 or E8M0 scales, or bf16 ones.
enum MmaKind { kMmaF32Scale = 0, kMmaE8M0 = 1, kMmaExact = 2 };

// A lane's 32 codes of a block: as they are, or as bf16 (4 operands of 8).
template <int KIND>
struct Operand {
  i32x8 v;
  Operand() = default;
  __device__ __forceinline__ explicit Operand(i32x8 x) : v(x) {}
};
template <>
struct Operand<kMmaExact> {
  bf16x8 v[4];
  Operand() = default;
  __device__ __forceinline__ explicit Operand(i32x8 x) {
    typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const bf16x2 lo = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(x[i], 1.0f, false);
      const bf16x2 hi = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(x[i], 1.0f, true);
      v[i / 2][4 * (i & 1) + 0] = lo[0];
      v[i / 2][4 * (i & 1) + 1] = lo[1];
      v[i / 2][4 * (i & 1) + 2] = hi[0];
      v[i / 2][4 * (i & 1) + 3] = hi[1];
    }
  }
};

// w x of one block of 128 inputs of 16 outputs and 16 rows, without scales.
template <int KIND>
__device__ __forceinline__ f32x4 block_dot(const Operand<KIND>& w, const Operand<KIND>& x) {
  f32x4 t = {0.0f, 0.0f, 0.0f, 0.0f};
  if constexpr (KIND == kMmaExact) {
#pragma unroll
    for (int i = 0; i < 4; ++i) t = __builtin_amdgcn_mfma_f32_16x16x32_bf16(w.v[i], x.v[i], t, 0, 0, 0);
    return t;
  } else {
    return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(w.v, x.v, t, 0, 0, 0, 0, 0, 0);
  }
}

// acc += (w x) sx sw for one block of 128 inputs of 16 outputs and 16 rows.
template <int KIND>
__device__ __forceinline__ void block_mma(const Operand<KIND>& w, const Operand<KIND>& x, float sx, float sw,
                                          f32x4& acc) {
  if constexpr (KIND == kMmaE8M0) {
    acc = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(w.v, x.v, acc, 0, 0, 0, __float_as_int(sw), 0,
                                                           __float_as_int(sx));
  } else {
    const f32x4 t = block_dot<KIND>(w, x);
    const float s = sx * sw;
#pragma unroll
    for (int r = 0; r < 4; ++r) acc[r] = fmaf(t[r], s, acc[r]);
  }
}

// Scale i of an array: fp32, or for kMmaE8M0 the code itself in a register.
template <int KIND>
__device__ __forceinline__ float load_scale(const MmArgs& a, const void* p, int64_t i) {
  if constexpr (KIND == kMmaE8M0) return __int_as_float(static_cast<const uint8_t*>(p)[i]);
  if constexpr (KIND == kMmaExact)
    if (a.e8) return e8m0_f32(static_cast<const uint8_t*>(p)[i]);
  return static_cast<const float*>(p)[i];
}
template <int KIND>
__device__ __forceinline__ float load_xs(const MmArgs& a, int64_t row, int b) {
  return load_scale<KIND>(a, a.xs, row * a.xsr + b * a.xsb);
}
template <int KIND>
__device__ __forceinline__ float load_ws(const MmArgs& a, int e, int ob, int b) {
  return load_scale<KIND>(a, a.ws, (static_cast<int64_t>(e) * a.nb + ob) * a.kb + b);
}

// Tiles of TM rows x TN outputs, WM x WN waves.  A stage is one block of 128 inputs: TM + TN
// rows of 128 bytes in LDS, two buffers, the next stage's copies in flight during this one's
// products.  The 16-byte piece c of row r lies at c ^ (r / 2 % 8), so that 16 lanes reading
// the same piece of 16 rows cover all 64 banks.  Bound by LDS reads and copies; two workgroups
// per CU cover each other's waits (4096 x 4096 at 1024 rows: 42 us, 0.82 PFLOP/s).
template <int TM, int TN, int WM, int WN, int KIND>
__global__ __launch_bounds__(WM* WN * 64) void fp8_tile_kernel(MmArgs a) {
  constexpr int NW = WM * WN, NT = NW * 64;
  constexpr int FM = TM / WM / 16, FN = TN / WN / 16;
  constexpr int STAGE = (TM + TN) * FB;
  constexpr int LD = (TM + TN) / 8 / NW;
  static_assert(NW % 2 == 0 && (TM + TN) % (8 * NW) == 0 && TM <= NT && FB % (TN / WN) == 0, "tile shape");
  __shared__ __attribute__((aligned(128))) uint8_t lds[2 * STAGE];
  __shared__ float sxs[2 * TM];
  __shared__ bool lost[TM];
  const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int64_t mt = blockIdx.x / a.tiles_n;
  const int n0 = static_cast<int>(blockIdx.x - mt * a.tiles_n) * TN;
  const Tile t = find_tile<TM>(a, mt);
  if (t.count <= 0) return;
  const uint8_t* We = a.W + static_cast<int64_t>(t.e) * a.n * a.k;
  const uint8_t* zeros = reinterpret_cast<const uint8_t*>(&zero16);

  const int c = (lane & 7) ^ ((4 * wave + lane / 16) & 7);   // this lane's piece: the same in every copy
  const uint8_t* src[LD];
#pragma unroll
  for (int i = 0; i < LD; ++i) {
    const int r = (wave + NW * i) * 8 + lane / 8;
    if (r < TM) {
      const int64_t row = source_row(a, t.p0 + min(r, t.count - 1));
      src[i] = row >= 0 ? a.X + row * a.ldx + 16 * c : nullptr;
    } else {
      src[i] = We + static_cast<int64_t>(min(n0 + r - TM, a.n - 1)) * a.k + 16 * c;
    }
  }
  const int64_t srow = tid < TM ? source_row(a, t.p0 + min(tid, t.count - 1)) : -1;
  if (tid < TM) lost[tid] = srow < 0;
  float sx_next = 0.0f;
  const unsigned lds0 = static_cast<unsigned>(reinterpret_cast<uintptr_t>(
      (__attribute__((address_space(3))) uint8_t*)lds));
  auto issue = [&](int s) {
    const int k0 = s * FB;
    const bool in = k0 + 16 * c < a.k;
    if (srow >= 0) sx_next = load_xs<KIND>(a, srow, s);
#pragma unroll
    for (int i = 0; i < LD; ++i)
      copy16(in && src[i] != nullptr ? src[i] + k0 : zeros, lds0 + (s & 1) * STAGE + (wave + NW * i) * 1024);
  };

  const int wm = wave / WN, wn = wave % WN;
  const int j = lane & 15, q = lane >> 4;
  const int ob = min((n0 + wn * (TN / WN)) / FB, a.nb - 1);
  const f32x4 zero = {0.0f, 0.0f, 0.0f, 0.0f};
  f32x4 y[FM][FN];
#pragma unroll
  for (int i = 0; i < FM; ++i)
#pragma unroll
    for (int h = 0; h < FN; ++h) y[i][h] = zero;
  auto frag = [&](const uint8_t* base, int r) {
    const int sw = (r >> 1) & 7;
    const i32x4 lo = *reinterpret_cast<const i32x4*>(base + r * FB + 16 * ((2 * q) ^ sw));
    const i32x4 hi = *reinterpret_cast<const i32x4*>(base + r * FB + 16 * ((2 * q + 1) ^ sw));
    return Operand<KIND>(i32x8{lo[0], lo[1], lo[2], lo[3], hi[0], hi[1], hi[2], hi[3]});
  };
  issue(0);
  for (int s = 0; s < a.kb; ++s) {
    wait_copies();
    if (tid < TM) sxs[(s & 1) * TM + tid] = sx_next;
    __syncthreads();
    if (s + 1 < a.kb) issue(s + 1);
    const float sw = load_ws<KIND>(a, t.e, ob, s);
    const uint8_t* xb = lds + (s & 1) * STAGE;
    const uint8_t* wb = xb + TM * FB;
    Operand<KIND> wf[FN];
#pragma unroll
    for (int h = 0; h < FN; ++h) wf[h] = frag(wb, wn * (TN / WN) + 16 * h + j);
#pragma unroll
    for (int i = 0; i < FM; ++i) {
      const Operand<KIND> xf = frag(xb, wm * (TM / WM) + 16 * i + j);
      const float sx = sxs[(s & 1) * TM + wm * (TM / WM) + 16 * i + j];
#pragma unroll
      for (int h = 0; h < FN; ++h) block_mma<KIND>(wf[h], xf, sx, sw, y[i][h]);
    }
  }
  // lane: row j of each 16, outputs 4 q .. 4 q + 3
#pragma unroll
  for (int i = 0; i < FM; ++i) {
    const int r = wm * (TM / WM) + 16 * i + j;
    if (r >= t.count) continue;
    const bool none = lost[r];
#pragma unroll
    for (int h = 0; h < FN; ++h) {
      const f32x4 s = none ? zero : y[i][h];
      const float v[4] = {s[0], s[1], s[2], s[3]};
      store_y(a, t.p0 + r, n0 + wn * (TN / WN) + 16 * h + 4 * q, v);
    }
  }
}

template <int TM, int TN, int WM, int WN>
gptq_status launch_tile(MmArgs a, hipStream_t stream) {
  a.tiles_n = (a.n + TN - 1) / TN;
  const dim3 g(static_cast<unsigned>(tile_rows(a, TM) * a.tiles_n)), b(WM * WN * 64);
  if (a.y_dtype == GPTQ_F32) GPTQ_LAUNCH((fp8_tile_kernel<TM, TN, WM, WN, kMmaExact>), g, b, 0, stream, a);
  else if (a.e8) GPTQ_LAUNCH((fp8_tile_kernel<TM, TN, WM, WN, kMmaE8M0>), g, b, 0, stream, a);
  else GPTQ_LAUNCH((fp8_tile_kernel<TM, TN, WM, WN, kMmaF32Scale>), g, b, 0, stream, a);
  return GPTQ_OK;
}

// The same product for large problems: 256 x 256 tiles, 8 waves of 128 x 64 (8 x 4 blocks of
// 16 x 16) or, with E8M0 scales, which leave no folds to do meanwhile, 4 of 128 x 128 (8192 x 4096 x
// 14336: 402 us = 2.39 PFLOP/s, and 358 = 2.69, which 8 waves take 382 for); one workgroup per CU.
// Bound by the matrix cores (67% busy).  Two buffers of 64 KB; operands go global -> LDS with a
// scalar base that moves by 128 bytes a stage and one 32-bit offset per lane and copy, so that
// a stage's copies cost little vector arithmetic.  Before a wave's last three rows of blocks it
// has read all it needs of the stage: there the workgroup waits for the next stage's copies, and
// the products of these rows cover the first reads of the next stage and half of the copies of the one
// after it; the other half goes out with the next stage's first products.  The fold of a
// product (y += t * scale) runs under the third product after it.
// A tile of up to 128 rows or outputs (the last of a ragged problem or expert) goes the same way
// with half the work per wave: 384 rows of operands a stage and waves of 128 x 64 or 64 x 64.
constexpr int BIG_KB = 2048;   // most blocks of inputs (LDS for the outputs' scales)
constexpr int BIG = 256, BIG_STAGE = 2 * BIG * FB;
struct BigLds {
  uint8_t* lds;     // two stages
  bool* lost;       // [BIG]
  float* scs;       // [2][2][BIG]: the rows' scales (fp32: twice, so that every wave copies 64)
  float* scw;       // [2][kb]: the outputs' scales
};
// Outputs n0 .. of the rows of t: xrows rows of X and ROWS - xrows of W, waves_n waves beside each
// other.
template <int KIND, int NW, int FM, int FN, int ROWS>
__device__ __forceinline__ void big_tile(const MmArgs& a, const Tile& t, int n0, int xrows, int waves_n, const BigLds& m) {
  constexpr int TM = BIG, STAGE = BIG_STAGE;
  constexpr int LD = ROWS / 8 / NW;   // copies per wave and stage
  constexpr bool E8 = KIND == kMmaE8M0;
  uint8_t* const lds = m.lds;
  bool* const lost = m.lost;
  float* const scw = m.scw;
  const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int ldx = xrows / 8 / NW;     // of them of X

  const int c = (lane & 7) ^ ((4 * wave + lane / 16) & 7);   // this lane's piece: the same in every copy
  const uint8_t* xbase = a.X + (a.rows == nullptr ? t.p0 * a.ldx : 0);
  const uint8_t* wbase = a.W + (static_cast<int64_t>(t.e) * a.n + n0) * a.k;
  uint32_t off[LD];
#pragma unroll
  for (int i = 0; i < LD; ++i) {
    const int r = (wave + NW * i) * 8 + lane / 8;
    if (i < ldx) {
      const int64_t row = source_row(a, t.p0 + min(r, t.count - 1));   // none: row 0, and zeros at the end
      off[i] = static_cast<uint32_t>(max(a.rows == nullptr ? row - t.p0 : row, static_cast<int64_t>(0)) * a.ldx) + 16 * c;
    } else {
      off[i] = static_cast<uint32_t>(min(r - xrows, a.n - 1 - n0)) * static_cast<uint32_t>(a.k) + 16 * c;
    }
  }
  constexpr int SB = E8 ? 1 : 4;   // bytes of a scale
  const int srow_r = tid & (TM - 1);
  const int64_t own = source_row(a, t.p0 + min(srow_r, t.count - 1)), srow = max(own, static_cast<int64_t>(0));
  lost[srow_r] = own < 0;
  const uint8_t* xsp = static_cast<const uint8_t*>(a.xs) + srow * a.xsr * SB;   // moves by a block of inputs a stage
  const int64_t xstep = a.xsb * SB;
  float sx_next = 0.0f;
  for (int b = tid; b < 2 * a.kb; b += NW * 64)
    scw[b] = load_ws<KIND>(a, t.e, min(n0 / FB + (b >= a.kb), a.nb - 1), b >= a.kb ? b - a.kb : b);
  const unsigned lds0 = static_cast<unsigned>(reinterpret_cast<uintptr_t>(
      (__attribute__((address_space(3))) uint8_t*)lds));
  const bool cut = 16 * c >= a.k - (a.kb - 1) * FB;   // this lane's piece of the last stage lies past K
  float(*const scs)[2][TM] = reinterpret_cast<float(*)[2][TM]>(m.scs);
  const unsigned scs0 = static_cast<unsigned>(reinterpret_cast<uintptr_t>(
      (__attribute__((address_space(3))) float*)m.scs));
  // the scales of the stage after the last call's.  fp32 ones go to LDS like the operands: loads
  // to registers between those copies cost 30 us of 400 at 8192 x 4096 x 14336
  auto issue_scales = [&](int s) {
    if constexpr (E8) sx_next = __int_as_float(*xsp);
    else copy4(xsp, scs0 + ((s & 1) * 2 * TM + wave * 64) * 4);
    xsp += xstep;
  };
  auto issue_copies = [&](int s, int from, int to) {
    const uint8_t* xb = xbase + static_cast<int64_t>(s) * FB;
    const uint8_t* wb = wbase + static_cast<int64_t>(s) * FB;
    const unsigned dst = lds0 + (s & 1) * STAGE + wave * 1024;
    const uint32_t back = s == a.kb - 1 && cut ? 16 * c : 0;   // the row's first piece instead; zeroed below
#pragma unroll
    for (int i = from; i < to; ++i) copy16_at(i < ldx ? xb : wb, off[i] - back, dst + NW * i * 1024);
  };
  // the copies and scales of stage s have landed; the next barrier makes them visible
  auto land = [&](int s, bool last) {
    wait_copies();
    if (last && cut) {
#pragma unroll
      for (int i = 0; i < LD; ++i)
        *reinterpret_cast<uint4*>(lds + (s & 1) * STAGE + (wave + NW * i) * 1024 + 16 * lane) = make_uint4(0, 0, 0, 0);
    }
    if constexpr (E8) scs[s & 1][0][srow_r] = sx_next;
  };
  auto barrier = [&] {
    asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
    __builtin_amdgcn_s_barrier();
    asm volatile("" ::: "memory");
  };

  const int wm = wave / waves_n, wn = wave % waves_n;
  const int j = lane & 15, q = lane >> 4;
  const int xr = wm * 16 * FM, wr = xrows + wn * 16 * FN;
  // pieces q and q + 4 of a row are this lane's 32 inputs (any order that both operands share):
  // the lanes that one LDS access serves together then meet no bank twice
  const int swz = (j >> 1) & 7;
  const int at0 = j * FB + 16 * (q ^ swz), at1 = j * FB + 16 * ((q + 4) ^ swz);
  auto half_frag = [&](int s, int r, int half, Operand<KIND>& o) {
    const i32x4 v = *reinterpret_cast<const i32x4*>(lds + (s & 1) * STAGE + r * FB + (half ? at1 : at0));
#pragma unroll
    for (int i = 0; i < 4; ++i) o.v[4 * half + i] = v[i];
  };
  auto scale_of = [&](int s, int i) { return scs[s & 1][E8 ? 0 : wn & 1][xr + 16 * i + j]; };
  const float* const swp = scw + wn * FN / 8 * a.kb;   // this wave's 128 outputs

  const f32x4 zero = {0.0f, 0.0f, 0.0f, 0.0f};
  f32x4 y[FM][FN], td[4];   // td: the last products, not folded yet
  float ts[4];              // and their scales
#pragma unroll
  for (int i = 0; i < FM; ++i)
#pragma unroll
    for (int h = 0; h < FN; ++h) y[i][h] = zero;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    td[i] = zero;
    ts[i] = 0.0f;
  }
  Operand<KIND> xf[4], wf[FN];   // row of blocks i in xf[i % 4]
  float sc[4], sw = 0.0f;
  // Products of a stage: rows of blocks one after another, then the last three together, output
  // block by output block.
  constexpr int LAST = 3, SPLIT = (FM - LAST) * FN;   // rows taken together, products before them
  constexpr int EARLY = LAST * FN / 2;                // copies issued with them, one after every second product
  auto row_at = [](int p) constexpr { return p < SPLIT ? p / FN : FM - LAST + (p - SPLIT) % LAST; };
  auto col_at = [](int p) constexpr { return p < SPLIT ? p % FN : (p - SPLIT) / LAST; };
  // issue product p and fold the one three before it; with E8M0 scales it goes straight into
  // y.  The empty constraint keeps the multiply-adds here and the barrier keeps everything in the
  // order written (left to itself the compiler puts all folds behind the last product, or all
  // reads before the first, and spills).
  auto product = [&](auto P) {
    constexpr int p = P, i = row_at(p), h = col_at(p);
    if constexpr (E8) {
      block_mma<KIND>(wf[h], xf[i % 4], sc[i % 4], sw, y[i][h]);
    } else {
      constexpr int o = (p + FM * FN - 3) % (FM * FN), oi = row_at(o), oh = col_at(o);
      td[p % 4] = block_dot<KIND>(wf[h], xf[i % 4]);
      if constexpr (h == 0) sc[i % 4] *= sw;
      ts[p % 4] = sc[i % 4];
#pragma unroll
      for (int r = 0; r < 4; ++r) y[oi][oh][r] = fmaf(td[o % 4][r], ts[o % 4], y[oi][oh][r]);
      asm volatile("" : "+v"(y[oi][oh]));
    }
    __builtin_amdgcn_sched_barrier(0);
  };
  // one stage; kMore: another follows, kIssue: and one after that (constants, so that the
  // loop's body has no branch)
  auto stage = [&](int s, auto kMore, auto kIssue) {
    // all rows but the last three; row i + 3 is read meanwhile, one access after each product
    static_for(std::make_integer_sequence<int, SPLIT>{}, [&](auto P) {
      constexpr int p = P, i = p / FN, h = p % FN;
      product(P);
      if constexpr (h == 0) half_frag(s, xr + 16 * (i + 3), 0, xf[(i + 3) % 4]);
      if constexpr (h == 1) half_frag(s, xr + 16 * (i + 3), 1, xf[(i + 3) % 4]);
      if constexpr (h == 2) sc[(i + 3) % 4] = scale_of(s, i + 3);
      // the rest of the next stage's copies
      if constexpr (kMore && p % 2 == 1 && EARLY + p / 2 < LD) issue_copies(s + 1, EARLY + p / 2, EARLY + p / 2 + 1);
      __builtin_amdgcn_sched_barrier(0);
    });
    float sw1 = 0.0f;
    if constexpr (kMore) {
      land(s + 1, !kIssue);
      barrier();
      if constexpr (kIssue) issue_scales(s + 2);
      // operand 0 is free: the next stage's first
      half_frag(s + 1, xr, 0, xf[0]);
      half_frag(s + 1, xr, 1, xf[0]);
      sc[0] = scale_of(s + 1, 0);
      sw1 = swp[s + 1];
      __builtin_amdgcn_sched_barrier(0);
    }
    // the last three rows: a weight operand makes room for the next stage's after its third product
    static_for(std::make_integer_sequence<int, LAST * FN>{}, [&](auto Q) {
      constexpr int n = Q, h = n / LAST;
      product(std::integral_constant<int, SPLIT + n>{});
      if constexpr (kMore && n % LAST == LAST - 1) {
        half_frag(s + 1, wr + 16 * h, 0, wf[h]);
        half_frag(s + 1, wr + 16 * h, 1, wf[h]);
      }
      // a copy takes the CU's address unit 16 cycles: issued together, the waves' copies hold up
      // their next products
      if constexpr (kIssue && n % 2 == 1) issue_copies(s + 2, n / 2, n / 2 + 1);
      __builtin_amdgcn_sched_barrier(0);
    });
    if constexpr (kMore) {
#pragma unroll
      for (int i = 1; i < 3; ++i) {
        half_frag(s + 1, xr + 16 * i, 0, xf[i]);
        half_frag(s + 1, xr + 16 * i, 1, xf[i]);
        sc[i] = scale_of(s + 1, i);
      }
      sw = sw1;
      __builtin_amdgcn_sched_barrier(0);
    }
  };

  issue_scales(0);
  issue_copies(0, 0, LD);
  land(0, a.kb == 1);
  barrier();
  if (a.kb > 1) {
    issue_scales(1);
    issue_copies(1, 0, EARLY);
  }
#pragma unroll
  for (int i = 0; i < 3; ++i) {
    half_frag(0, xr + 16 * i, 0, xf[i]);
    half_frag(0, xr + 16 * i, 1, xf[i]);
    sc[i] = scale_of(0, i);
  }
#pragma unroll
  for (int h = 0; h < FN; ++h) {
    half_frag(0, wr + 16 * h, 0, wf[h]);
    half_frag(0, wr + 16 * h, 1, wf[h]);
  }
  sw = swp[0];
  const std::true_type yes;
  const std::false_type no;
  for (int s = 0; s + 2 < a.kb; ++s) stage(s, yes, yes);
  if (a.kb > 1) stage(a.kb - 2, yes, no);
  stage(a.kb - 1, no, no);
  if constexpr (!E8)
    static_for(std::make_integer_sequence<int, 3>{}, [&](auto P) {
      constexpr int p = FM * FN - 3 + P, i = row_at(p), h = col_at(p);
#pragma unroll
      for (int r = 0; r < 4; ++r) y[i][h][r] = fmaf(td[p % 4][r], ts[p % 4], y[i][h][r]);
    });
  // Of outputs 16 h + 4 q .. of two neighbouring h, lanes of odd and even q exchange one each (they
  // are of one row): a lane then stores 8 in 16 bytes, and four lanes 64 bytes of a row in one
  // piece.  The code is short because it runs once a tile, from outside the instruction cache.
  const int o0 = n0 + wn * 16 * FN + 16 * (q & 1) + 8 * (q >> 1);
  const bool wide = n0 + (wn + 1) * 16 * FN <= a.n;
  auto store = [&](auto kBf16, auto kWide) {
    uint16_t* out = static_cast<uint16_t*>(a.Y) + (t.p0 + xr + j) * a.ldy + o0;
#pragma unroll
    for (int i = 0; i < FM; ++i) {
      if (xr + 16 * i + j < t.count) {
        const bool none = lost[xr + 16 * i + j];
#pragma unroll
        for (int h = 0; h < FN; h += 2) {
          const uint2 u = pack16<kBf16>(y[i][h]), v = pack16<kBf16>(y[i][h + 1]);
          const auto lo = __builtin_amdgcn_permlane16_swap(u.x, v.x, false, false);
          const auto hi = __builtin_amdgcn_permlane16_swap(u.y, v.y, false, false);
          const uint4 w = none ? make_uint4(0, 0, 0, 0) : make_uint4(lo[0], hi[0], lo[1], hi[1]);
          if constexpr (kWide) __builtin_memcpy(out + 16 * h, &w, sizeof(w));
          else store_narrow(a, out + 16 * h, o0 + 16 * h, w);
        }
      }
      out += 16 * a.ldy;
    }
  };
  if (a.y_dtype == GPTQ_BF16) {
    if (wide) store(yes, yes);
    else store(yes, no);
  } else {
    if (wide) store(no, yes);
    else store(no, no);
  }
}

template <int KIND, int NW>
__global__ __launch_bounds__(NW * 64) void fp8_big_kernel(MmArgs a) {
  __shared__ __attribute__((aligned(128))) uint8_t lds[2 * BIG_STAGE];
  __shared__ bool lost[BIG];
  __shared__ float scs[2 * 2 * BIG];
  extern __shared__ float scw[];
  int64_t mt;
  int nt;
  if (!ordered_tile(a.order, blockIdx.x, &mt, &nt)) return;
  const int n0 = nt * BIG;
  const Tile t = find_tile<BIG>(a, mt);
  if (t.count <= 0) return;
  const BigLds m{lds, lost, scs, scw};
  const bool few_rows = t.count <= BIG / 2;
  if (few_rows || a.n - n0 <= BIG / 2)
    big_tile<KIND, NW, 32 / NW, 4, BIG + BIG / 2>(a, t, n0, few_rows ? BIG / 2 : BIG, few_rows ? 4 : 2, m);
  else
    big_tile<KIND, NW, 8, 32 / NW, 2 * BIG>(a, t, n0, BIG, NW / 2, m);
}

gptq_status launch_big(MmArgs a, hipStream_t stream) {
  a.order = {(a.n + 255) / 256, tile_rows(a, 256)};
  const dim3 g(static_cast<unsigned>(order_grid(a.order)));
  const size_t lds = 2 * static_cast<size_t>(a.kb) * sizeof(float);
  if (a.e8) GPTQ_LAUNCH((fp8_big_kernel<kMmaE8M0, 4>), g, dim3(256), lds, stream, a);
  else GPTQ_LAUNCH((fp8_big_kernel<kMmaF32Scale, 8>), g, dim3(512), lds, stream, a);
  return GPTQ_OK;
}

// The same product for grids of few tiles: 64 x 64 tiles by 4 waves of 32 x 32, four buffers of
// 16 KB and three stages of copies in flight.  One such group of waves issues its stage's
// instructions in about 0.47 us however early the copies come (eight buffers, or operands read
// a stage ahead, gained nothing); a second group with every other stage and buffers of its own
// (KG = 2) fills the gaps where the CU has room for it.  All scales of the tile are in LDS before
// the first stage, so that the loop has no other loads and can wait for copies by their number.
constexpr int MID_KB[3] = {0, 224, 112};   // most blocks of inputs (260 bytes of scales each) by groups
constexpr int MID_PAIR = 60;               // most blocks with which two workgroups of one group fit a CU
// Two groups where a CU has one workgroup of one group at a time, by the number of workgroups or by
// their LDS (4096 x 14336 at 256 rows: 34.8 us with two, 55 with one; 1416 x 2000 at 333 rows, fp32
// Y: 10.8 and 13.8), and there are stages enough to share.
__host__ inline int mid_groups(int kb, double grid) {
  return kb >= 8 && kb <= MID_KB[2] && (grid <= 256 || kb > MID_PAIR) ? 2 : 1;
}
template <int KIND, int KG>
__global__ __launch_bounds__(KG * 256) void fp8_mid_kernel(MmArgs a) {
  constexpr int TM = 64, TN = 64, NW = 4, NB = 4;
  constexpr int STAGE = (TM + TN) * FB;
  constexpr int LD = (TM + TN) / 8 / NW;
  __shared__ __attribute__((aligned(128))) uint8_t lds[KG * NB * STAGE];
  extern __shared__ float scales[];   // [kb][TM] of the rows, then [kb] of the outputs
  __shared__ bool lost[TM];
  const int tid = threadIdx.x, lane = tid & 63, wave = uniform(tid >> 6) % NW, group = uniform(tid >> 6) / NW;
  int64_t mt;
  int nt;
  if (!ordered_tile(a.order, blockIdx.x, &mt, &nt)) return;
  const int n0 = nt * TN;
  const Tile t = find_tile<TM>(a, mt);
  if (t.count <= 0) return;
  const uint8_t* We = a.W + static_cast<int64_t>(t.e) * a.n * a.k;
  const uint8_t* zeros = reinterpret_cast<const uint8_t*>(&zero16);
  const int c = (lane & 7) ^ ((4 * wave + lane / 16) & 7);
  const uint8_t* src[LD];
#pragma unroll
  for (int i = 0; i < LD; ++i) {
    const int r = (wave + NW * i) * 8 + lane / 8;
    if (r < TM) {
      const int64_t row = source_row(a, t.p0 + min(r, t.count - 1));
      src[i] = row >= 0 ? a.X + row * a.ldx + 16 * c : nullptr;
    } else {
      src[i] = We + static_cast<int64_t>(min(n0 + r - TM, a.n - 1)) * a.k + 16 * c;
    }
  }
  const unsigned lds0 = static_cast<unsigned>(reinterpret_cast<uintptr_t>(
      (__attribute__((address_space(3))) uint8_t*)lds)) + group * NB * STAGE + wave * 1024;
  const int own = (a.kb - group + KG - 1) / KG;   // this group's stages: blocks group, group + KG, ..
  auto issue = [&](int s) {
    const int k0 = (s * KG + group) * FB;
    const bool in = k0 + 16 * c < a.k;
#pragma unroll
    for (int i = 0; i < LD; ++i)
      copy16(in && src[i] != nullptr ? src[i] + k0 : zeros, lds0 + (s % NB) * STAGE + NW * i * 1024);
  };
  {
    const int64_t row = source_row(a, t.p0 + min(lane, t.count - 1));
    if (tid < TM) lost[tid] = row < 0;
    for (int b = tid / 64; b < a.kb; b += KG * NW) scales[b * TM + lane] = row >= 0 ? load_xs<KIND>(a, row, b) : 0.0f;
    for (int b = tid; b < a.kb; b += KG * 256) scales[a.kb * TM + b] = load_ws<KIND>(a, t.e, n0 / FB, b);
  }
  const int wm = wave / 2, wn = wave % 2;
  const int j = lane & 15, q = lane >> 4;
  const int swz = (j >> 1) & 7;
  const int at0 = j * FB + 16 * (q ^ swz), at1 = j * FB + 16 * ((q + 4) ^ swz);
  const f32x4 zero = {0.0f, 0.0f, 0.0f, 0.0f};
  f32x4 y[2][2] = {{zero, zero}, {zero, zero}};
  // the loads above are done with before the first copy: the loop counts copies alone
  asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
#pragma unroll
  for (int s = 0; s < NB - 1; ++s)
    if (s < own) issue(s);
  for (int s = 0; s < (a.kb + KG - 1) / KG; ++s) {   // the first group's number of stages: the longest
    // this stage's copies are the oldest of those of up to three stages
    if (s + 2 < own) wait_vmcnt<2 * LD>();
    else if (s + 1 < own) wait_vmcnt<LD>();
    else wait_vmcnt<0>();
    __syncthreads();   // everyone's copies have landed, and everyone is done with the stage before
    if (s + NB - 1 < own) issue(s + NB - 1);
    if (s >= own) break;   // behind the last barrier of the loop
    const int b = s * KG + group;
    const uint8_t* xb = lds + (group * NB + s % NB) * STAGE + wm * 32 * FB;
    const uint8_t* wb = lds + (group * NB + s % NB) * STAGE + (TM + wn * 32) * FB;
    auto frag = [&](const uint8_t* p) {
      const i32x4 lo = *reinterpret_cast<const i32x4*>(p + at0);
      const i32x4 hi = *reinterpret_cast<const i32x4*>(p + at1);
      return Operand<KIND>(i32x8{lo[0], lo[1], lo[2], lo[3], hi[0], hi[1], hi[2], hi[3]});
    };
    const Operand<KIND> xf[2] = {frag(xb), frag(xb + 16 * FB)}, wf[2] = {frag(wb), frag(wb + 16 * FB)};
    const float sw = scales[a.kb * TM + b];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const float sx = scales[b * TM + wm * 32 + 16 * i + j];
#pragma unroll
      for (int h = 0; h < 2; ++h) block_mma<KIND>(wf[h], xf[i], sx, sw, y[i][h]);
    }
  }
  if constexpr (KG == 2) {
    // the second group's sums through LDS, in one order: first + second
    f32x4* const part = reinterpret_cast<f32x4*>(lds);
    __syncthreads();
    if (group == 1)
#pragma unroll
      for (int i = 0; i < 2; ++i)
#pragma unroll
        for (int h = 0; h < 2; ++h) part[((wave * 2 + i) * 2 + h) * 64 + lane] = y[i][h];
    __syncthreads();
    if (group == 1) return;
#pragma unroll
    for (int i = 0; i < 2; ++i)
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const f32x4 o = part[((wave * 2 + i) * 2 + h) * 64 + lane];
#pragma unroll
        for (int e = 0; e < 4; ++e) y[i][h][e] += o[e];
      }
  }
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const int r = wm * 32 + 16 * i + j;
    if (r >= t.count) continue;
    const bool none = lost[r];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const f32x4 s = none ? zero : y[i][h];
      const float v[4] = {s[0], s[1], s[2], s[3]};
      store_y(a, t.p0 + r, n0 + wn * 32 + 16 * h + 4 * q, v);
    }
  }
}

template <int KG>
gptq_status launch_mid_groups(const MmArgs& a, unsigned grid, hipStream_t stream) {
  const dim3 g(grid), b(KG * 256);
  const size_t lds = static_cast<size_t>(a.kb) * 65 * sizeof(float);
  if (a.y_dtype == GPTQ_F32) GPTQ_LAUNCH((fp8_mid_kernel<kMmaExact, KG>), g, b, lds, stream, a);
  else if (a.e8) GPTQ_LAUNCH((fp8_mid_kernel<kMmaE8M0, KG>), g, b, lds, stream, a);
  else GPTQ_LAUNCH((fp8_mid_kernel<kMmaF32Scale, KG>), g, b, lds, stream, a);
  return GPTQ_OK;
}

gptq_status launch_mid(MmArgs a, hipStream_t stream) {
  a.order = {(a.n + 63) / 64, tile_rows(a, 64)};
  const int64_t grid = order_grid(a.order);
  if (mid_groups(a.kb, static_cast<double>(grid)) == 2) return launch_mid_groups<2>(a, static_cast<unsigned>(grid), stream);
  return launch_mid_groups<1>(a, static_cast<unsigned>(grid), stream);
}

// Few rows: 16 outputs x 16 FM rows per workgroup, whose WK waves take every WK-th block of
// inputs straight from memory to registers, U blocks in flight per wave; their sums meet in LDS
// and are added in wave order.  (Several groups of 16 outputs per workgroup, with fewer waves
// along the inputs, measured the same or slower.)
// T: 16-bit activations, rounded by every workgroup for itself while its first weights are
// on the way, into LDS (void: 8-bit ones from memory).  That saves a launch: one row of 4096 x
// 14336 takes 12.7 us after a 3.5 us launch that rounds it, and 14.2 us together.
template <int FM, int WK, int KIND, typename T>
__global__ __launch_bounds__(WK * 64) void fp8_rows_kernel(MmArgs a) {
  constexpr int U = FM <= 2 ? 4 : 2, TM = 16 * FM;
  constexpr bool kRaw = !std::is_void_v<T>;
  extern __shared__ __attribute__((aligned(16))) uint8_t raw[];   // kRaw: rows of codes, then [row][block] scales
  __shared__ __attribute__((aligned(16))) float part[WK][TM][16];
  __shared__ bool lost[TM];
  const int tid = threadIdx.x, lane = tid & 63, wk = uniform(tid >> 6);
  const int64_t mt = blockIdx.x / a.tiles_n;
  const int n0 = static_cast<int>(blockIdx.x - mt * a.tiles_n) * 16;
  const Tile t = find_tile<TM>(a, mt);
  if (t.count <= 0) return;
  const int j = lane & 15, q = lane >> 4;
  const uint8_t* zeros = reinterpret_cast<const uint8_t*>(&zero16);
  const uint8_t* w = a.W + (static_cast<int64_t>(t.e) * a.n + min(n0 + j, a.n - 1)) * a.k + 32 * q;
  const uint8_t* x[FM];
  int64_t row[FM];
#pragma unroll
  for (int i = 0; i < FM; ++i) {
    row[i] = source_row(a, t.p0 + min(16 * i + j, t.count - 1));
    x[i] = a.X + row[i] * a.ldx + 32 * q;
    if (tid < 16) lost[16 * i + j] = row[i] < 0;
  }
  i32x4 wl[U], wh[U], xl[U][FM], xh[U][FM];
  float sw[U], sx[U][FM];
  auto load = [&](int u, int b) {
    const int c = FB * b + 32 * q;
    const bool lo = c < a.k, hi = c + 16 < a.k;
    wl[u] = *reinterpret_cast<const i32x4*>(lo ? w + FB * b : zeros);
    wh[u] = *reinterpret_cast<const i32x4*>(hi ? w + FB * b + 16 : zeros);
    sw[u] = load_ws<KIND>(a, t.e, n0 / FB, b);
    if constexpr (!kRaw)
#pragma unroll
    for (int i = 0; i < FM; ++i) {
      xl[u][i] = *reinterpret_cast<const i32x4*>(lo && row[i] >= 0 ? x[i] + FB * b : zeros);
      xh[u][i] = *reinterpret_cast<const i32x4*>(hi && row[i] >= 0 ? x[i] + FB * b + 16 : zeros);
      sx[u][i] = row[i] >= 0 ? load_xs<KIND>(a, row[i], b) : 0.0f;
    }
  };
  const f32x4 zero = {0.0f, 0.0f, 0.0f, 0.0f};
  f32x4 y[FM];
#pragma unroll
  for (int i = 0; i < FM; ++i) y[i] = zero;
#pragma unroll
  for (int u = 0; u < U; ++u)
    if (wk + WK * u < a.kb) load(u, wk + WK * u);
  const int pitch = a.kb * FB + 16;   // rows start 16 bytes apart mod 128
  float* const rs = reinterpret_cast<float*>(raw + (a.off == nullptr ? min(static_cast<int64_t>(TM), a.m) : TM) * pitch);
  if constexpr (kRaw) {
    for (int g = tid / 8; g < min(TM, t.count) * a.kb; g += WK * 8) {
      const int r = g / a.kb, b = g - r * a.kb, col = b * FB + (tid & 7) * 16;
      const int64_t p = source_row(a, t.p0 + r);
      float v[16];
#pragma unroll
      for (int i = 0; i < 16; ++i) v[i] = 0.0f;
      if (p >= 0 && col < a.k)
        load_row<T, 16>(reinterpret_cast<const T*>(a.X) + p * a.ldx + col, v);
      const uint32_t top = eight_lanes_max(top_bits<16>(v));
      const bool e8 = KIND == kMmaE8M0 || (KIND == kMmaExact && a.e8);
      const Scale sc = e8 ? block_scale<true>(top) : block_scale<false>(top);
      uint32_t o[4];
      if (e8) round_values<true, 16>(v, sc, o);
      else round_values<false, 16>(v, sc, o);
      *reinterpret_cast<uint4*>(raw + r * pitch + col) = make_uint4(o[0], o[1], o[2], o[3]);
      if ((tid & 7) == 0) rs[r * a.kb + b] = KIND == kMmaE8M0 ? __int_as_float(sc.code) : sc.s;
    }
    __syncthreads();
  }
  for (int b0 = wk; b0 < a.kb; b0 += WK * U) {
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int b = b0 + WK * u;
      if (b < a.kb) {
        const Operand<KIND> wf(i32x8{wl[u][0], wl[u][1], wl[u][2], wl[u][3], wh[u][0], wh[u][1], wh[u][2], wh[u][3]});
#pragma unroll
        for (int i = 0; i < FM; ++i) {
          if constexpr (kRaw) {
            const int r = min(16 * i + j, t.count - 1);
            const i32x4* p = reinterpret_cast<const i32x4*>(raw + r * pitch + FB * b + 32 * q);
            const i32x4 lo = p[0], hi = p[1];
            const Operand<KIND> xf(i32x8{lo[0], lo[1], lo[2], lo[3], hi[0], hi[1], hi[2], hi[3]});
            block_mma<KIND>(wf, xf, rs[r * a.kb + b], sw[u], y[i]);
          } else {
            const Operand<KIND> xf(i32x8{xl[u][i][0], xl[u][i][1], xl[u][i][2], xl[u][i][3], xh[u][i][0], xh[u][i][1],
                                         xh[u][i][2], xh[u][i][3]});
            block_mma<KIND>(wf, xf, sx[u][i], sw[u], y[i]);
          }
        }
        if (b + WK * U < a.kb) load(u, b + WK * U);
      }
    }
  }
#pragma unroll
  for (int i = 0; i < FM; ++i) *reinterpret_cast<f32x4*>(&part[wk][16 * i + j][4 * q]) = y[i];
  __syncthreads();
  for (int g = tid; g < min(TM, t.count) * 4; g += WK * 64) {
    const int c = g & 3, r = g >> 2;
    f32x4 v = zero;
#pragma unroll
    for (int h = 0; h < WK; ++h) {
      const f32x4 o = *reinterpret_cast<const f32x4*>(&part[h][r][4 * c]);
#pragma unroll
      for (int e = 0; e < 4; ++e) v[e] += o[e];
    }
    if (lost[r]) v = zero;
    const float f[4] = {v[0], v[1], v[2], v[3]};
    store_y(a, t.p0 + r, n0 + 4 * c, f);
  }
}

// LDS of a tile's 16-bit rows, rounded: of the rows that it can hold.
size_t raw_lds(const MmArgs& a, int tm) {
  const size_t rows = a.off == nullptr ? std::min<int64_t>(tm, a.m) : tm;
  return rows * (static_cast<size_t>(a.kb) * FB + 16 + a.kb * sizeof(float));
}

template <int FM, int WK, typename T>
gptq_status launch_rows(MmArgs a, hipStream_t stream) {
  constexpr int TM = 16 * FM;
  a.tiles_n = (a.n + 15) / 16;
  const dim3 g(static_cast<unsigned>(tile_rows(a, TM) * a.tiles_n)), b(WK * 64);
  const size_t lds = std::is_void_v<T> ? 0 : raw_lds(a, TM);
  if (a.y_dtype == GPTQ_F32) GPTQ_LAUNCH((fp8_rows_kernel<FM, WK, kMmaExact, T>), g, b, lds, stream, a);
  else if (a.e8) GPTQ_LAUNCH((fp8_rows_kernel<FM, WK, kMmaE8M0, T>), g, b, lds, stream, a);
  else GPTQ_LAUNCH((fp8_rows_kernel<FM, WK, kMmaF32Scale, T>), g, b, lds, stream, a);
  return GPTQ_OK;
}

// Which kernel: the least of four estimates in microseconds.  Their constants are device times
// of the kernels on one MI355X, per stage of 128 inputs and round of workgroups:
//   rows  2.5 + bytes through the L2s at 7 TB/s, every 16 outputs reading all of X again
//         (4096 x 14336: 11.9 us at 1 row, 18.3 at 16, 27.7 at 32, 45.8 at 64)
//   mid   64 x 64, 0.29 us with two groups of waves; with one 0.46 us, two workgroups per CU 0.57
//         (4096 x 14336: 32 us at 64 rows, rows 46; 35 at 256, tile 131; 14336 x 4096 at 64: 14)
//   tile  128 x 128, one workgroup per CU 1.17 us, two 1.5
//         (4096 x 4096: 42 us at 1024 rows, mid 44, big 48)
//   big   256 x 256, a round 1.4 us on up to half of the CUs, else 1.85
//         (4096 x 4096: 48 us at 2048 rows, tile 54; 67 at 4096, tile 100; 49152 rows of 64
//         experts: 195 to 200, tile 280 to 298)
// Grouped problems have about half a tile more per expert, and every kernel needs the time to
// read the weights once (5 TB/s).  The large tiles are not built for fp32 Y (their operands would
// not fit the registers) and address a tile's rows by 32-bit offsets.
enum Product { kRows, kMid, kTile, kBig };
Product choose_product(const MmArgs& a) {
  const bool grouped = a.off != nullptr;
  const double used = grouped ? static_cast<double>(std::min<int64_t>(a.experts, a.m)) : 1.0;
  const double weights = static_cast<double>(a.n) * a.k;
  auto tiles = [&](int tm, int tn) {
    const double rows = grouped ? static_cast<double>(a.m) / tm + 0.5 * used : static_cast<double>((a.m + tm - 1) / tm);
    return rows * ((a.n + tn - 1) / tn);
  };
  auto rounds = [](double t, double slots, double half, double full) {   // time of t workgroups
    const double r = static_cast<double>(static_cast<int64_t>(t / slots)), rest = t - r * slots;
    return r * full + (rest <= 0.0 ? 0.0 : rest <= slots / 2 ? half : full);
  };
  const double read = 0.7 * used * weights / 5e6;
  const double row_tiles = grouped ? static_cast<double>(a.m) / 16 + 0.5 * used : 1.0;
  const double t_rows = a.m > 64 && !grouped ? 1e30
                        : 2.5 + std::max(read, (row_tiles * weights + static_cast<double>(a.m) * a.k * a.n / 16) / 7e6);
  const double mid = tiles(64, 64);
  const double t_mid = a.kb > MID_KB[1] ? 1e30
                       : 3 + std::max(read, a.kb * (mid_groups(a.kb, mid) == 2 ? rounds(mid, 256, 0.29, 0.29)
                                                    : a.kb <= MID_PAIR         ? rounds(mid, 512, 0.46, 0.57)
                                                                               : rounds(mid, 256, 0.47, 0.47)));
  const double t_tile = 3 + std::max(read, a.kb * rounds(tiles(128, 128), 512, 1.17, 1.5));
  const int64_t span = a.rows == nullptr ? 256 * a.ldx : a.x_rows * a.ldx;
  const bool narrow = span <= INT32_MAX && 256 * static_cast<int64_t>(a.k) <= INT32_MAX;
  const double t_big = a.y_dtype == GPTQ_F32 || !narrow || a.x_rows == 0 || a.kb > BIG_KB
                           ? 1e30
                           : 6 + std::max(read, a.kb * rounds(tiles(256, 256), 256, 1.4, 1.85));
  const double best = std::min(std::min(t_rows, t_mid), std::min(t_tile, t_big));
  if (best == t_mid) return kMid;   // the smallest tile of those that wait for the weights
  return best == t_tile ? kTile : best == t_big ? kBig : kRows;
}

// Rows of fp8_rows_kernel's tiles: 16 for grouped rows.
int rows_tile(const MmArgs& a) { return a.off != nullptr || a.m <= 16 ? 16 : a.m <= 32 ? 32 : 64; }

// Whether the launch is one the kernels number their tiles for (asked before anything is enqueued).
bool launchable(const MmArgs& a, Product kind) {
  const int tm = kind == kBig ? 256 : kind == kTile ? 128 : kind == kMid ? 64 : rows_tile(a);
  const int tn = kind == kRows ? 16 : tm;
  return tile_rows(a, tm) <= (1 << 22) / ((a.n + tn - 1) / tn);
}

gptq_status launch_product(const MmArgs& a, Product kind, hipStream_t stream) {
  if (kind == kMid) return launch_mid(a, stream);
  if (kind == kTile) return launch_tile<128, 128, 2, 2>(a, stream);
  if (kind == kBig) return launch_big(a, stream);
  // 8 waves along the inputs while each has 3 blocks or more
  // (4096 x 4096 at 1 row: 5.5 us with 8, 6.5 with 4; 64 experts of 1408 x 2048, 96 rows: 35 and 24)
  if (rows_tile(a) == 64) return launch_rows<4, 8, void>(a, stream);
  if (rows_tile(a) == 32) return launch_rows<2, 8, void>(a, stream);
  return a.kb >= 24 ? launch_rows<1, 8, void>(a, stream) : launch_rows<1, 4, void>(a, stream);
}

// 16-bit rows straight into the kernel for few rows, where the workgroups' repeated rounding stays
// small: at most 32 values a thread, 4 M over the launch
// (4096 x 14336 at 1 row: 14.2 us, against 3.5 + 12.7 in two launches; 4096 x 4096 at 8 rows: 11.5
// against 3.6 + 6.6; 96 rows of 64 experts of 1408 x 2048: 29.4 against 3.9 + 23.8), and 16 rows
// of a group fit 48 KB, which leaves three workgroups on a CU.
bool rounds_itself(const MmArgs& a) {
  if (a.m * a.k > (1 << 22)) return false;
  if (a.m * a.k * ((a.n + 15) / 16) > (1 << 22)) return false;
  if (a.off != nullptr) return a.m <= 2 * static_cast<int64_t>(a.experts) && raw_lds(a, 16) <= 48 * 1024;
  return a.m <= 16 && a.m * a.k <= 16384;
}
template <typename T>
gptq_status launch_raw(const MmArgs& a, hipStream_t stream) {
  return a.kb >= 24 ? launch_rows<1, 8, T>(a, stream) : launch_rows<1, 4, T>(a, stream);
}

struct Fp8Layout {
  size_t q, s, total;
};
Fp8Layout fp8_layout(int64_t rows, int k) {
  const size_t kb = (static_cast<size_t>(k) + FB - 1) / FB;
  Fp8Layout l{};
  l.s = align_up(static_cast<size_t>(rows) * k, 256);
  l.total = std::max<size_t>(256, l.s + align_up(static_cast<size_t>(rows) * kb * 4, 256));
  return l;
}

}  // namespace

size_t fp8_workspace(int64_t x_rows, int k) { return fp8_layout(x_rows, k).total; }

gptq_status fp8_quantize_enqueue(int batch, int64_t rows, int cols, gptq_dtype x_dtype, const void* X, int64_t ldx,
                                 int64_t bsx, int block_rows, bool e8, uint8_t* Q, void* S, int64_t lsr, int64_t lsb,
                                 int64_t bss, hipStream_t stream) {
  const QuantArgs a{rows, cols, X, ldx, bsx, Q, S, lsr, lsb, bss};
  if (x_dtype == GPTQ_F32) return launch_quant_t<float>(a, batch, block_rows, e8, stream);
  if (x_dtype == GPTQ_BF16) return launch_quant_t<BF16>(a, batch, block_rows, e8, stream);
  return launch_quant_t<F16>(a, batch, block_rows, e8, stream);
}

gptq_status fp8_matmul_enqueue(const Fp8Problem& p, hipStream_t stream) {
  MmArgs a{};
  a.m = p.n_rows; a.n = p.n; a.k = p.k; a.kb = (p.k + FB - 1) / FB; a.nb = (p.n + FB - 1) / FB;
  a.x_rows = p.x_rows; a.W = p.W; a.ws = p.ws; a.Y = p.Y; a.ldy = p.ldy; a.y_dtype = p.y_dtype; a.e8 = p.e8;
  a.off = p.offsets; a.rows = p.row_index; a.experts = p.batch;
  if (a.off != nullptr && (a.m / 16 + 1) * a.experts > INT32_MAX) return GPTQ_ERR_UNSUPPORTED;
  a.X = static_cast<const uint8_t*>(p.X);
  a.ldx = p.ldx; a.xs = p.xs; a.xsr = p.xsr; a.xsb = p.xsb;
  if (p.x_dtype == GPTQ_E4M3) {
    const Product kind = choose_product(a);
    return launchable(a, kind) ? launch_product(a, kind, stream) : GPTQ_ERR_UNSUPPORTED;
  }
  const Fp8Layout l = fp8_layout(p.x_rows, p.k);
  if (p.x_rows > 0 && (p.workspace == nullptr || p.workspace_bytes < l.total)) return GPTQ_ERR_WORKSPACE;
  a.ldx = p.k;   // as the product will read them
  const Product kind = choose_product(a);
  if (!launchable(a, kind)) return GPTQ_ERR_UNSUPPORTED;
  if (kind == kRows && rounds_itself(a)) {
    a.ldx = p.ldx;
    return p.x_dtype == GPTQ_BF16 ? launch_raw<BF16>(a, stream) : launch_raw<F16>(a, stream);
  }
  uint8_t* ws = static_cast<uint8_t*>(p.workspace);
  if (p.x_rows > 0) {
    const gptq_status st = fp8_quantize_enqueue(1, p.x_rows, p.k, p.x_dtype, p.X, p.ldx, 0, 1, p.e8, ws, ws + l.s, 1,
                                                p.x_rows, 0, stream);
    if (st != GPTQ_OK) return st;
  }
  a.X = ws; a.xs = ws + l.s; a.xsr = 1; a.xsb = p.x_rows;
  return launch_product(a, kind, stream);
}

}  // namespace gptq
