// Linear layers in the 4-bit microscaled form on gfx950: rounding to e2m1 with a power-of-two scale
// per 32 inputs, the values back, and products with such weights, dense or grouped by expert.
//
//   scale_b = 2^(floor(log2 max |x|) - 2) or 2^ceil(log2(max |x| / 6)),  q = rne_e2m1(x / scale_b)
//   Y[r, o] = sum_b xs[r, b] ws[o, b] sum_{c in b} xq[r, c] q[o, c]      4-bit activations
//   Y[r, o] = sum_b ws[o, b] sum_{c in b} X[r, c] q[o, c]                16-bit ones, not rounded
//
// 4-bit activations: v_mfma_scale_f32_16x16x128_f8f6f4, whose operands' four groups of 16 lanes hold
// one block of 32 inputs each with its own scale.  Products of codes are whole multiples of 1/4 below
// 2^6 and their sums within a block are exact; with scales apart by up to 2^40 a result is within
// 2^-23.3 of sum |x q| (by experiment): fp32 sums, for every type of Y.
// 16-bit activations: the weights become bf16 in registers, exactly, in front of
// v_mfma_f32_16x16x32_bf16 with fp32 sums.
// Weights are the first operand and activations the second: a lane then holds one activation row
// and 4 consecutive outputs, which are stored together.
#include <algorithm>

#include "mx.h"

namespace gptq {
namespace {

// ---------------------------------------------------------------------------- rounding

struct MxQuantArgs {
  int64_t rows;
  int cols, kb;
  const void* X;
  int64_t ldx, bsx;
  uint8_t* Q;
  uint8_t* S;
  int shift;   // 2^shift blocks of a row per workgroup
};

// The scale's E8M0 code for a block whose largest magnitude has these bits (255: an infinity or a
// NaN).
template <bool CEIL>
__device__ __forceinline__ uint32_t mx_scale(uint32_t top) {
  if (top >= 0x7F800000u) return 255;
  const int e = static_cast<int>(top >> 23) - 2 + (CEIL && (top & 0x7FFFFFu) > 0x400000u);   // 6 = 1.5 * 2^2
  return static_cast<uint32_t>(max(e, 1));
}

// Four lanes per block, 8 values each; a workgroup takes 2^shift blocks of 64 >> shift rows.  The
// conversion rounds x / scale to nearest even and cuts at 6 (by experiment at all ties, also where
// the scale is 2^-126 and x subnormal).  Bound by memory.
template <typename T, bool CEIL>
__global__ __launch_bounds__(256) void mx_quant_kernel(MxQuantArgs a) {
  const int u = threadIdx.x >> 2, part = threadIdx.x & 3;
  const int b = (blockIdx.y << a.shift) + (u & ((1 << a.shift) - 1));
  const int64_t row = static_cast<int64_t>(blockIdx.x) * (64 >> a.shift) + (u >> a.shift);
  if (row >= a.rows || b >= a.kb) return;   // all four lanes of a block
  const int col = b * MXB + part * 8;
  float x[8];
  load_row<T, 8>(static_cast<const T*>(a.X) + blockIdx.z * a.bsx + row * a.ldx + col, x);
  uint32_t top = top_bits<8>(x);
  top = max(top, static_cast<uint32_t>(__shfl_xor(static_cast<int>(top), 1)));
  top = max(top, static_cast<uint32_t>(__shfl_xor(static_cast<int>(top), 2)));
  const uint32_t code = mx_scale<CEIL>(top);
  const float s = __uint_as_float(code << 23);
  uint32_t w = 0;
  w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, x[0], x[1], s, 0);
  w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, x[2], x[3], s, 1);
  w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, x[4], x[5], s, 2);
  w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, x[6], x[7], s, 3);
  if (code == 255) w = 0;
  const int64_t at = blockIdx.z * a.rows + row;
  *reinterpret_cast<uint32_t*>(a.Q + at * (a.cols / 2) + col / 2) = w;
  if (part == 0) a.S[at * a.kb + b] = static_cast<uint8_t>(code);
}

struct MxDequantArgs {
  int64_t rows;
  int cols, kb;
  const uint8_t* Q;
  const uint8_t* S;
  void* Y;
  int shift;
};

// The values back, split like the rounding.  Bound by memory.
template <typename T>
__global__ __launch_bounds__(256) void mx_dequant_kernel(MxDequantArgs a) {
  const int u = threadIdx.x >> 2, part = threadIdx.x & 3;
  const int b = (blockIdx.y << a.shift) + (u & ((1 << a.shift) - 1));
  const int64_t row = static_cast<int64_t>(blockIdx.x) * (64 >> a.shift) + (u >> a.shift);
  if (row >= a.rows || b >= a.kb) return;
  const int col = b * MXB + part * 8;
  const uint32_t w = *reinterpret_cast<const uint32_t*>(a.Q + row * (a.cols / 2) + col / 2);
  const float s = __uint_as_float(static_cast<uint32_t>(a.S[row * a.kb + b]) << 23);
  const f32x2 v[4] = {__builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w, s, 0), __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w, s, 1),
                      __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w, s, 2), __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w, s, 3)};
  Vec<T, 8> o;
#pragma unroll
  for (int i = 0; i < 8; ++i) o.v[i] = from_f32<T>(v[i / 2][i & 1]);
  __builtin_memcpy(static_cast<T*>(a.Y) + row * a.cols + col, &o, sizeof(o));
}

// Blocks of a row per workgroup, as a shift: the power of two that holds them, at most 64.
int block_shift(int kb) {
  int s = 0;
  while (s < 6 && (1 << s) < kb) ++s;
  return s;
}
// Grid of the two kernels above; false where it is too large.
bool block_grid(int64_t rows, int kb, int batch, int shift, dim3* grid) {
  const int64_t gx = (rows + (64 >> shift) - 1) / (64 >> shift), gy = (kb + (1 << shift) - 1) >> shift;
  if (gx > (1 << 24) - 1 || gy > 65535 || batch > 65535) return false;
  *grid = dim3(static_cast<unsigned>(gx), static_cast<unsigned>(gy), static_cast<unsigned>(batch));
  return true;
}

template <typename T>
gptq_status launch_mx_quant(const MxQuantArgs& a, dim3 grid, bool ceil, hipStream_t stream) {
  if (ceil) GPTQ_LAUNCH((mx_quant_kernel<T, true>), grid, dim3(256), 0, stream, a);
  else GPTQ_LAUNCH((mx_quant_kernel<T, false>), grid, dim3(256), 0, stream, a);
  return GPTQ_OK;
}

// ---------------------------------------------------------------------------- product

// MmArgs as these kernels read it: ldx in bytes, k / 2 bytes a row of W, kb blocks of 32, xs and ws
// E8M0 codes (those of a row one after another).
struct MxArgs : MmArgs {
  int stages;     // of the LDS kernels
  int splits, per;   // parts of the inputs, and their stages
  float* part;       // [splits][m][n] sums, where there is more than one
};

// Few rows: 16 outputs x 16 FM rows per workgroup, whose WK waves take every WK-th pair of chunks of
// 128 inputs straight from memory to registers (a block of 32 per lane and chunk), U chunks in
// flight per wave; their sums meet in LDS and are added in wave order.
template <int FM, int WK, int KIND>
__global__ __launch_bounds__(WK * 64) void mx_rows_kernel(MxArgs a) {
  constexpr int U = FM == 1 ? 4 : 2, TM = 16 * FM, XR = KIND == kMx4 ? 1 : 4;   // 16-byte pieces of X a block
  __shared__ __attribute__((aligned(16))) float part[WK][TM][16];
  __shared__ bool lost[TM];
  const int tid = threadIdx.x, lane = tid & 63, wk = uniform(tid >> 6);
  const int64_t mt = blockIdx.x / a.tiles_n;
  const int n0 = static_cast<int>(blockIdx.x - mt * a.tiles_n) * 16;
  const Tile t = find_tile<TM>(a, mt);
  if (t.count <= 0) return;
  const int j = lane & 15, q = lane >> 4;
  const uint8_t* zeros = reinterpret_cast<const uint8_t*>(&zero16);
  const int64_t wrow = static_cast<int64_t>(t.e) * a.n + min(n0 + j, a.n - 1);
  const uint8_t* w = a.W + wrow * (a.k / 2);
  const uint8_t* ws = static_cast<const uint8_t*>(a.ws) + wrow * a.kb;
  const uint8_t* x[FM];
  const uint8_t* xs[FM];
  bool have[FM];
#pragma unroll
  for (int i = 0; i < FM; ++i) {
    const int64_t row = source_row(a, t.p0 + min(16 * i + j, t.count - 1));
    if (tid < 16) lost[16 * i + j] = row < 0;
    have[i] = row >= 0 && 16 * i + j < t.count;
    x[i] = a.X + max(row, static_cast<int64_t>(0)) * a.ldx;
    if constexpr (KIND == kMx4) xs[i] = static_cast<const uint8_t*>(a.xs) + max(row, static_cast<int64_t>(0)) * a.xsr;
  }
  const int chunks = (a.kb + 3) / 4;
  i32x4 wv[U], xv[U][FM][XR];
  uint32_t sw[U], sx[U][FM];
  auto load = [&](int u, int c) {
    const int b = 4 * c + q;
    const bool in = b < a.kb;
    wv[u] = *reinterpret_cast<const i32x4*>(in ? w + 16 * b : zeros);
    sw[u] = in ? ws[b] : 127u;
#pragma unroll
    for (int i = 0; i < FM; ++i) {
      const bool ok = in && have[i];
#pragma unroll
      for (int p = 0; p < XR; ++p) xv[u][i][p] = i32x4{0, 0, 0, 0};
      if (ok)
#pragma unroll
        for (int p = 0; p < XR; ++p) __builtin_memcpy(&xv[u][i][p], x[i] + 16 * XR * b + 16 * p, 16);
      if constexpr (KIND == kMx4) sx[u][i] = ok ? xs[i][b] : 127u;
    }
  };
  auto chunk = [&](int g, int u) { return 2 * (wk + WK * (g + u / 2)) + (u & 1); };
  f32x4 y[FM];
#pragma unroll
  for (int i = 0; i < FM; ++i) y[i] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
  for (int u = 0; u < U; ++u)
    if (chunk(0, u) < chunks) load(u, chunk(0, u));
  for (int g = 0; chunk(g, 0) < chunks; g += U / 2) {
#pragma unroll
    for (int u = 0; u < U; ++u) {
      if (chunk(g, u) < chunks) {
        if constexpr (KIND == kMx4) {
#pragma unroll
          for (int i = 0; i < FM; ++i)
            y[i] = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(widen(wv[u]), widen(xv[u][i][0]), y[i], 4, 4, 0,
                                                                    static_cast<int>(sw[u]), 0, static_cast<int>(sx[u][i]));
        } else {
#pragma unroll
          for (int p = 0; p < 4; ++p) {
            const bf16x8 wf = mx_bf16(static_cast<uint32_t>(wv[u][p]), sw[u]);
#pragma unroll
            for (int i = 0; i < FM; ++i) y[i] = mx_mma16<KIND>(wf, XValues<KIND>(xv[u][i][p]), y[i]);
          }
        }
        if (chunk(g + U / 2, u) < chunks) load(u, chunk(g + U / 2, u));
      }
    }
  }
#pragma unroll
  for (int i = 0; i < FM; ++i) *reinterpret_cast<f32x4*>(&part[wk][16 * i + j][4 * q]) = y[i];
  __syncthreads();
  for (int g = tid; g < min(TM, t.count) * 4; g += WK * 64) {
    const int c = g & 3, r = g >> 2;
    f32x4 v = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
    for (int h = 0; h < WK; ++h) {
      const f32x4 o = *reinterpret_cast<const f32x4*>(&part[h][r][4 * c]);
#pragma unroll
      for (int e = 0; e < 4; ++e) v[e] += o[e];
    }
    const bool none = lost[r];
    const float f[4] = {none ? 0.0f : v[0], none ? 0.0f : v[1], none ? 0.0f : v[2], none ? 0.0f : v[3]};
    store_y(a, t.p0 + r, n0 + 4 * c, f);
  }
}

// The LDS kernels' stage is 128 bytes of every row of X: 256 inputs of 4-bit rows, 64 of 16-bit
// ones, whose weights are 32 bytes a row.  Two instructions each use one half: with 4 bits the 16-byte
// pieces q and q + 4 of a row are the lane's blocks of the first and the second, and with 16 bits
// its 8 inputs of the stage's first and second block.
constexpr int ROW = 128;   // bytes of a row of X a stage
template <int KIND>
struct MxStage {
  static constexpr int WBYTES = KIND == kMx4 ? 128 : 32;   // bytes of a row of W
  static constexpr int BLOCKS = KIND == kMx4 ? 8 : 2;      // scales of a row
};

// A lane's operands of a stage: 16 outputs' weights and 16 rows' activations.
template <int KIND>
struct MxW {
  bf16x8 v[2];
};
template <>
struct MxW<kMx4> {
  i32x4 v[2];
  int s;   // the scales of both halves in its two low bytes
};
template <int KIND>
struct MxX {
  XValues<KIND> v[2];
};
template <>
struct MxX<kMx4> {
  i32x4 v[2];
  int s;
};
template <int KIND>
__device__ __forceinline__ void mx_mma(const MxW<KIND>& w, const MxX<KIND>& x, f32x4& acc) {
  if constexpr (KIND == kMx4) {
    acc = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(widen(w.v[0]), widen(x.v[0]), acc, 4, 4, 0, w.s, 0, x.s);
    acc = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(widen(w.v[1]), widen(x.v[1]), acc, 4, 4, 1, w.s, 1, x.s);
  } else {
    acc = mx_mma16<KIND>(w.v[0], x.v[0], acc);
    acc = mx_mma16<KIND>(w.v[1], x.v[1], acc);
  }
}

// The scale codes of stage s of a row (those behind the last block count as 1), 4-bit operands' in
// the order 0 4 1 5 2 6 3 7, so that a lane's two are neighbours.
template <int KIND>
__device__ __forceinline__ uint2 stage_scales(const uint8_t* row, int s, int kb) {
  constexpr int N = MxStage<KIND>::BLOCKS;
  uint8_t b[8];
  if (N * (s + 1) <= kb) {
    __builtin_memcpy(b, row + N * s, N);
  } else {
#pragma unroll
    for (int i = 0; i < N; ++i) b[i] = N * s + i < kb ? row[N * s + i] : 127;
  }
  if constexpr (KIND == kMx4) {
    uint2 v;
    __builtin_memcpy(&v, b, 8);
    return make_uint2(__builtin_amdgcn_perm(v.y, v.x, 0x05010400u), __builtin_amdgcn_perm(v.y, v.x, 0x07030602u));
  } else {
    return make_uint2(b[0] | static_cast<uint32_t>(b[1]) << 8, 0);
  }
}

// Tiles of TM rows x TN outputs, 2 x 2 waves, two buffers, the next stage's copies in flight during
// this one's products.  The 16-byte piece c of a row r of 128 bytes lies at c ^ (r / 2 % 8), so that
// 16 lanes reading the same piece of 16 rows cover all 64 banks.  gridDim.y parts of the inputs:
// few tiles would leave most of the chip idle (sums of parts are added by mx_sum_kernel).
template <int TM, int TN, int KIND>
__global__ __launch_bounds__(256) void mx_tile_kernel(MxArgs a) {
  constexpr int NW = 4, FM = TM / 32, FN = TN / 32;
  constexpr int WB = MxStage<KIND>::WBYTES, STAGE = TM * ROW + TN * WB;
  constexpr int LX = TM / 8 / NW, WC = TN * WB / 1024, LW = (WC + NW - 1) / NW;   // copies of 1 KB: per wave, in all, per wave
  constexpr int SROWS = KIND == kMx4 ? TM + TN : TN;
  static_assert(SROWS <= 256 && TM <= 256 && TM % 32 == 0 && TN % 32 == 0, "tile shape");
  __shared__ __attribute__((aligned(128))) uint8_t lds[2 * STAGE];
  __shared__ uint2 scales[2][SROWS];
  __shared__ bool lost[TM];
  const int tid = threadIdx.x, lane = tid & 63, wave = uniform(tid >> 6);
  int64_t mt;
  int nt;
  if (!ordered_tile(a.order, blockIdx.x, &mt, &nt)) return;
  const int n0 = nt * TN;
  const Tile t = find_tile<TM>(a, mt);
  if (t.count <= 0) return;
  const int first = blockIdx.y * a.per, end = min(first + a.per, a.stages);
  const uint8_t* We = a.W + static_cast<int64_t>(t.e) * a.n * (a.k / 2);
  const uint8_t* zeros = reinterpret_cast<const uint8_t*>(&zero16);
  const int64_t xbytes = KIND == kMx4 ? a.k / 2 : 2 * static_cast<int64_t>(a.k);

  const int c = (lane & 7) ^ ((4 * wave + lane / 16) & 7);   // this lane's piece of a 128-byte row: the same in every copy
  const uint8_t* xsrc[LX];
#pragma unroll
  for (int i = 0; i < LX; ++i) {
    const int64_t row = source_row(a, t.p0 + min((wave + NW * i) * 8 + lane / 8, t.count - 1));
    xsrc[i] = row >= 0 ? a.X + row * a.ldx + 16 * c : nullptr;
  }
  const uint8_t* wsrc[LW];
  const int wc = KIND == kMx4 ? c : lane & 1;
#pragma unroll
  for (int i = 0; i < LW; ++i) {
    const int r = KIND == kMx4 ? (wave + NW * i) * 8 + lane / 8 : (wave + NW * i) * 32 + lane / 2;
    wsrc[i] = We + static_cast<int64_t>(min(n0 + r, a.n - 1)) * (a.k / 2) + 16 * wc;
  }
  if (tid < TM) lost[tid] = source_row(a, t.p0 + min(tid, t.count - 1)) < 0;
  const uint8_t* srow = nullptr;   // this thread's row of scales; null: no such row
  if (tid < SROWS) {
    const int o = KIND == kMx4 ? tid - TM : tid;
    if (o >= 0) {
      srow = static_cast<const uint8_t*>(a.ws) + (static_cast<int64_t>(t.e) * a.n + min(n0 + o, a.n - 1)) * a.kb;
    } else {
      const int64_t row = source_row(a, t.p0 + min(tid, t.count - 1));
      if (row >= 0) srow = static_cast<const uint8_t*>(a.xs) + row * a.xsr;
    }
  }
  uint2 s_next = make_uint2(0x7F7F7F7Fu, 0x7F7F7F7Fu);
  const unsigned lds0 = static_cast<unsigned>(reinterpret_cast<uintptr_t>(
      (__attribute__((address_space(3))) uint8_t*)lds));
  auto issue = [&](int s) {
    if (srow != nullptr) s_next = stage_scales<KIND>(srow, s, a.kb);
    const unsigned to = lds0 + (s & 1) * STAGE;
    const bool xin = static_cast<int64_t>(s) * ROW + 16 * c < xbytes, win = s * WB + 16 * wc < a.k / 2;
#pragma unroll
    for (int i = 0; i < LX; ++i)
      copy16(xin && xsrc[i] != nullptr ? xsrc[i] + static_cast<int64_t>(s) * ROW : zeros, to + (wave + NW * i) * 1024);
#pragma unroll
    for (int i = 0; i < LW; ++i)
      if (wave + NW * i < WC) copy16(win ? wsrc[i] + s * WB : zeros, to + TM * ROW + (wave + NW * i) * 1024);
  };

  const int wm = wave / 2, wn = wave % 2;
  const int j = lane & 15, q = lane >> 4;
  const int swz = (j >> 1) & 7;
  const int at0 = j * ROW + 16 * (q ^ swz), at1 = j * ROW + 16 * ((q + 4) ^ swz);
  f32x4 y[FM][FN];
#pragma unroll
  for (int i = 0; i < FM; ++i)
#pragma unroll
    for (int h = 0; h < FN; ++h) y[i][h] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
  if (first < end) issue(first);
  for (int s = first; s < end; ++s) {
    wait_copies();
    if (tid < SROWS) scales[s & 1][tid] = s_next;
    __syncthreads();
    if (s + 1 < end) issue(s + 1);
    const uint8_t* xb = lds + (s & 1) * STAGE + wm * (TM / 2) * ROW;
    const uint8_t* wb = lds + (s & 1) * STAGE + TM * ROW + wn * (TN / 2) * WB;
    MxW<KIND> wf[FN];
#pragma unroll
    for (int h = 0; h < FN; ++h) {
      const int o = wn * (TN / 2) + 16 * h + j;
      if constexpr (KIND == kMx4) {
        wf[h].v[0] = *reinterpret_cast<const i32x4*>(wb + 16 * h * ROW + at0);
        wf[h].v[1] = *reinterpret_cast<const i32x4*>(wb + 16 * h * ROW + at1);
        wf[h].s = reinterpret_cast<const uint16_t*>(&scales[s & 1][TM + o])[q];
      } else {
        const uint32_t* p = reinterpret_cast<const uint32_t*>(wb + (16 * h + j) * WB) + q;
        const uint32_t sc = scales[s & 1][o].x;
        wf[h].v[0] = mx_bf16(p[0], sc & 255);
        wf[h].v[1] = mx_bf16(p[4], sc >> 8);
      }
    }
#pragma unroll
    for (int i = 0; i < FM; ++i) {
      const i32x4 lo = *reinterpret_cast<const i32x4*>(xb + 16 * i * ROW + at0);
      const i32x4 hi = *reinterpret_cast<const i32x4*>(xb + 16 * i * ROW + at1);
      MxX<KIND> xf;
      if constexpr (KIND == kMx4) {
        xf.v[0] = lo;
        xf.v[1] = hi;
        xf.s = reinterpret_cast<const uint16_t*>(&scales[s & 1][wm * (TM / 2) + 16 * i + j])[q];
      } else {
        xf.v[0] = XValues<KIND>(lo);
        xf.v[1] = XValues<KIND>(hi);
      }
#pragma unroll
      for (int h = 0; h < FN; ++h) mx_mma<KIND>(wf[h], xf, y[i][h]);
    }
  }
  MxArgs out = a;
  if (a.splits > 1) {
    out.Y = a.part + static_cast<int64_t>(blockIdx.y) * a.m * a.n;
    out.ldy = a.n;
    out.y_dtype = GPTQ_F32;
  }
#pragma unroll
  for (int i = 0; i < FM; ++i) {
    const int r = wm * (TM / 2) + 16 * i + j;
    if (r >= t.count) continue;
    const bool none = lost[r];
#pragma unroll
    for (int h = 0; h < FN; ++h) {
      const f32x4 s = y[i][h];
      const float v[4] = {none ? 0.0f : s[0], none ? 0.0f : s[1], none ? 0.0f : s[2], none ? 0.0f : s[3]};
      store_y(out, t.p0 + r, n0 + wn * (TN / 2) + 16 * h + 4 * q, v);
    }
  }
}

// Y from the sums of the parts, in their order, all loads at once.
template <int SPLITS>
__global__ __launch_bounds__(256) void mx_sum_kernel(MxArgs a) {
  const int row = blockIdx.y, o = (blockIdx.x * 256 + threadIdx.x) * 4, n = min(4, a.n - o);
  if (n <= 0) return;
  const float* p = a.part + static_cast<int64_t>(row) * a.n + o;
  f32x4 u[SPLITS];
#pragma unroll
  for (int z = 0; z < SPLITS; ++z, p += a.m * a.n) {
    u[z] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
    if (n == 4) __builtin_memcpy(&u[z], p, 16);
    else
      for (int i = 0; i < n; ++i) u[z][i] = p[i];
  }
#pragma unroll
  for (int z = 1; z < SPLITS; ++z) u[0] += u[z];
  const float v[4] = {u[0][0], u[0][1], u[0][2], u[0][3]};
  store_y(a, row, o, v);
}

// ---------------------------------------------------------------------------- host side

enum MxProduct { kMxRows, kMxTile64, kMxTile128 };
struct MxPlan {
  MxProduct kind;
  int splits;
};

int stage_blocks(int kind) { return kind == kMx4 ? MxStage<kMx4>::BLOCKS : MxStage<kMxBf16>::BLOCKS; }

// Rows of a tile of the kernel for few rows: 16 for grouped rows.
int mx_rows_tile(int64_t m, bool grouped) { return grouped || m <= 16 ? 16 : m <= 32 ? 32 : 64; }

// Which kernel, by sizes alone (the workspace's size goes by the same rule).
MxPlan mx_plan(int64_t m, int n, int k, int kind, bool grouped, int experts) {
  const double used = grouped ? static_cast<double>(std::min<int64_t>(experts, m)) : 1.0;
  const double rows = static_cast<double>(m) / used;
  if (rows <= 16) return {kMxRows, 1};
  auto tiles = [&](int t) {
    const double r = grouped ? static_cast<double>(m) / t + 0.5 * used : static_cast<double>((m + t - 1) / t);
    return r * ((n + t - 1) / t);
  };
  const int stages = (k / MXB + stage_blocks(kind) - 1) / stage_blocks(kind);
  if (tiles(128) >= 384) return {kMxTile128, 1};
  int splits = 1;
  if (!grouped) {
    while (splits < 8 && tiles(64) * splits < 384 && stages / (2 * splits) >= 8) splits *= 2;
    while (splits > 1 && static_cast<double>(splits) * static_cast<double>(m) * n * 4 > 64e6) splits /= 2;
  }
  return {kMxTile64, splits};
}

size_t mx_part_bytes(const MxPlan& p, int64_t m, int n) {
  return p.splits > 1 ? static_cast<size_t>(p.splits) * static_cast<size_t>(m) * n * sizeof(float) : 0;
}

template <int FM, int WK, int KIND>
gptq_status launch_mx_rows(MxArgs a, hipStream_t stream) {
  a.tiles_n = (a.n + 15) / 16;
  const dim3 g(static_cast<unsigned>(tile_rows(a, 16 * FM) * a.tiles_n));
  GPTQ_LAUNCH((mx_rows_kernel<FM, WK, KIND>), g, dim3(WK * 64), 0, stream, a);
  return GPTQ_OK;
}

template <int T, int KIND>
gptq_status launch_mx_tile(MxArgs a, hipStream_t stream) {
  a.order = {(a.n + T - 1) / T, tile_rows(a, T)};
  const dim3 g(static_cast<unsigned>(order_grid(a.order)), static_cast<unsigned>(a.splits));
  GPTQ_LAUNCH((mx_tile_kernel<T, T, KIND>), g, dim3(256), 0, stream, a);
  return GPTQ_OK;
}

template <int KIND>
gptq_status launch_mx(MxArgs a, const MxPlan& p, void* workspace, hipStream_t stream) {
  const int blocks = stage_blocks(KIND);
  a.stages = (a.kb + blocks - 1) / blocks;
  a.splits = p.splits;
  a.per = (a.stages + p.splits - 1) / p.splits;
  a.part = static_cast<float*>(workspace);
  gptq_status st;
  if (p.kind == kMxRows) {
    const int tm = mx_rows_tile(a.m, a.off != nullptr);
    if (tm == 64) return launch_mx_rows<4, 8, KIND>(a, stream);
    if (tm == 32) return launch_mx_rows<2, 8, KIND>(a, stream);
    return a.kb >= 96 ? launch_mx_rows<1, 8, KIND>(a, stream) : launch_mx_rows<1, 4, KIND>(a, stream);
  }
  st = p.kind == kMxTile64 ? launch_mx_tile<64, KIND>(a, stream) : launch_mx_tile<128, KIND>(a, stream);
  if (st != GPTQ_OK || p.splits == 1) return st;
  const dim3 g((a.n + 1023) / 1024, static_cast<unsigned>(a.m));   // parts are of few tiles: m is small
  if (p.splits == 2) GPTQ_LAUNCH(mx_sum_kernel<2>, g, dim3(256), 0, stream, a);
  else if (p.splits == 4) GPTQ_LAUNCH(mx_sum_kernel<4>, g, dim3(256), 0, stream, a);
  else GPTQ_LAUNCH(mx_sum_kernel<8>, g, dim3(256), 0, stream, a);
  return GPTQ_OK;
}

// Whether the launch is one the kernels number their tiles for.
bool mx_launchable(const MxArgs& a, const MxPlan& p) {
  const int tm = p.kind == kMxTile128 ? 128 : p.kind == kMxTile64 ? 64 : mx_rows_tile(a.m, a.off != nullptr);
  const int tn = p.kind == kMxRows ? 16 : tm;
  return tile_rows(a, tm) <= (1 << 22) / ((a.n + tn - 1) / tn);
}

}  // namespace

gptq_status mx_quantize_enqueue(int batch, int64_t rows, int cols, gptq_dtype x_dtype, const void* X, int64_t ldx,
                                int64_t bsx, bool ceil, uint8_t* Q, uint8_t* S, hipStream_t stream) {
  const int kb = cols / MXB;
  const MxQuantArgs a{rows, cols, kb, X, ldx, bsx, Q, S, block_shift(kb)};
  dim3 grid;
  if (!block_grid(rows, kb, batch, a.shift, &grid)) return GPTQ_ERR_UNSUPPORTED;
  if (x_dtype == GPTQ_F32) return launch_mx_quant<float>(a, grid, ceil, stream);
  if (x_dtype == GPTQ_BF16) return launch_mx_quant<BF16>(a, grid, ceil, stream);
  return launch_mx_quant<F16>(a, grid, ceil, stream);
}

gptq_status mx_dequantize_enqueue(int64_t rows, int cols, const uint8_t* Q, const uint8_t* S, gptq_dtype y_dtype,
                                  void* Y, hipStream_t stream) {
  const int kb = cols / MXB;
  const MxDequantArgs a{rows, cols, kb, Q, S, Y, block_shift(kb)};
  dim3 grid;
  if (!block_grid(rows, kb, 1, a.shift, &grid)) return GPTQ_ERR_UNSUPPORTED;
  if (y_dtype == GPTQ_F32) GPTQ_LAUNCH(mx_dequant_kernel<float>, grid, dim3(256), 0, stream, a);
  else if (y_dtype == GPTQ_BF16) GPTQ_LAUNCH(mx_dequant_kernel<BF16>, grid, dim3(256), 0, stream, a);
  else GPTQ_LAUNCH(mx_dequant_kernel<F16>, grid, dim3(256), 0, stream, a);
  return GPTQ_OK;
}

size_t mx_workspace(int64_t m, int n, int k) {
  const size_t parts = std::max(mx_part_bytes(mx_plan(m, n, k, kMx4, false, 1), m, n),
                                mx_part_bytes(mx_plan(m, n, k, kMxBf16, false, 1), m, n));
  return std::max<size_t>(256, parts);
}

gptq_status mx_matmul_enqueue(const MxProblem& p, hipStream_t stream) {
  MxArgs a{};
  a.m = p.n_rows; a.n = p.n; a.k = p.k; a.kb = p.k / MXB;
  a.x_rows = p.x_rows; a.W = p.W; a.ws = p.ws; a.Y = p.Y; a.ldy = p.ldy; a.y_dtype = p.y_dtype;
  a.off = p.offsets; a.rows = p.row_index; a.experts = p.batch;
  a.X = static_cast<const uint8_t*>(p.X);
  a.xs = p.xs; a.xsr = p.xsr;
  const int kind = p.x_dtype == GPTQ_E2M1 ? kMx4 : p.x_dtype == GPTQ_BF16 ? kMxBf16 : kMxF16;
  a.ldx = kind == kMx4 ? p.ldx : 2 * p.ldx;
  if (a.off != nullptr && (a.m / 16 + 1) * a.experts > INT32_MAX) return GPTQ_ERR_UNSUPPORTED;
  const MxPlan plan = mx_plan(a.m, a.n, a.k, kind, a.off != nullptr, a.experts);
  if (!mx_launchable(a, plan)) return GPTQ_ERR_UNSUPPORTED;
  if (plan.splits > 1 && (p.workspace == nullptr || p.workspace_bytes < mx_part_bytes(plan, a.m, a.n)))
    return GPTQ_ERR_WORKSPACE;
  if (kind == kMx4) return launch_mx<kMx4>(a, plan, p.workspace, stream);
  if (kind == kMxBf16) return launch_mx<kMxBf16>(a, plan, p.workspace, stream);
  return launch_mx<kMxF16>(a, plan, p.workspace, stream);
}

}  // namespace gptq
