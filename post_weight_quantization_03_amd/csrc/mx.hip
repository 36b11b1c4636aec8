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
// v_mfma_f32_16x16x32_bf16 with fp32 sums; beside fp16 activations they become fp16 where their scales
// allow it, else the activations go as two bf16 numbers each (333 x 1416 x 2016 25 us so, 14 as fp16).
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
// the scale is 2^-126 and x subnormal).  Bound by memory: 32768 x 8192 bf16 132 us, 5.1 TB/s, which is a
// large copy's rate; 16 x 4096 2.2 us, a launch.
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

// The values back, split like the rounding.  Bound by memory: 32768 x 8192 to bf16 130 us, 5.2 TB/s.
template <typename T>
__global__ __launch_bounds__(256) void mx_dequant_kernel(MxDequantArgs a) {
  const int u = threadIdx.x >> 2, part = threadIdx.x & 3;
  const int b = (blockIdx.y << a.shift) + (u & ((1 << a.shift) - 1));
  const int64_t row = static_cast<int64_t>(blockIdx.x) * (64 >> a.shift) + (u >> a.shift);
  if (row >= a.rows || b >= a.kb) return;
  const int col = b * MXB + part * 8;
  const uint32_t w = *reinterpret_cast<const uint32_t*>(a.Q + row * (a.cols / 2) + col / 2);
  const float s = __uint_as_float(static_cast<uint32_t>(a.S[row * a.kb + b]) << 23);
  const f32x2 v[4] = {
      __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w, s, 0), __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w, s, 1),
      __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w, s, 2), __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w, s, 3)};
  Vec<T, 8> o;
#pragma unroll
  for (int i = 0; i < 8; ++i) o.v[i] = from_f32<T>(v[i / 2][i & 1]);
  __builtin_memcpy(static_cast<T*>(a.Y) + row * a.cols + col, &o, sizeof(o));
}

// No launch here has more rows, nor outputs (2^22 tiles of 256 rows, 2^24 workgroups of 64): refused ahead of the
// arithmetic on them, which would overflow at the end of int64.
constexpr int MX_ROWS = 1 << 30, MX_OUTPUTS = 1 << 30;

// Blocks of a row per workgroup, as a shift: the power of two that holds them, at most 64.
int block_shift(int kb) {
  int s = 0;
  while (s < 6 && (1 << s) < kb) ++s;
  return s;
}
// Grid of the two kernels above; false where it is too large.
bool block_grid(int64_t rows, int kb, int batch, int shift, dim3* grid) {
  if (rows > MX_ROWS) return false;
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
  int cap, slots;    // of the kernel for few rows: rows of a tile, units in a wave's ring
  bool copied;       // and whether scales lie so that they can be copied to LDS
  uint2* xst;        // of the largest tiles: scales by stage
  uint2* wst;
  int64_t mp;        // and their rows
  int np;
  int parts;         // 2 or 4: workgroups of a tile that is behind the last whole round of them
};

// Few rows, at most `cap` (up to 16) of one expert or of the one problem: a workgroup has NW / KS tiles
// of 16 NM outputs, KS waves of it share a tile's inputs.  All comes by copies to LDS: the rows at once,
// and weights in units of 256 inputs, up to DEPTH of them in a ring of each wave's own, so that nothing but
// the matrix instruction's own reads goes through registers.  The waves' sums are added in their order.
// Bound by reading the weights: one row of 4096 x 14336 8.0 to 8.9 us by card (31 MB: 3.7 TB/s from the launch on; 12.7 with
// loads to registers), 16 tokens with 6 of 64 experts of 1408 x 2048 13.4 us (5.8 TB/s, part of it from the
// last-level cache; 26 with loads to registers).  8 waves share a tile of 16 outputs; where there are many
// tiles 4 waves take one of 32 outputs each, so that 8 times the outputs share the rows of X (these 16 tokens:
// 17 us with the fastest other form).
constexpr int UNIT = 2048;   // bytes of a unit of 16 outputs: 8 blocks each
template <int NW, int KS, int NM, int DEPTH, int KIND>
__global__ __launch_bounds__(NW * 64) void mx_few_kernel(MxArgs a) {
  constexpr int GROUPS = NW / KS, COPIES = 2 * NM, XP = KIND == kMx4 ? 1 : 4;   // 16-byte pieces of a block of X
  extern __shared__ __attribute__((aligned(128))) uint8_t few_lds[];
  __shared__ f32x4 part[KS == 1 ? 1 : NW][NM][64];
  const int tid = threadIdx.x, lane = tid & 63, wave = uniform(tid >> 6);
  const int64_t mt = blockIdx.x / a.tiles_n;
  const int tile0 = static_cast<int>(blockIdx.x - mt * a.tiles_n) * GROUPS;
  const Tile t = find_tile(a, mt, a.cap);
  if (t.count <= 0) return;
  const int kb = a.kb, group = wave / KS, wk = wave % KS;
  const int j = lane & 15, q = lane >> 4;
  // the rings, the tiles' scales, zeros, rows of X and their scales
  const int scale_bytes = (16 * NM * kb + 15) / 16 * 16, pitch = 16 * XP * kb + 16, xs_pitch = (kb + 3) / 4 * 4;
  uint8_t* const ring = few_lds + wave * a.slots * NM * UNIT;
  uint8_t* const scales = few_lds + NW * a.slots * NM * UNIT;
  uint8_t* const zeros = scales + GROUPS * scale_bytes;
  uint8_t* const xrows = zeros + 64;
  uint8_t* const xscales = xrows + a.cap * pitch;
  const uint32_t lds0 = static_cast<uint32_t>(reinterpret_cast<uintptr_t>(
      (__attribute__((address_space(3))) uint8_t*)few_lds));
  const uint32_t ring0 = lds0 + wave * a.slots * NM * UNIT;
  const int n0 = 16 * NM * (tile0 + group);   // this wave's outputs
  const int64_t w0 = static_cast<int64_t>(t.e) * a.n + min(n0, a.n - 1);
  const uint8_t* const w = a.W + w0 * (16 * kb);
  const int units = (kb + 7) / 8, mine = (units + KS - 1) / KS;   // of this wave: wk, wk + KS, ..
  // Piece c of row r of a unit lies at c ^ (r / 2 % 8), so that 16 lanes reading the same piece of 16 rows
  // cover all banks.  Behind the last block or output the last one is copied again.
  auto issue = [&](int k) {
    const int unit = wk + KS * k;
#pragma unroll
    for (int i = 0; i < COPIES; ++i) {
      const int r = 8 * i + (lane >> 3), c = (lane & 7) ^ ((r >> 1) & 7);
      const uint32_t off = 16 * (min(r, max(a.n - 1 - n0, 0)) * kb + min(8 * unit + c, kb - 1));
      copy16_at(w, off, ring0 + (k % DEPTH) * NM * UNIT + 1024 * i);
    }
  };
  const int64_t row_j = source_row(a, t.p0 + min(j, t.count - 1));   // columns behind the last row repeat it
  const bool lost = row_j < 0;
  auto row_of = [&](int r) {
    const uint32_t lo = __builtin_amdgcn_readlane(static_cast<int>(row_j), r);
    return static_cast<int64_t>(static_cast<uint64_t>(static_cast<uint32_t>(
               __builtin_amdgcn_readlane(static_cast<int>(row_j >> 32), r))) << 32 | lo);
  };
  // rows, scales and first weights, in this order: the loop starts when the scales are there.  Scales that do not
  // start at multiples of 16 bytes (of X: 4) go through registers, and the first weights are waited for with them.
  if (tid < 16) reinterpret_cast<uint32_t*>(zeros)[tid] = 0;
  const int chunks = (XP * kb + 63) / 64;
  for (int i = wave; i < t.count * chunks; i += NW) {
    const int r = i / chunks, c = i - r * chunks;
    const int64_t row = row_of(r);
    if (row >= 0 && 64 * c + lane < XP * kb)
      copy16_at(a.X + row * a.ldx, 1024 * c + 16 * lane,
                lds0 + static_cast<uint32_t>(xrows - few_lds) + r * pitch + 1024 * c);
  }
  // the outputs' scales are one piece of memory a tile
  const int have = max(0, min(16 * NM, a.n - n0)) * kb;
  const uint8_t* const from = static_cast<const uint8_t*>(a.ws) + (static_cast<int64_t>(t.e) * a.n + n0) * kb;
  if (a.copied) {
    for (int c = wk; 1024 * c < have; c += KS)
      if (1024 * c + 16 * lane < have)
        copy16_at(from, 1024 * c + 16 * lane,
                  lds0 + static_cast<uint32_t>(scales - few_lds) + group * scale_bytes + 1024 * c);
    if constexpr (KIND == kMx4) {
      const int parts = (kb / 4 + 63) / 64;
      for (int i = wave; i < t.count * parts; i += NW) {
        const int r = i / parts, c = i - r * parts;
        const int64_t row = row_of(r);
        if (row >= 0 && 64 * c + lane < kb / 4)
          copy4(static_cast<const uint8_t*>(a.xs) + row * a.xsr + 256 * c + 4 * lane,
                lds0 + static_cast<uint32_t>(xscales - few_lds) + r * xs_pitch + 256 * c);
      }
    }
  }
  for (int k = 0; k < min(DEPTH, mine); ++k) issue(k);
  if (!a.copied) {
    const int g = group, at = tid % (NW * 64 / GROUPS);
    for (int i = 16 * at; i < have; i += 16 * (NW * 64 / GROUPS)) {
      uint8_t v[16];
      if (i + 16 <= have) {
        __builtin_memcpy(v, from + i, 16);
      } else {
#pragma unroll
        for (int b = 0; b < 16; ++b) v[b] = i + b < have ? from[i + b] : 127;
      }
      *reinterpret_cast<uint4*>(scales + g * scale_bytes + i) = *reinterpret_cast<const uint4*>(v);
    }
    if constexpr (KIND == kMx4)
      for (int i = tid; i < t.count * (xs_pitch / 4); i += NW * 64) {
        const int r = i / (xs_pitch / 4), b0 = 4 * (i - r * (xs_pitch / 4));
        const int64_t row = source_row(a, t.p0 + r);
        uint8_t v[4] = {127, 127, 127, 127};
        if (row >= 0) {
          const uint8_t* s = static_cast<const uint8_t*>(a.xs) + row * a.xsr + b0;
          if (b0 + 4 <= kb) __builtin_memcpy(v, s, 4);
          else
            for (int b = 0; b < kb - b0; ++b) v[b] = s[b];
        }
        *reinterpret_cast<uint32_t*>(xscales + r * xs_pitch + b0) = *reinterpret_cast<const uint32_t*>(v);
      }
  }
  if (a.copied && mine >= DEPTH) wait_vmcnt<DEPTH * COPIES>();
  else wait_copies();
  lds_barrier();
  const int jr = min(j, t.count - 1);
  const uint8_t* const x = xrows + jr * pitch;
  const uint8_t* const scale = scales + group * scale_bytes;
  f32x4 y[NM];
#pragma unroll
  for (int g = 0; g < NM; ++g) y[g] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
  auto sum = [&](auto kKind) {
    for (int k = 0; k < mine; ++k) {
      // this unit's copies are the oldest of those of up to DEPTH units
      if (k + DEPTH <= mine) wait_vmcnt<(DEPTH - 1) * COPIES>();
      else wait_copies();
      asm volatile("" ::: "memory");
      const uint8_t* const at = ring + (k % DEPTH) * NM * UNIT + j * 128;
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const int b = 8 * (wk + KS * k) + q + 4 * h;   // this lane's block
        const bool in = b < kb;
        i32x4 v[XP], wv[NM];
        uint32_t s[NM];
#pragma unroll
        for (int g = 0; g < NM; ++g) {
          wv[g] = *reinterpret_cast<const i32x4*>(at + g * UNIT + 16 * ((q + 4 * h) ^ ((j >> 1) & 7)));
          s[g] = scale[(16 * g + j) * kb + min(b, kb - 1)];
        }
        const uint8_t* from = in && !lost ? x + 16 * XP * b : zeros;
#pragma unroll
        for (int p = 0; p < XP; ++p) v[p] = *reinterpret_cast<const i32x4*>(from + 16 * p);
#pragma unroll
        for (int g = 0; g < NM; ++g) s[g] = in ? s[g] : 127u;
        if constexpr (KIND == kMx4) {
          int sx = xscales[jr * xs_pitch + min(b, kb - 1)];
          sx = in ? sx : 127;
#pragma unroll
          for (int g = 0; g < NM; ++g)
            y[g] = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(widen(wv[g]), widen(v[0]), y[g], 4, 4, 0,
                                                                    static_cast<int>(s[g]), 0, sx);
        } else {
#pragma unroll
          for (int p = 0; p < 4; ++p) {
            const XValues<kKind> xv(v[p]);
#pragma unroll
            for (int g = 0; g < NM; ++g)
              y[g] = mx_mma16<kKind>(mx_weights16<kKind>(static_cast<uint32_t>(wv[g][p]), s[g]), xv, y[g]);
          }
        }
      }
      if (k + DEPTH < mine) {
        asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");   // the unit has been read
        issue(k + DEPTH);
      }
    }
  };
  if constexpr (KIND == kMxF16) {
    ScaleRange range;   // of this wave's tile
    for (int i = 16 * lane; i < have; i += 1024) {
      const uint4 v = *reinterpret_cast<const uint4*>(scale + i);
      range.add(v.x), range.add(v.y), range.add(v.z), range.add(v.w);
    }
    if (__all(range.f16())) sum(MxConst<kMxF16Direct>{});
    else sum(MxConst<kMxF16>{});
  } else {
    sum(MxConst<KIND>{});
  }
  if constexpr (KS > 1) {
#pragma unroll
    for (int g = 0; g < NM; ++g) part[wave][g][lane] = y[g];
    __syncthreads();
    if (wk != 0) return;
#pragma unroll
    for (int h = 1; h < KS; ++h)
#pragma unroll
      for (int g = 0; g < NM; ++g) y[g] += part[wave + h][g][lane];
  }
  if (j >= t.count) return;
#pragma unroll
  for (int g = 0; g < NM; ++g) {
    const float f[4] = {lost ? 0.0f : y[g][0], lost ? 0.0f : y[g][1], lost ? 0.0f : y[g][2], lost ? 0.0f : y[g][3]};
    store_y(a, t.p0 + j, n0 + 16 * g + 4 * q, f);
  }
}

// The tile kernel's stage is XB bytes of every row of X: XB / 64 instructions for each 16 outputs x 16
// rows, the h-th of which takes the row's 16-byte pieces 4 h + q, q = 0..3 by lane: with 4 bits a block of
// 32 inputs each, with 16 bits 8 inputs of one block, whose 8 codes are word q of piece h of the weights.
template <int KIND, int XB>
struct MxStage {
  static constexpr int WB = KIND == kMx4 ? XB : XB / 4;            // bytes of a row of W
  static constexpr int BLOCKS = KIND == kMx4 ? XB / 16 : XB / 64;  // scales of a row
  // where piece c of row r lies: 16 lanes reading the same piece (of W in 16 bits: word of one) of 16 rows
  // cover all banks
  static __device__ __forceinline__ int x_at(int r, int c) { return XB == 128 ? c ^ ((r >> 1) & 7) : c ^ (r & 15); }
  static __device__ __forceinline__ int w_at(int r, int c) {
    return KIND == kMx4 ? x_at(r, c) : WB == 32 ? c ^ ((r >> 3) & 1) : c ^ ((r >> 2) & 3);
  }
};

// Tiles of TM rows x TN outputs, 2 x 2 waves (1 x 4 where it is wider than high), NB buffers, NB - 1 stages of
// copies on the way.  The scales of up to PB blocks are in LDS before their first stage, so that the loop has no
// loads but copies and can wait for them by their number.  gridDim.y parts of the inputs: few tiles would leave
// most of the chip idle (sums of parts are added by mx_sum_kernel).
// Bound by the copies, which take two workgroups' 60 to 160 KB of LDS from L2 with a latency of 1 to 2 us: the
// more outputs a tile has for its rows of 16 bits, the less is copied (4096 x 14336, 16-bit rows: 16 rows 32 x 128
// 15 us, 64 x 64 18; 256 rows 64 x 128 45 us, 64 x 64 52; 1024 rows 64 x 128 132, 128 x 128 151).
template <int TM, int TN, int XB, int NB, int KIND>
__global__ __launch_bounds__(256) void mx_tile_kernel(MxArgs a) {
  typedef MxStage<KIND, XB> St;
  constexpr int NW = 4, WM = TM < TN ? 1 : 2, WN = NW / WM, XW = TM / WM, WW = TN / WN;   // waves, and their tiles
  constexpr int FM = XW / 16, FN = WW / 16, H = XB / 64;
  constexpr int STAGE = TM * XB + TN * St::WB, XROWS = 1024 / XB, WROWS = 1024 / St::WB;   // rows of one copy
  constexpr int LX = TM * XB / 1024 / NW, LW = TN * St::WB / 1024 / NW, LD = LX + LW;
  // two workgroups on a CU, of 32 rows three: what the buffers leave of their LDS is for scales (experts of 1408 x
  // 2048, 64 tokens with 6 of 64: 22 us, 28 with three buffers and two workgroups)
  constexpr int SPACE = (TM == 32 ? 52 : 80) * 1024 - 256;
  constexpr int SROWS = KIND == kMx4 ? TM + TN : TN;
  constexpr int PB = std::min(256, ((SPACE - NB * STAGE) / SROWS - 4) / 16 * 16), PITCH = PB + 4;
  static_assert(LX >= 1 && LW >= 1 && PB >= 16 && PB % St::BLOCKS == 0 && SROWS <= 256, "tile shape");
  static_assert(TM % (16 * WM) == 0 && TN % (16 * WN) == 0, "tile shape");
  __shared__ __attribute__((aligned(128))) uint8_t lds[NB * STAGE];
  __shared__ __attribute__((aligned(16))) uint8_t scales[SROWS * PITCH];
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

  const uint8_t* xsrc[LX];
  const uint8_t* wsrc[LW];
  int xc[LX], wc[LW];   // this lane's pieces
#pragma unroll
  for (int i = 0; i < LX; ++i) {
    const int r = (wave + NW * i) * XROWS + lane / (XB / 16);
    const int64_t row = source_row(a, t.p0 + min(r, t.count - 1));
    xc[i] = St::x_at(r, lane % (XB / 16));
    xsrc[i] = row >= 0 ? a.X + row * a.ldx + 16 * xc[i] : nullptr;
  }
#pragma unroll
  for (int i = 0; i < LW; ++i) {
    const int r = (wave + NW * i) * WROWS + lane / (St::WB / 16);
    wc[i] = St::w_at(r, lane % (St::WB / 16));
    wsrc[i] = We + static_cast<int64_t>(min(n0 + r, a.n - 1)) * (a.k / 2) + 16 * wc[i];
  }
  if (tid < TM) lost[tid] = source_row(a, t.p0 + min(tid, t.count - 1)) < 0;
  const unsigned lds0 = static_cast<unsigned>(reinterpret_cast<uintptr_t>(
      (__attribute__((address_space(3))) uint8_t*)lds));
  auto issue = [&](int s, int buffer) {
    const unsigned to = lds0 + buffer * STAGE + wave * 1024;
#pragma unroll
    for (int i = 0; i < LX; ++i) {
      const int64_t at = static_cast<int64_t>(s) * XB;
      copy16(at + 16 * xc[i] < xbytes && xsrc[i] != nullptr ? xsrc[i] + at : zeros, to + NW * i * 1024);
    }
#pragma unroll
    for (int i = 0; i < LW; ++i) {
      const int64_t at = static_cast<int64_t>(s) * St::WB;
      copy16(at + 16 * wc[i] < a.k / 2 ? wsrc[i] + at : zeros, to + TM * XB + NW * i * 1024);
    }
  };

  const int wm = wave / WN, wn = wave % WN;
  const int j = lane & 15, q = lane >> 4;
  f32x4 y[FM][FN];
#pragma unroll
  for (int i = 0; i < FM; ++i)
#pragma unroll
    for (int h = 0; h < FN; ++h) y[i][h] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
  for (int p0 = first; p0 < end; p0 += PB / St::BLOCKS) {
    const int p1 = min(p0 + PB / St::BLOCKS, end);
    if (p0 > first) __syncthreads();   // everyone is done with the scales and buffers before
    ScaleRange range;
    for (int i = tid; i < SROWS * (((p1 - p0) * St::BLOCKS + 15) / 16); i += 256) {
      const int r = i % SROWS, b0 = p0 * St::BLOCKS + 16 * (i / SROWS);
      const int o = KIND == kMx4 ? r - TM : r;
      const uint8_t* row = nullptr;
      if (o >= 0) {
        row = static_cast<const uint8_t*>(a.ws) + (static_cast<int64_t>(t.e) * a.n + min(n0 + o, a.n - 1)) * a.kb;
      } else {
        const int64_t x = source_row(a, t.p0 + min(r, t.count - 1));
        if (x >= 0) row = static_cast<const uint8_t*>(a.xs) + x * a.xsr;
      }
      uint32_t v[4] = {0x7F7F7F7Fu, 0x7F7F7F7Fu, 0x7F7F7F7Fu, 0x7F7F7F7Fu};   // behind the last block: 1
      if (row != nullptr && b0 + 16 <= a.kb) {
        __builtin_memcpy(v, row + b0, 16);
      } else if (row != nullptr && b0 < a.kb) {
        uint8_t b[16];
#pragma unroll
        for (int e = 0; e < 16; ++e) b[e] = b0 + e < a.kb ? row[b0 + e] : 127;
        __builtin_memcpy(v, b, 16);
      }
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        *reinterpret_cast<uint32_t*>(scales + r * PITCH + 16 * (i / SROWS) + 4 * e) = v[e];
        if constexpr (KIND == kMxF16) range.add(v[e]);
      }
    }
    asm volatile("s_waitcnt vmcnt(0)" ::: "memory");   // the loop counts copies alone
#pragma unroll
    for (int s = 0; s < NB - 1; ++s)
      if (p0 + s < p1) issue(p0 + s, s);
    auto sum = [&](auto kKind) {
      for (int s = p0; s < p1; ++s) {
        // this stage's copies are the oldest of those of up to NB - 1 stages
        if (NB >= 4 && s + 2 < p1) wait_vmcnt<2 * LD>();
        else if (NB >= 3 && s + 1 < p1) wait_vmcnt<LD>();
        else wait_vmcnt<0>();
        __syncthreads();   // everyone's copies have landed, and everyone is done with the stage before
        if (s + NB - 1 < p1) issue(s + NB - 1, (s - p0 + NB - 1) % NB);
        const uint8_t* xb = lds + (s - p0) % NB * STAGE + wm * XW * XB;
        const uint8_t* wb = lds + (s - p0) % NB * STAGE + TM * XB + wn * WW * St::WB;
        const uint8_t* sc = scales + (s - p0) * St::BLOCKS;
        const uint8_t* ws = sc + ((KIND == kMx4 ? TM : 0) + wn * WW + j) * PITCH;
#pragma unroll
        for (int h = 0; h < H; ++h) {
          i32x4 w4[FN];
          decltype(mx_weights16<kKind>(0u, 0u)) w16[FN];
          int sw[FN];
#pragma unroll
          for (int f = 0; f < FN; ++f) {
            const uint8_t* row = wb + (16 * f + j) * St::WB;
            if constexpr (KIND == kMx4) {
              w4[f] = *reinterpret_cast<const i32x4*>(row + 16 * St::w_at(j, 4 * h + q));
              sw[f] = ws[16 * f * PITCH + 4 * h + q];
            } else {
              w16[f] = mx_weights16<kKind>(*reinterpret_cast<const uint32_t*>(row + 16 * St::w_at(j, h) + 4 * q),
                                           ws[16 * f * PITCH + h]);
            }
          }
#pragma unroll
          for (int i = 0; i < FM; ++i) {
            const i32x4 v = *reinterpret_cast<const i32x4*>(xb + (16 * i + j) * XB + 16 * St::x_at(j, 4 * h + q));
            if constexpr (KIND == kMx4) {
              const int sx = sc[(wm * XW + 16 * i + j) * PITCH + 4 * h + q];
#pragma unroll
              for (int f = 0; f < FN; ++f)
                y[i][f] = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(widen(w4[f]), widen(v), y[i][f], 4, 4, 0,
                                                                           sw[f], 0, sx);
            } else {
              const XValues<kKind> xv(v);
#pragma unroll
              for (int f = 0; f < FN; ++f) y[i][f] = mx_mma16<kKind>(w16[f], xv, y[i][f]);
            }
          }
        }
      }
    };
    if constexpr (KIND == kMxF16) {
      if (__syncthreads_and(range.f16())) sum(MxConst<kMxF16Direct>{});
      else sum(MxConst<kMxF16>{});
    } else {
      sum(MxConst<KIND>{});
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
    const int r = wm * XW + 16 * i + j;
    if (r >= t.count) continue;
    const bool none = lost[r];
#pragma unroll
    for (int h = 0; h < FN; ++h) {
      const f32x4 s = y[i][h];
      const float v[4] = {none ? 0.0f : s[0], none ? 0.0f : s[1], none ? 0.0f : s[2], none ? 0.0f : s[3]};
      store_y(out, t.p0 + r, n0 + wn * WW + 16 * h + 4 * q, v);
    }
  }
}

// The same product for large problems: 256 x 256 tiles, 4 waves of 128 x 128 (8 x 8 blocks of 16 x 16),
// one workgroup per CU.  Bound by the matrix cores: 8192 x 4096 x 14336 of 4-bit rows 204 us, 4.7 PFLOP/s (on
// another card 221, and 169 without copies, scales and stores; the cores are busy 55% of the time),
// 4096 x 14336 x 4096 of 16-bit rows 370 us, 1.30 PFLOP/s, where the library's large bf16 product reaches
// 1.36 (without the weights' conversion it is no faster).  Two buffers; a stage is 128 bytes of every row of
// X, two instructions for a block (four for fp16 as two bf16), here together called a product.  Operands go
// global -> LDS with a scalar base that moves by a stage and one 32-bit offset per lane and copy.  Before a wave's last
// three rows of blocks it has read all it needs of the stage: there the workgroup waits for the next stage's
// copies, and the products of these rows cover the first reads of the next stage and half of the copies
// of the one after it; the other half goes out with the next stage's first products.
// A tile of up to 128 rows or outputs (the last of a ragged problem or expert) goes the same way with half
// the work per wave.
constexpr int BIG = 256;
template <int KIND>
struct BigW {
  decltype(mx_weights16<KIND>(0u, 0u)) v[2];
};
template <>
struct BigW<kMx4> {
  i32x4 v[2];
  int s;   // the scales of both halves in its two low bytes
};
template <int KIND>
struct BigX {
  i32x4 v[2];
  int s;
};
template <int KIND>
__device__ __forceinline__ void big_product(const BigW<KIND>& w, const BigX<KIND>& x, f32x4& acc) {
  if constexpr (KIND == kMx4) {
    acc = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(widen(w.v[0]), widen(x.v[0]), acc, 4, 4, 0, w.s, 0, x.s);
    acc = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(widen(w.v[1]), widen(x.v[1]), acc, 4, 4, 1, w.s, 1, x.s);
  } else {
    acc = mx_mma16<KIND>(w.v[0], XValues<KIND>(x.v[0]), acc);
    acc = mx_mma16<KIND>(w.v[1], XValues<KIND>(x.v[1]), acc);
  }
}

// The scales of 4-bit operands stage by stage, for this kernel: 8 codes of every output row [stages][mp]
// and of every output [experts][stages][np], those behind the last block 1, in the order 0 4 1 5 2 6 3 7, so
// that a lane's two are neighbours.  (Read where they are, 8 bytes a stage come out of lines of 128, which
// doubles what a CU reads: 8192 x 4096 x 14336 286 us, 221 so, this kernel's 7 in it.)
constexpr int GATHER = 8;   // stages of a thread
__global__ __launch_bounds__(256) void mx_gather_scales_kernel(MxArgs a) {
  const int64_t g = static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x;
  const uint8_t* row = nullptr;
  uint2* to;
  int64_t step;
  if (g < a.mp) {
    const int64_t x = g < a.m ? source_row(a, g) : -1;
    if (x >= 0) row = static_cast<const uint8_t*>(a.xs) + x * a.xsr;
    to = a.xst + g;
    step = a.mp;
  } else {
    const int64_t w = g - a.mp, e = w / a.np;
    const int o = static_cast<int>(w - e * a.np);
    if (e >= a.experts) return;
    if (o < a.n) row = static_cast<const uint8_t*>(a.ws) + (e * a.n + o) * a.kb;
    to = a.wst + e * a.stages * a.np + o;
    step = a.np;
  }
  for (int s = blockIdx.y * GATHER; s < min(static_cast<int>(blockIdx.y + 1) * GATHER, a.stages); ++s) {
    uint32_t v[2] = {0x7F7F7F7Fu, 0x7F7F7F7Fu};
    if (row != nullptr && 8 * s + 8 <= a.kb) {
      __builtin_memcpy(v, row + 8 * s, 8);
    } else if (row != nullptr) {
#pragma unroll 1
      for (int i = 0; i < a.kb - 8 * s; ++i) {
        const uint32_t c = static_cast<uint32_t>(row[8 * s + i] ^ 0x7F) << (8 * (i & 3));
        if (i < 4) v[0] ^= c;
        else v[1] ^= c;
      }
    }
    to[s * step] =
        make_uint2(__builtin_amdgcn_perm(v[1], v[0], 0x05010400u), __builtin_amdgcn_perm(v[1], v[0], 0x07030602u));
  }
}

// Outputs n0 .. of the rows of t: XR rows of X and WR of W, waves_n waves beside each other.
template <int KIND, int XR, int WR, int FM, int FN>
__device__ __forceinline__ void big_tile(const MxArgs& a, const Tile& t, int n0, int waves_n, uint8_t* lds, uint2* scs,
                                         bool* lost) {
  typedef MxStage<KIND, 128> St;
  constexpr bool F4 = KIND == kMx4;
  constexpr int NW = 4, STAGE = XR * 128 + WR * St::WB, WROWS = 1024 / St::WB;
  constexpr int LX = XR / 8 / NW, LW = WR / WROWS / NW, LD = LX + LW;
  constexpr int SROWS = F4 ? 2 * BIG : BIG;   // rows of scales: of X, then of W
  const int tid = threadIdx.x, lane = tid & 63, wave = uniform(tid >> 6);
  const int stages = a.stages;
  const uint8_t* xbase = a.X + (a.rows == nullptr ? t.p0 * a.ldx : 0);
  const uint8_t* wbase = a.W + (static_cast<int64_t>(t.e) * a.n + n0) * (a.k / 2);
  // this lane's pieces: the same in every copy of X, and of W; whether they lie past K in the last stage
  const int cx = St::x_at(8 * wave + lane / 8, lane & 7);
  const int cw = St::w_at(WROWS * wave + lane / (St::WB / 16), lane % (St::WB / 16));
  const bool cut_x = (stages - 1) * 128 + 16 * cx >= (F4 ? a.k / 2 : 2 * a.k);
  const bool cut_w = (stages - 1) * St::WB + 16 * cw >= a.k / 2;
  uint32_t off[LD];
#pragma unroll
  for (int i = 0; i < LD; ++i) {
    if (i < LX) {
      const int r = (wave + NW * i) * 8 + lane / 8;
      const int64_t row = source_row(a, t.p0 + min(r, t.count - 1));   // none: row 0, and zeros at the end
      const int64_t from = max(a.rows == nullptr ? row - t.p0 : row, static_cast<int64_t>(0));
      off[i] = static_cast<uint32_t>(from * a.ldx) + 16 * cx;
    } else {
      const int r = (wave + NW * (i - LX)) * WROWS + lane / (St::WB / 16);
      off[i] = static_cast<uint32_t>(min(r, a.n - 1 - n0)) * static_cast<uint32_t>(a.k / 2) + 16 * cw;
    }
  }
  const int64_t own = source_row(a, t.p0 + min(tid, t.count - 1));
  lost[tid] = own < 0;
  // 4-bit operands' scales are copied; those of the weights of 16-bit rows go through a register, 2 in
  // 4 bytes that end with the row at the latest
  const uint8_t* const wsrow =
      static_cast<const uint8_t*>(a.ws) + (static_cast<int64_t>(t.e) * a.n + min(n0 + tid, a.n - 1)) * a.kb;
  uint32_t sw_next = 0;
  const unsigned scs0 = static_cast<unsigned>(reinterpret_cast<uintptr_t>(
      (__attribute__((address_space(3))) uint2*)scs));
  const unsigned lds0 = static_cast<unsigned>(reinterpret_cast<uintptr_t>(
      (__attribute__((address_space(3))) uint8_t*)lds));
  auto issue_scales = [&](int s) {
    if constexpr (F4) {
      const uint2* x = a.xst + static_cast<int64_t>(s) * a.mp + t.p0;
      const uint2* w = a.wst + (static_cast<int64_t>(t.e) * a.stages + s) * a.np + n0;
#pragma unroll
      for (int i = 0; i < XR / 128; ++i) {
        const int at = 2 * XR * wave + 256 * i;   // bytes
        copy4(reinterpret_cast<const uint8_t*>(x) + at + 4 * lane, scs0 + (s & 1) * SROWS * 8 + at);
      }
#pragma unroll
      for (int i = 0; i < WR / 128; ++i) {
        const int at = 2 * WR * wave + 256 * i;
        copy4(reinterpret_cast<const uint8_t*>(w) + at + 4 * lane, scs0 + (s & 1) * SROWS * 8 + BIG * 8 + at);
      }
    } else {
      __builtin_memcpy(&sw_next, wsrow + min(2 * s, a.kb - 4), 4);
    }
  };
  auto issue_copies = [&](int s, int from, int to) {
    const uint8_t* xb = xbase + static_cast<int64_t>(s) * 128;
    const uint8_t* wb = wbase + static_cast<int64_t>(s) * St::WB;
    const unsigned dst = lds0 + (s & 1) * STAGE + wave * 1024;
    // past K the row's first piece instead; zeroed below
    const uint32_t back_x = s == stages - 1 && cut_x ? 16 * cx : 0, back_w = s == stages - 1 && cut_w ? 16 * cw : 0;
#pragma unroll
    for (int i = from; i < to; ++i) {
      if (i < LX) copy16_at(xb, off[i] - back_x, dst + NW * i * 1024);
      else copy16_at(wb, off[i] - back_w, dst + XR * 128 + NW * (i - LX) * 1024);
    }
  };
  // the copies and scales of stage s have landed; the next barrier makes them visible
  auto land = [&](int s, bool last) {
    wait_copies();
    if (last) {
#pragma unroll
      for (int i = 0; i < LD; ++i)
        if (i < LX ? cut_x : cut_w) {
          const int at = i < LX ? NW * i * 1024 : XR * 128 + NW * (i - LX) * 1024;
          *reinterpret_cast<uint4*>(lds + (s & 1) * STAGE + wave * 1024 + at + 16 * lane) = make_uint4(0, 0, 0, 0);
        }
    }
    if constexpr (!F4)
      reinterpret_cast<uint16_t*>(scs)[(s & 1) * BIG + tid] =
          static_cast<uint16_t>(sw_next >> (8 * (2 * s - min(2 * s, a.kb - 4))));
  };
  auto barrier = [&] {
    asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
    __builtin_amdgcn_s_barrier();
    asm volatile("" ::: "memory");
  };

  const int wm = wave / waves_n, wn = wave % waves_n;
  const int j = lane & 15, q = lane >> 4;
  const int xr = wm * 16 * FM, wr = wn * 16 * FN;
  const int at0 = j * 128 + 16 * St::x_at(j, q), at1 = j * 128 + 16 * St::x_at(j, q + 4);
  auto half_x = [&](int s, int i, int half, BigX<KIND>& o) {
    o.v[half] = *reinterpret_cast<const i32x4*>(lds + (s & 1) * STAGE + (xr + 16 * i) * 128 + (half ? at1 : at0));
  };
  auto scale_x = [&](int s, int i, BigX<KIND>& o) {
    if constexpr (F4) o.s = reinterpret_cast<const uint16_t*>(&scs[(s & 1) * SROWS + xr + 16 * i + j])[q];
  };
  auto read_w = [&](int s, int h, BigW<KIND>& o) {
    const uint8_t* base = lds + (s & 1) * STAGE + XR * 128 + (wr + 16 * h) * St::WB;
    if constexpr (F4) {
      o.v[0] = *reinterpret_cast<const i32x4*>(base + at0);
      o.v[1] = *reinterpret_cast<const i32x4*>(base + at1);
      o.s = reinterpret_cast<const uint16_t*>(&scs[(s & 1) * SROWS + BIG + wr + 16 * h + j])[q];
    } else {
      const uint32_t sc = reinterpret_cast<const uint16_t*>(scs)[(s & 1) * BIG + wr + 16 * h + j];
      const uint8_t* row = base + j * St::WB + 4 * q;
      o.v[0] = mx_weights16<KIND>(*reinterpret_cast<const uint32_t*>(row + 16 * St::w_at(j, 0)), sc & 255);
      o.v[1] = mx_weights16<KIND>(*reinterpret_cast<const uint32_t*>(row + 16 * St::w_at(j, 1)), sc >> 8);
    }
  };

  f32x4 y[FM][FN];
#pragma unroll
  for (int i = 0; i < FM; ++i)
#pragma unroll
    for (int h = 0; h < FN; ++h) y[i][h] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
  BigX<KIND> xf[4];   // row of blocks i in xf[i % 4]
  BigW<KIND> wf[FN];
  // Products of a stage: rows of blocks one after another, then the last three together, output block by
  // output block.
  constexpr int LAST = 3, SPLIT = (FM - LAST) * FN;   // rows taken together, products before them
  // copies issued with them, one after every second product
  constexpr int EARLY = LAST * FN / 2 < LD ? LAST * FN / 2 : LD;
  // the barrier keeps everything in the order written
  auto product = [&](auto P) {
    constexpr int p = P, i = p < SPLIT ? p / FN : FM - LAST + (p - SPLIT) % LAST;
    constexpr int h = p < SPLIT ? p % FN : (p - SPLIT) / LAST;
    big_product<KIND>(wf[h], xf[i % 4], y[i][h]);
    __builtin_amdgcn_sched_barrier(0);
  };
  // one stage; kMore: another follows, kIssue: and one after that (constants, so that the loop's body has no
  // branch)
  auto stage = [&](int s, auto kMore, auto kIssue) {
    // all rows but the last three; row i + 3 is read meanwhile, one access after each product
    static_for(std::make_integer_sequence<int, SPLIT>{}, [&](auto P) {
      constexpr int p = P, i = p / FN, h = p % FN;
      product(P);
      if constexpr (h == 0) half_x(s, i + 3, 0, xf[(i + 3) % 4]);
      if constexpr (h == 1) half_x(s, i + 3, 1, xf[(i + 3) % 4]);
      if constexpr (h == 2) scale_x(s, i + 3, xf[(i + 3) % 4]);
      // the rest of the next stage's copies
      if constexpr (kMore && p % 2 == 1 && EARLY + p / 2 < LD) issue_copies(s + 1, EARLY + p / 2, EARLY + p / 2 + 1);
      __builtin_amdgcn_sched_barrier(0);
    });
    if constexpr (kMore) {
      land(s + 1, !kIssue);
      barrier();
      if constexpr (kIssue) issue_scales(s + 2);
      // operand 0 is free: the next stage's first
      half_x(s + 1, 0, 0, xf[0]);
      half_x(s + 1, 0, 1, xf[0]);
      scale_x(s + 1, 0, xf[0]);
      __builtin_amdgcn_sched_barrier(0);
    }
    // the last three rows: a weight operand makes room for the next stage's after its third product
    static_for(std::make_integer_sequence<int, LAST * FN>{}, [&](auto Q) {
      constexpr int n = Q, h = n / LAST;
      product(std::integral_constant<int, SPLIT + n>{});
      if constexpr (kMore && n % LAST == LAST - 1) read_w(s + 1, h, wf[h]);
      if constexpr (kIssue && n % 2 == 1 && n / 2 < EARLY) issue_copies(s + 2, n / 2, n / 2 + 1);
      __builtin_amdgcn_sched_barrier(0);
    });
    if constexpr (kMore) {
#pragma unroll
      for (int i = 1; i < 3; ++i) {
        half_x(s + 1, i, 0, xf[i]);
        half_x(s + 1, i, 1, xf[i]);
        scale_x(s + 1, i, xf[i]);
      }
      __builtin_amdgcn_sched_barrier(0);
    }
  };

  issue_scales(0);
  issue_copies(0, 0, LD);
  land(0, stages == 1);
  barrier();
  if (stages > 1) {
    issue_scales(1);
    issue_copies(1, 0, EARLY);
  }
#pragma unroll
  for (int i = 0; i < 3; ++i) {
    half_x(0, i, 0, xf[i]);
    half_x(0, i, 1, xf[i]);
    scale_x(0, i, xf[i]);
  }
#pragma unroll
  for (int h = 0; h < FN; ++h) read_w(0, h, wf[h]);
  const std::true_type yes;
  const std::false_type no;
  for (int s = 0; s + 2 < stages; ++s) stage(s, yes, yes);
  if (stages > 1) stage(stages - 2, yes, no);
  stage(stages - 1, no, no);

  if (a.y_dtype == GPTQ_F32) {
#pragma unroll
    for (int i = 0; i < FM; ++i) {
      const int r = xr + 16 * i + j;
      if (r >= t.count) continue;
      const bool none = lost[r];
#pragma unroll
      for (int h = 0; h < FN; ++h) {
        const float v[4] = {none ? 0.0f : y[i][h][0], none ? 0.0f : y[i][h][1], none ? 0.0f : y[i][h][2],
                            none ? 0.0f : y[i][h][3]};
        store_y(a, t.p0 + r, n0 + wr + 16 * h + 4 * q, v);
      }
    }
    return;
  }
  // Of outputs 16 h + 4 q .. of two neighbouring h, lanes of odd and even q exchange one each (they are of one
  // row): a lane then stores 8 in 16 bytes, and four lanes 64 bytes of a row in one piece.
  const int o0 = n0 + wr + 16 * (q & 1) + 8 * (q >> 1);
  const bool whole = n0 + wr + 16 * FN <= a.n;
  auto store = [&](auto kBf16, auto kWhole) {
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
          if constexpr (kWhole) __builtin_memcpy(out + 16 * h, &w, sizeof(w));
          else store_narrow(a, out + 16 * h, o0 + 16 * h, w);
        }
      }
      out += 16 * a.ldy;
    }
  };
  if (a.y_dtype == GPTQ_BF16) {
    if (whole) store(yes, yes);
    else store(yes, no);
  } else {
    if (whole) store(no, yes);
    else store(no, no);
  }
}

template <int KIND>
__global__ __launch_bounds__(256) void mx_big_kernel(MxArgs a) {
  __shared__ __attribute__((aligned(128))) uint8_t lds[2 * BIG * (128 + MxStage<KIND, 128>::WB)];
  __shared__ uint2 scs[KIND == kMx4 ? 4 * BIG : BIG / 2];
  __shared__ bool lost[BIG];
  // Behind the last whole round of 256 tiles up to 128 go as halves of 128 rows and up to 64 as quarters,
  // those of a tile on one XCD (4096 x 14336 x 4096, half a round left, 16-bit rows 416 us, 385 so; 4096 x 4608
  // x 8192, an eighth, 390 and 285, 4-bit rows 110 and 97).
  uint32_t id = blockIdx.x, part = 0;
  const uint32_t whole = static_cast<uint32_t>(a.order.tiles_m) * static_cast<uint32_t>(a.order.tiles_n) & ~255u;
  if (a.parts > 1 && id >= whole) {
    const uint32_t i = (id - whole) / 8;
    part = i % a.parts;
    id = whole + i / a.parts * 8 + (id - whole) % 8;
  }
  int64_t mt;
  int nt;
  if (!ordered_tile(a.order, id, &mt, &nt)) return;
  Tile t = find_tile<BIG>(a, mt);
  int n0 = nt * BIG;
  const bool narrow = a.parts == 4 && id >= whole;
  if (a.parts > 1 && id >= whole) {
    t.p0 += BIG / 2 * (part & 1);
    t.count = min(BIG / 2, t.count - BIG / 2 * static_cast<int>(part & 1));
    n0 += BIG / 2 * static_cast<int>(part >> 1);
  }
  if (t.count <= 0 || n0 >= a.n) return;
  auto tile = [&](auto kKind) {
    if (narrow) big_tile<kKind, BIG / 2, BIG / 2, 4, 4>(a, t, n0, 2, lds, scs, lost);
    else if (t.count <= BIG / 2) big_tile<kKind, BIG / 2, BIG, 8, 4>(a, t, n0, 4, lds, scs, lost);
    else if (a.n - n0 <= BIG / 2) big_tile<kKind, BIG, BIG / 2, 8, 4>(a, t, n0, 2, lds, scs, lost);
    else big_tile<kKind, BIG, BIG, 8, 8>(a, t, n0, 2, lds, scs, lost);
  };
  if constexpr (KIND == kMxF16) {
    const uint8_t* row = static_cast<const uint8_t*>(a.ws) +
                         (static_cast<int64_t>(t.e) * a.n + min(n0 + static_cast<int>(threadIdx.x), a.n - 1)) * a.kb;
    ScaleRange range;
    for (int b = 0; b < a.kb; b += 4) {
      uint32_t v;
      __builtin_memcpy(&v, row + min(b, a.kb - 4), 4);
      range.add(v);
    }
    if (__syncthreads_and(range.f16())) tile(MxConst<kMxF16Direct>{});
    else tile(MxConst<kMxF16>{});
  } else {
    tile(MxConst<KIND>{});
  }
}

// Y from the sums of the parts, in their order, all loads at once (8 parts of 64 x 4096: 4 us, mostly a
// launch's; 18 with a loop of loads).  A thread takes 4 outputs of a row, and threads are numbered through all
// rows: there may be millions of rows of a few outputs.
template <int SPLITS>
__global__ __launch_bounds__(256) void mx_sum_kernel(MxArgs a) {
  const uint32_t quads = static_cast<uint32_t>(a.n + 3) / 4, g = blockIdx.x * 256 + threadIdx.x, row = g / quads;
  if (row >= a.m) return;
  const int o = static_cast<int>(g - row * quads) * 4, n = min(4, a.n - o);
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

enum MxProduct { kMxFew, kMxTile32, kMxWide64, kMxTile64, kMxTile128, kMxBig };
struct MxPlan {
  MxProduct kind;
  int splits;
  int cap;     // kMxFew: rows of a tile
  bool wide;   // kMxFew: 4 tiles of 32 outputs a workgroup, else one of 16
};

// The tile kernel's stages: 256 inputs of 4-bit rows; of 16-bit ones 128 in the small tiles, else 64.
constexpr int tile_rows_of(MxProduct p) {
  return p == kMxBig ? BIG : p == kMxTile128 ? 128 : p == kMxTile32 ? 32 : 64;
}
constexpr int tile_outputs(MxProduct p) { return p == kMxBig ? BIG : p == kMxTile64 ? 64 : 128; }
constexpr int tile_xb(MxProduct p, int kind) { return kind != kMx4 && p != kMxTile128 ? 256 : 128; }
constexpr int tile_blocks(MxProduct p, int kind) { return tile_xb(p, kind) / (kind == kMx4 ? 16 : 64); }
constexpr int tile_buffers(MxProduct p) { return p == kMxTile128 || p == kMxTile32 ? 2 : 3; }

// The kernel for few rows: 8 waves sharing one tile of 16 outputs, or 4 waves with one of 32 each.
// (units of a ring: 3 rows of 5120 x 5120 7.1 us with 2, 9.1 with 3, 9.5 with 4; one of 4096 x 14336 8.5, 8.9, 9.4)
constexpr int FEW_DEPTH = 2;
// Two workgroups on a CU, and one.  Waves that share a tile hold 8 KB of sums besides, so that a tile of theirs that takes
// all of the first leaves one there too (5 rows of 16 bits and 4096 inputs: 84 KB).
constexpr int FEW_LDS = 78 * 1024, FEW_MOST_LDS = 150 * 1024;
int few_slots(int kb, bool wide) { return std::min((kb + 7) / 8 / (wide ? 1 : 8) + 1, FEW_DEPTH); }
// LDS without rows of X, and of a row.
int64_t few_fixed(int kb, bool wide) {
  const int64_t scales = wide ? 4 * ((32 * static_cast<int64_t>(kb) + 15) / 16 * 16) : 16 * static_cast<int64_t>(kb);
  return (wide ? 4 * 2 : 8) * few_slots(kb, wide) * UNIT + scales + 64;
}
int64_t few_row(int kb, int kind) {
  return kind == kMx4 ? 16 * static_cast<int64_t>(kb) + 16 + (kb + 3) / 4 * 4 : 64 * static_cast<int64_t>(kb) + 16;
}

// Whether the launch is one the kernels number their tiles for; experts 0: not grouped.
bool mx_launchable(int64_t m, int n, int experts, const MxPlan& p) {
  const int tm = p.kind == kMxFew ? p.cap : tile_rows_of(p.kind);
  const int tn = p.kind == kMxFew ? 16 : tile_outputs(p.kind);
  const int64_t rows = experts == 0 ? (m + tm - 1) / tm : m / tm + std::min<int64_t>(experts, m);
  return rows <= (1 << 22) / ((n + tn - 1) / tn);
}

// What a kernel takes, in us, as measured on the card (two sides of each choice below): the start of a launch
// and its loop, and its stages of 128 inputs of 16-bit rows or 256 of 4-bit ones where a CU has one workgroup
// and where it has as many as it holds.  Those of 32 x 128 tiles were taken with three buffers and two workgroups
// on a CU, where there are now two buffers and three workgroups.
struct MxCost {
  double start, one, full;
  int held;   // workgroups of a CU
};
constexpr MxCost mx_cost(MxProduct kind, bool four) {
  return kind == kMxTile32   ? MxCost{4.0, 0.57, 0.82, 2}
         : kind == kMxWide64 ? MxCost{3.5, 0.85, 1.18, 2}   // of 16-bit rows
         : kind == kMxTile64 ? (four ? MxCost{2.5, 0.51, 0.72, 2} : MxCost{3.0, 0.59, 0.83, 2})
         : kind == kMxTile128 ? (four ? MxCost{4.0, 1.02, 1.68, 2} : MxCost{5.0, 1.36, 2.14, 2})
                              : (four ? MxCost{10.0, 1.9, 1.9, 1} : MxCost{8.0, 3.1, 3.1, 1});
}
constexpr double FEW_START = 2.0;
// a CU's bytes in 1 us of the kernel for few rows, weights and rows of X (conversions slow 16-bit ones)
constexpr double few_rate(int kind) { return kind == kMx4 ? 23e3 : 18e3; }
constexpr double SUM_START = 2.5, SUM_RATE = 4e6;   // of adding parts: bytes written and read in 1 us
// experts differ, and few large tiles do not even that out (16-bit rows, 4096 tokens: 232 us, 128 x 128 196)
constexpr double BIG_UNEVEN = 0.6;
// a round of halves or quarters, as a part of one of whole tiles: more is copied for as many products
constexpr double big_rest(bool quarters, bool four) {
  return quarters ? (four ? 0.78 : 0.5) : four ? 0.95 : 0.62;
}
constexpr int CUS = 256;

// Which kernel, by sizes alone (the workspace's size goes by the same rule): the one with the least estimate.
// What it takes (us, in brackets the best of the other kernels on the same card; experts: 6 of 64 for each token,
// 1408 x 2048):
//   16-bit rows   4096 x 14336           14336 x 4096          experts, tokens
//      2          few 9.5 (14.1)         few 10.7 (13.4)       16: few 14.6 (18.2)
//      16         32 x 128 14.8 (17.6)   32 x 128 14.4 (17.1)  256: 32 x 128 33 (42)
//      256        64 x 128 46 (52)       64 x 128 43 (49)      1024: 64 x 128 69 (69)
//      512        64 x 128 77 (86)       256 x 256 64 (64)     8192: 128 x 128 335 (348)
//      2048       256 x 256 213 (217)    256 x 256 207 (224)   16384: 256 x 256 579 (633)
//   4-bit rows    8: few 9.2 (12.6)      8: few 11.1 (11.8)    4: few 9.0 (11.1)
//      32         64 x 64 13.8 (13.8)    64 x 64 12.1 (13.9)   64: 32 x 128 17.9 (20.6)
//      512        64 x 64 43 (47)        128 x 128 31 (35)     256: 32 x 128 25 (29)
//      1024       128 x 128 67 (66)      256 x 256 40 (59)     1024: 128 x 128 43 (45)
//      4096       256 x 256 105 (171)    256 x 256 139 (196)   4096: 256 x 256 97 (106)
// It is off where kernels are close and the estimate is that of other buffers, or that of experts, which is low
// throughout: 16-bit rows, experts of 384, 512 and 4096 tokens 64 x 128 48, 49 and 210 (32 x 128 39 and 43, 128 x 128
// 192), 4 rows of 14336 x 4096 32 x 128 13.6 (few 11.6); 4-bit rows, experts of 16 and 384 tokens 32 x 128 14.6 and
// 64 x 64 33 (few 12.9, 32 x 128 27.5).
MxPlan mx_plan(int64_t m, int n, int k, int kind, bool grouped, int experts) {
  const bool four = kind == kMx4;
  const double used = grouped ? static_cast<double>(std::min<int64_t>(experts, m)) : 1.0;
  const double rows = static_cast<double>(m) / used;
  const int kb = k / MXB;
  MxPlan best{kMxTile64, 1, 0, false};
  double least = 1e30;
  auto take = [&](const MxPlan& p, double t) {
    if (t < least && mx_launchable(m, n, grouped ? experts : 0, p)) least = t, best = p;
  };
  // few rows: as many a tile as LDS holds with two workgroups on a CU, or one if that spares reading weights twice
  const bool wide = kb <= 128 && used * ((n + 15) / 16) > 1024;
  const int64_t most = std::min<int64_t>(16, m);
  const int64_t want = std::min<int64_t>(most, static_cast<int64_t>(grouped ? 1.5 * rows + 2 : m));
  const int64_t fit = (FEW_LDS - few_fixed(kb, wide)) / few_row(kb, kind);
  const int64_t alone = (FEW_MOST_LDS - few_fixed(kb, wide)) / few_row(kb, kind);
  const int64_t cap = std::min(most, std::max(fit, std::min(want, alone)));
  if (cap >= 1 && rows <= 16) {
    const int outputs = wide ? 128 : 16;
    const double groups = std::max(1.0, used * ((n + outputs - 1) / outputs) / CUS);
    const double passes = std::ceil(rows / static_cast<double>(cap));
    const double bytes = passes * 17.0 * outputs * kb + rows * few_row(kb, kind);
    take({kMxFew, 1, static_cast<int>(cap), wide}, FEW_START + groups * bytes / few_rate(kind));
  }
  for (const MxProduct p : {kMxTile32, kMxTile64, kMxWide64, kMxTile128, kMxBig}) {
    if ((p == kMxBig && kb < 8) || (p == kMxWide64 && four)) continue;
    const MxCost c = mx_cost(p, four);
    const int tm = tile_rows_of(p), tn = tile_outputs(p);
    // experts' last tiles are half full on average, and one has at least one
    const double mts = grouped ? used * std::max(1.0, rows / tm + 0.5) : static_cast<double>((m + tm - 1) / tm);
    const double tiles = mts * ((n + tn - 1) / tn);
    const int units = (kb + (four ? 7 : 3)) / (four ? 8 : 4);
    for (int splits = 1; splits <= 16; splits *= 2) {
      if (splits > 1 && (grouped || p == kMxTile128 || p == kMxBig || units < 2 * splits ||
                         static_cast<double>(splits) * static_cast<double>(m) * n * 4 > 64e6))
        break;
      const double groups = tiles * splits, full = std::floor(groups / (c.held * CUS));
      const double rest = groups - full * c.held * CUS;
      double round = full * c.full + (rest == 0 ? 0.0 : rest <= CUS ? c.one : c.full);
      if (p == kMxBig && grouped) round += BIG_UNEVEN * c.full;
      else if (p == kMxBig && rest > 0 && rest <= 128) round -= c.full * (1.0 - big_rest(rest <= 64, four));
      const double parts = splits == 1 ? 0.0 : SUM_START + 8.0 * splits * static_cast<double>(m) * n / SUM_RATE;
      take({p, splits, 0, false}, c.start + (units + splits - 1) / splits * round + parts);
    }
  }
  return best;
}

// The largest tiles' scales: rows and outputs that a tile may read behind the last.
int64_t big_rows(int64_t m) { return m + BIG; }
int big_outputs(int n) { return (n + BIG - 1) / BIG * BIG; }

// Workspace: sums of parts, or scales by stage.
size_t mx_plan_bytes(const MxPlan& p, int64_t m, int n, int k, int kind, int experts) {
  if (p.kind == kMxBig && kind == kMx4)
    return static_cast<size_t>((k / MXB + 7) / 8) * 8 * (big_rows(m) + static_cast<size_t>(experts) * big_outputs(n));
  return p.splits > 1 ? static_cast<size_t>(p.splits) * static_cast<size_t>(m) * n * sizeof(float) : 0;
}

template <int NW, int KS, int NM, int DEPTH, int KIND>
gptq_status launch_mx_few(MxArgs a, const MxPlan& p, hipStream_t stream) {
  constexpr int OUTPUTS = NW / KS * NM * 16;
  a.tiles_n = (a.n + OUTPUTS - 1) / OUTPUTS;
  a.cap = p.cap;
  a.copied = reinterpret_cast<uintptr_t>(a.ws) % 16 == 0 && static_cast<int64_t>(a.n) * a.kb % 16 == 0 &&
             (KIND != kMx4 || (reinterpret_cast<uintptr_t>(a.xs) % 4 == 0 && a.xsr % 4 == 0 && a.kb % 4 == 0));
  a.slots = few_slots(a.kb, p.wide);
  const dim3 g(static_cast<unsigned>(tile_rows(a, a.cap) * a.tiles_n));
  GPTQ_LAUNCH((mx_few_kernel<NW, KS, NM, DEPTH, KIND>), g, dim3(NW * 64),
              static_cast<size_t>(few_fixed(a.kb, p.wide) + a.cap * few_row(a.kb, KIND)), stream, a);
  return GPTQ_OK;
}

template <MxProduct P, int KIND>
gptq_status launch_mx_tile(MxArgs a, const MxPlan& p, void* workspace, hipStream_t stream) {
  constexpr int TM = tile_rows_of(P), TN = tile_outputs(P), BLOCKS = tile_blocks(P, KIND);
  a.order = {(a.n + TN - 1) / TN, tile_rows(a, TM)};
  a.stages = (a.kb + BLOCKS - 1) / BLOCKS;
  a.splits = p.splits;
  a.per = (a.stages + p.splits - 1) / p.splits;
  a.part = static_cast<float*>(workspace);
  const dim3 g(static_cast<unsigned>(order_grid(a.order)), static_cast<unsigned>(a.splits));
  GPTQ_LAUNCH((mx_tile_kernel<TM, TN, tile_xb(P, KIND), tile_buffers(P), KIND>), g, dim3(256), 0, stream, a);
  if (p.splits == 1) return GPTQ_OK;
  // parts are of at most 64e6 bytes, so there are fewer than 2^23 groups of 4 outputs
  const dim3 s(static_cast<unsigned>((a.m * ((a.n + 3) / 4) + 255) / 256));
  if (p.splits == 2) GPTQ_LAUNCH(mx_sum_kernel<2>, s, dim3(256), 0, stream, a);
  else if (p.splits == 4) GPTQ_LAUNCH(mx_sum_kernel<4>, s, dim3(256), 0, stream, a);
  else if (p.splits == 8) GPTQ_LAUNCH(mx_sum_kernel<8>, s, dim3(256), 0, stream, a);
  else GPTQ_LAUNCH(mx_sum_kernel<16>, s, dim3(256), 0, stream, a);
  return GPTQ_OK;
}

template <int KIND>
gptq_status launch_mx_big(MxArgs a, void* workspace, hipStream_t stream) {
  constexpr int BLOCKS = MxStage<KIND, 128>::BLOCKS;
  a.stages = (a.kb + BLOCKS - 1) / BLOCKS;
  a.order = {(a.n + BIG - 1) / BIG, tile_rows(a, BIG)};
  if constexpr (KIND == kMx4) {
    a.mp = big_rows(a.m);
    a.np = big_outputs(a.n);
    a.xst = static_cast<uint2*>(workspace);
    a.wst = a.xst + a.stages * a.mp;
    const int64_t rows = a.mp + static_cast<int64_t>(a.experts) * a.np;
    const dim3 g(static_cast<unsigned>((rows + 255) / 256), (a.stages + GATHER - 1) / GATHER);
    GPTQ_LAUNCH(mx_gather_scales_kernel, g, dim3(256), 0, stream, a);
  }
  const int64_t tiles = a.order.tiles_m * a.order.tiles_n, whole = tiles & ~static_cast<int64_t>(255);
  a.parts = a.off != nullptr || tiles - whole > 128 ? 1 : tiles - whole > 64 ? 2 : 4;
  const int64_t grid = whole + a.parts * (order_grid(a.order) - whole);
  GPTQ_LAUNCH(mx_big_kernel<KIND>, dim3(static_cast<unsigned>(grid)), dim3(256), 0, stream, a);
  return GPTQ_OK;
}

template <int KIND>
gptq_status launch_mx(const MxArgs& a, const MxPlan& p, void* workspace, hipStream_t stream) {
  if (p.kind == kMxFew)
    return p.wide ? launch_mx_few<4, 1, 2, FEW_DEPTH, KIND>(a, p, stream)
                  : launch_mx_few<8, 8, 1, FEW_DEPTH, KIND>(a, p, stream);
  if (p.kind == kMxBig) return launch_mx_big<KIND>(a, workspace, stream);
  if (p.kind == kMxTile32) return launch_mx_tile<kMxTile32, KIND>(a, p, workspace, stream);
  if constexpr (KIND != kMx4)
    if (p.kind == kMxWide64) return launch_mx_tile<kMxWide64, KIND>(a, p, workspace, stream);
  if (p.kind == kMxTile64) return launch_mx_tile<kMxTile64, KIND>(a, p, workspace, stream);
  return launch_mx_tile<kMxTile128, KIND>(a, p, workspace, stream);
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

size_t mx_workspace(int batch, bool grouped, int64_t m, int n, int k) {
  size_t most = 256;
  if (m < 1 || m > MX_ROWS || n > MX_OUTPUTS) return most;   // nothing is launched
  for (const int kind : {kMx4, kMxBf16})
    most = std::max(most, mx_plan_bytes(mx_plan(m, n, k, kind, grouped, batch), m, n, k, kind, batch));
  return most;
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
  if (a.m > MX_ROWS || a.n > MX_OUTPUTS || (a.off != nullptr && (a.m / 16 + 1) * a.experts > INT32_MAX)) return GPTQ_ERR_UNSUPPORTED;
  MxPlan plan = mx_plan(a.m, a.n, a.k, kind, a.off != nullptr, a.experts);
  // the largest tiles address a tile's rows by 32-bit offsets
  const int64_t span = a.rows == nullptr ? BIG * a.ldx : a.x_rows * a.ldx;
  if (plan.kind == kMxBig && (span > INT32_MAX || BIG * static_cast<int64_t>(a.k / 2) > INT32_MAX || a.x_rows == 0))
    plan.kind = kMxTile128;
  if (!mx_launchable(a.m, a.n, a.off != nullptr ? a.experts : 0, plan)) return GPTQ_ERR_UNSUPPORTED;
  const size_t need = mx_plan_bytes(plan, a.m, a.n, a.k, kind, a.experts);
  if (need > 0 && (p.workspace == nullptr || p.workspace_bytes < need)) return GPTQ_ERR_WORKSPACE;
  if (kind == kMx4) return launch_mx<kMx4>(a, plan, p.workspace, stream);
  if (kind == kMxBf16) return launch_mx<kMxBf16>(a, plan, p.workspace, stream);
  return launch_mx<kMxF16>(a, plan, p.workspace, stream);
}

}  // namespace gptq

// Which form a product takes, for tests that cover every form; not part of the interface.  kind as MxKind,
// experts 0: not grouped.  MxProduct | wide << 3 | splits << 4 | cap << 9.
extern "C" int gptq_internal_mxfp4_form(int64_t m, int n, int k, int kind, int experts) {
  const gptq::MxPlan p = gptq::mx_plan(m, n, k, kind, experts > 0, std::max(experts, 1));
  return p.kind | p.wide << 3 | p.splits << 4 | p.cap << 9;
}
