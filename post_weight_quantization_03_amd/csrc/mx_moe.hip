// The expert layer of a mixture-of-experts block for few tokens on gfx950, in two launches:
//
//   out[t, :] = sum_j weights[t, j] W2[e] (act(G[e] x_t) * U[e] x_t),   e = ids[t, j]
//
// with W1[e] = [G[e]; U[e]] and W2[e] in the 4-bit microscaled form and 16-bit x.  Both kernels are
// bound by reading the weights of the experts that some token chose, each once; the weights become
// bf16 in registers, exactly, in front of v_mfma_f32_16x16x32_bf16, as the first operand, with
// an expert's tokens as the columns of the second.  The activations between the kernels carry the routing
// weight and are two bf16 planes (the value and the rest, 16 bits together): one plane would add
// an error like the output's own rounding, and the matrix cores are idle anyway.
#include <algorithm>
#include <cfloat>

#include "mx.h"

namespace gptq {
namespace {

constexpr int APART = 32;   // counters in a 128-byte line each
constexpr int MLP_NW = 4, MLP_NT = MLP_NW * 64;
// Two workgroups on a CU, and one.  Waves that share a tile's inputs hold 8 KB of sums besides, so that one of theirs that
// takes all of the first leaves one there too (16 tokens, 2 of 8 experts, d 2048, inner 1408: 86 and 85 KB).
constexpr int MLP_LDS = 78 * 1024, MLP_MOST_LDS = 150 * 1024;

struct MlpArgs {
  int tokens, top_k, experts, d, inner;
  int kb1, kb2;          // blocks of d and of inner
  const uint8_t* X;
  int64_t ldx;           // bytes
  const int32_t* ids;
  const float* weights;
  const uint8_t* W1;
  const uint8_t* s1;
  const uint8_t* W2;
  const uint8_t* s2;
  int act;
  uint16_t* H;           // [2][pairs][inner]
  float* Z;              // [pairs][d]
  int32_t* clean;        // [pairs] ids, -1 for those that add nothing, then how many add something
  int* done;             // [d / 16], APART apart: how many of them the second launch has finished, by part
  void* out;
  int64_t ldo;
  int cap;               // tokens at a time
};

enum MlpAct { kSilu = 0, kGeluTanh = 1 };
__device__ __forceinline__ float mlp_act(float g, int act) {
  // 0.5 g (1 + tanh z) = g / (1 + exp(-2 z)), z = sqrt(2 / pi) (g + 0.044715 g^3)
  // in powers of two: within (|z| + 4) 2^-22
  const float z = act == kSilu ? g : 1.5957691216057308f * (g + 0.044715f * g * g * g);
  return g * __builtin_amdgcn_rcpf(1.0f + __builtin_amdgcn_exp2f(-1.4426950408889634f * z));
}

// A token that names an expert twice takes it once, at its first choice, with both weights.
__device__ __forceinline__ bool first_choice(const int16_t* ids, int i, int top_k) {
  for (int k = i / top_k * top_k; k < i; ++k)
    if (ids[k] == ids[i]) return false;
  return true;
}

// Values that workgroups of one launch hand over: past the L2s, which the 8 XCDs do not share (writing
// back and invalidating them around plain accesses took 195 us for 32 tokens).
__device__ __forceinline__ void store_through(float* p, f32x4 v) {
  uint64_t u[2];
  __builtin_memcpy(u, &v, 16);
  __hip_atomic_store(reinterpret_cast<uint64_t*>(p), u[0], __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
  __hip_atomic_store(reinterpret_cast<uint64_t*>(p) + 1, u[1], __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}
__device__ __forceinline__ f32x4 load_through(const float* p) {
  uint64_t u[2];
  u[0] = __hip_atomic_load(reinterpret_cast<const uint64_t*>(p), __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
  u[1] = __hip_atomic_load(reinterpret_cast<const uint64_t*>(p) + 1, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
  f32x4 v;
  __builtin_memcpy(&v, u, 16);
  return v;
}

// What the second launch needs to know, from one workgroup of the first: the ids, -1 for those that add
// nothing, how many do, and counters at 0.
__device__ __forceinline__ void prepare_second(const MlpArgs& a, int16_t* ids) {
  __shared__ int total;
  const int pairs = a.tokens * a.top_k;
  if (threadIdx.x == 0) total = 0;
  for (int i = threadIdx.x; i < pairs; i += MLP_NT) {
    const int v = a.ids[i];
    ids[i] = static_cast<int16_t>(v >= 0 && v < a.experts ? v : -1);
  }
  for (int i = threadIdx.x; i < a.d / 16; i += MLP_NT) a.done[i * APART] = 0;
  __syncthreads();
  for (int i = threadIdx.x; i < pairs; i += MLP_NT) {
    const bool counts = ids[i] >= 0 && first_choice(ids, i, a.top_k);
    a.clean[i] = counts ? ids[i] : -1;
    if (counts) atomicAdd(&total, 1);
  }
  __syncthreads();
  if (threadIdx.x == 0) a.clean[pairs] = total;
}

// The outputs of tiles tile0 .. of all tokens: their choices' results in order.
template <int KIND>
__device__ __forceinline__ void finish_part(const MlpArgs& a, const int16_t* ids, int tile0, int tiles) {
  for (int g = threadIdx.x; g < a.tokens * tiles * 4; g += MLP_NT) {
    const int t = g / (tiles * 4), o = 16 * tile0 + 4 * (g - t * (tiles * 4));
    f32x4 v = {0.0f, 0.0f, 0.0f, 0.0f};
    for (int k0 = 0; k0 < a.top_k; k0 += 8) {
      f32x4 z[8];
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        const int i = t * a.top_k + k0 + k;
        z[k] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
        if (k0 + k < a.top_k && ids[i] >= 0) z[k] = load_through(a.Z + static_cast<int64_t>(i) * a.d + o);
      }
#pragma unroll
      for (int k = 0; k < 8; ++k) v += z[k];
    }
    uint16_t u[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) u[i] = KIND == kMxBf16 ? from_f32<BF16>(v[i]).bits : from_f32<F16>(v[i]).bits;
    __builtin_memcpy(static_cast<uint16_t*>(a.out) + t * a.ldo + o, u, sizeof(u));
  }
}

// One of the two launches.  Workgroup (slot, part) takes one expert and GROUPS of its tiles of 16 rows of
// weights (of G and U each in the first launch), for all of the expert's tokens, `cap` at a time.  The
// expert is the slot-th, or where there are fewer choices than experts the slot-th choice's, if no choice
// before names it.  Everything comes by copies to LDS, which arrive in the order they were asked for: the
// tokens' rows and a tile's scales at once, and its weights in units of 256 inputs, DEPTH of them in a ring
// of each wave's own.  (Loads to registers in the order of the matrix instruction need as many registers
// as bytes in flight, and steps behind the last that load something too: 32 tokens of 6 of 64 experts
// 82.8 us, 78.6 so; one token 19.2 and 16.5.)  Workgroups of 4 waves, two on a CU, cover each other's
// start (8 waves, one on a CU: 90 us).  KS waves share a tile's inputs: 1 where there are tiles for all
// waves of the chip, 2 or 4 otherwise.  Bound by reading the weights: of 32 tokens with 6 of 64 experts (d 2048,
// inner 1408) the first launch takes 37 us, 5.0 TB/s, the second 32, 2.9 TB/s with the sum of the choices at
// its end; of one token 8.3 and 7.1 us, half of which is the way to the first weights.
//
// The first launch writes H: weight * act(gate) * up.  The second adds nothing up between experts: it
// writes each choice's result to Z, and the last workgroup of a part to finish sums a token's choices in
// their order.  Its tiles are of 32 rows, which share the reads of H's two planes from LDS.
constexpr int NM = 2;           // sets of 16 rows of a tile: of G and U, or 32 rows of W2
constexpr int UNIT = 2048;      // bytes of a unit of one of them: 16 rows of 8 blocks
constexpr int COPIES = 2 * NM;  // of a unit
constexpr int DEPTH = 2;
template <bool UP, int KS, int KIND>
__global__ __launch_bounds__(MLP_NT) void mlp_kernel(MlpArgs a) {
  constexpr int PLANES = UP ? 1 : 2, GROUPS = MLP_NW / KS;
  extern __shared__ __attribute__((aligned(128))) uint8_t mlp_lds[];
  __shared__ int listed;
  __shared__ f32x4 part[KS == 1 ? 1 : MLP_NW][NM][64];
  const int tid = threadIdx.x, lane = tid & 63, wave = uniform(tid >> 6);
  const int pairs = a.tokens * a.top_k, rows = UP ? a.inner : a.d, kb = UP ? a.kb1 : a.kb2;
  const int all = rows / (UP ? 16 : 32), parts = (all + GROUPS - 1) / GROUPS;   // tiles
  const int slot = blockIdx.x / parts, which = blockIdx.x - slot * parts, tile0 = which * GROUPS;
  const int tiles = min(GROUPS, all - tile0);
  // the rings, the tiles' scales, a block of zeros, rows of the second operand [cap][PLANES], the expert's
  // list of pairs [tokens] and ids [pairs]
  const int scale_bytes = (16 * kb + 1023) / 1024 * 1024;   // of one matrix
  const int pitch = 64 * kb + 16;                           // 16 rows' pieces at one place cover all banks
  uint8_t* const scales = mlp_lds + MLP_NW * DEPTH * NM * UNIT;
  uint8_t* const zeros = scales + GROUPS * NM * scale_bytes;
  uint8_t* const xrows = zeros + 64;
  int16_t* const list = reinterpret_cast<int16_t*>(xrows + a.cap * PLANES * pitch);
  int16_t* const ids = list + a.tokens;
  const int32_t* const from_ids = UP ? a.ids : a.clean;
  if constexpr (UP)
    if (blockIdx.x == 0) prepare_second(a, ids);
  const bool by_choice = pairs <= a.experts;
  const int e = by_choice ? from_ids[slot] : slot;
  if constexpr (!UP)
    if (slot == 0 && a.clean[pairs] == 0) {   // zeros
      for (int i = tid; i < pairs; i += MLP_NT) ids[i] = -1;
      __syncthreads();
      finish_part<KIND>(a, ids, 2 * tile0, 2 * tiles);
      return;
    }
  if (e < 0 || e >= a.experts) return;

  // the expert's pairs, in order
  if (tid < 16) reinterpret_cast<uint32_t*>(zeros)[tid] = 0;
  for (int i = tid; i < pairs; i += MLP_NT) {
    const int v = from_ids[i];
    ids[i] = static_cast<int16_t>(v >= 0 && v < a.experts ? v : -1);
  }
  __syncthreads();
  if (wave == 0) {
    int n = 0;
    for (int i0 = 0; i0 < pairs; i0 += 64) {
      const int i = i0 + lane;
      const bool mine = i < pairs && ids[i] == e && (!UP || first_choice(ids, i, a.top_k));
      const uint64_t all = __ballot(mine);
      if (mine) list[n + __popcll(all & ((1ull << lane) - 1))] = static_cast<int16_t>(i);
      n += __popcll(all);
    }
    if (lane == 0) listed = n;
  }
  __syncthreads();
  const int count = uniform(listed);
  if (count == 0 || (by_choice && list[0] != slot)) return;

  const int j = lane & 15, q = lane >> 4, group = wave / KS, wk = wave % KS;
  const int64_t row0 = static_cast<int64_t>(e) * (UP ? 2 : 1) * rows + (UP ? 16 : 32) * (tile0 + min(group, tiles - 1));
  const uint8_t* const w = (UP ? a.W1 : a.W2) + row0 * (16 * kb);
  const uint8_t* const ws = (UP ? a.s1 : a.s2) + row0 * kb;
  const int64_t s_up = static_cast<int64_t>(UP ? rows : 16) * kb, w_up = 16 * s_up;   // to the second matrix
  const int units = (kb + 7) / 8, mine = (units + KS - 1) / KS;   // of a tile, of this wave: wk, wk + KS, ..
  const uint32_t lds0 = static_cast<uint32_t>(reinterpret_cast<uintptr_t>(
      (__attribute__((address_space(3))) uint8_t*)mlp_lds));
  const uint32_t ring0 = lds0 + wave * DEPTH * NM * UNIT;
  uint8_t* const ring = mlp_lds + wave * DEPTH * NM * UNIT;
  uint8_t* const scale = scales + group * NM * scale_bytes;
  // Piece c of row r of a unit lies at c ^ (r / 2 % 8), so that 16 lanes reading the same piece of 16 rows
  // cover all banks.  Behind the last block the last one is copied again (its scale counts as 1, and the
  // other operand is zeros).
  auto issue = [&](int k) {
    const int unit = wk + KS * k;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int r = 8 * i + (lane >> 3), c = (lane & 7) ^ ((r >> 1) & 7);
      const uint32_t off = 16 * (r * kb + min(8 * unit + c, kb - 1));
#pragma unroll
      for (int g = 0; g < NM; ++g) copy16_at(w + g * w_up, off, ring0 + ((k % DEPTH) * NM + g) * UNIT + 1024 * i);
    }
  };
  for (int r0 = 0; r0 < count; r0 += a.cap) {
    const int n = min(a.cap, count - r0);
    if (r0 > 0) __syncthreads();   // the rows before have been read
    // copies arrive in order: rows and scales, then weights
    const int chunks = (4 * kb + 63) / 64;
    for (int i = wave; i < n * PLANES * chunks; i += MLP_NW) {
      const int r = i / chunks, c = i - r * chunks, pair = uniform(static_cast<int>(list[r0 + r / PLANES]));
      const uint8_t* from =
          UP ? a.X + static_cast<int64_t>(pair / a.top_k) * a.ldx
             : reinterpret_cast<const uint8_t*>(a.H + (static_cast<int64_t>(r % PLANES) * pairs + pair) * a.inner);
      const uint32_t to = static_cast<uint32_t>(xrows - mlp_lds) + r * pitch + 1024 * c;
      if (64 * c + lane < 4 * kb) copy16_at(from, 1024 * c + 16 * lane, lds0 + to);
    }
    if (r0 == 0)
      for (int i = wk; i < NM * (scale_bytes / 1024); i += KS) {
        const int g = i / (scale_bytes / 1024), c = i - g * (scale_bytes / 1024);
        copy16_at(ws + g * s_up, min(1024 * c + 16 * lane, 16 * kb - 16),
                  lds0 + static_cast<uint32_t>(scale - mlp_lds) + g * scale_bytes + 1024 * c);
      }
    for (int k = 0; k < min(DEPTH, mine); ++k) issue(k);
    if (mine >= DEPTH) wait_vmcnt<DEPTH * COPIES>();
    else wait_copies();
    const int pair = list[r0 + min(j, n - 1)];   // columns behind the last token repeat it; nothing reads them
    lds_barrier();
    const uint8_t* const x = xrows + min(j, n - 1) * PLANES * pitch;
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
          i32x4 v[PLANES][4], wv[NM];
          uint32_t s[NM];
#pragma unroll
          for (int g = 0; g < NM; ++g) {
            wv[g] = *reinterpret_cast<const i32x4*>(at + g * UNIT + 16 * ((q + 4 * h) ^ ((j >> 1) & 7)));
            s[g] = scale[g * scale_bytes + j * kb + min(b, kb - 1)];
          }
#pragma unroll
          for (int l = 0; l < PLANES; ++l) {
            const uint8_t* from = in ? x + l * pitch + 64 * b : zeros;
#pragma unroll
            for (int p = 0; p < 4; ++p) v[l][p] = *reinterpret_cast<const i32x4*>(from + 16 * p);
          }
#pragma unroll
          for (int g = 0; g < NM; ++g) s[g] = in ? s[g] : 127u;
#pragma unroll
          for (int p = 0; p < 4; ++p) {
#pragma unroll
            for (int g = 0; g < NM; ++g) {
              const auto wf = mx_weights16<kKind>(static_cast<uint32_t>(wv[g][p]), s[g]);
              if constexpr (UP) {
                y[g] = mx_mma16<kKind>(wf, XValues<kKind>(v[0][p]), y[g]);
              } else {
                y[g] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(wf, __builtin_bit_cast(bf16x8, v[1][p]), y[g], 0, 0, 0);
                y[g] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(wf, __builtin_bit_cast(bf16x8, v[0][p]), y[g], 0, 0, 0);
              }
            }
          }
        }
        if (k + DEPTH < mine) {
          asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");   // the unit has been read
          issue(k + DEPTH);
        }
      }
    };
    if constexpr (UP && KIND == kMxF16) {
      ScaleRange range;   // of this wave's tile
      for (int i = 4 * lane; i < 16 * kb; i += 256)
#pragma unroll
        for (int g = 0; g < NM; ++g) range.add(*reinterpret_cast<const uint32_t*>(scale + g * scale_bytes + i));
      if (__all(range.f16())) sum(MxConst<kMxF16Direct>{});
      else sum(MxConst<kMxF16>{});
    } else {
      sum(MxConst<UP ? KIND : kMxBf16>{});
    }
    if constexpr (KS > 1) {
      if (r0 > 0) lds_barrier();   // the sums before have been read
#pragma unroll
      for (int g = 0; g < NM; ++g) part[wave][g][lane] = y[g];
      lds_barrier();
      if (wk == 0)
#pragma unroll
        for (int h = 1; h < KS; ++h)
#pragma unroll
          for (int g = 0; g < NM; ++g) y[g] += part[wave + h][g][lane];
    }
    if (wk == 0 && group < tiles && j < n) {
      const int o = (UP ? 16 : 32) * (tile0 + group) + 4 * q;
      if constexpr (UP) {
        float weight = a.weights[pair];
        for (int i = pair + 1, end = (pair / a.top_k + 1) * a.top_k; i < end; ++i)
          if (ids[i] == e) weight += a.weights[i];   // the token names the expert again
        Vec<BF16, 4> hi, lo;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const float h = weight * (mlp_act(y[0][i], a.act) * y[1][i]);
          hi.v[i] = from_f32<BF16>(h);
          const float near = bf16_to_f32(hi.v[i].bits);
          lo.v[i] = from_f32<BF16>(fabsf(near) <= FLT_MAX ? h - near : 0.0f);   // an infinity has no rest
        }
        uint16_t* to = a.H + static_cast<int64_t>(pair) * a.inner + o;
        *reinterpret_cast<Vec<BF16, 4>*>(to) = hi;
        *reinterpret_cast<Vec<BF16, 4>*>(to + static_cast<int64_t>(pairs) * a.inner) = lo;
      } else {
        store_through(a.Z + static_cast<int64_t>(pair) * a.d + o, y[0]);
        store_through(a.Z + static_cast<int64_t>(pair) * a.d + o + 16, y[1]);
      }
    }
  }
  if constexpr (!UP) {
    __builtin_amdgcn_s_waitcnt(0);   // this wave's stores have reached memory
    __syncthreads();                 // and everyone's
    if (tid == 0)
      listed = __hip_atomic_fetch_add(&a.done[which * APART], count, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    __syncthreads();
    if (listed + count != a.clean[pairs]) return;
    finish_part<KIND>(a, ids, 2 * tile0, 2 * tiles);
  }
}

template <bool UP, int KS, int KIND>
gptq_status launch_half(MlpArgs a, hipStream_t stream) {
  constexpr int GROUPS = MLP_NW / KS, NM = 2, PLANES = UP ? 1 : 2;
  const int pairs = a.tokens * a.top_k, slots = std::min(a.experts, pairs), tiles = UP ? a.inner / 16 : a.d / 32;
  const int kb = UP ? a.kb1 : a.kb2;
  const int fixed = MLP_NW * DEPTH * NM * UNIT + GROUPS * NM * ((16 * kb + 1023) / 1024 * 1024) + 64 +
                    2 * (a.tokens + pairs);
  const int row = PLANES * (64 * kb + 16), most = std::min(16, a.tokens);
  // An expert's weights are read again for every `cap` of its tokens.  Two workgroups on a CU are worth more
  // than room for the few experts that have more tokens than the average and its square root (64 tokens, 6 of
  // 64 experts, d = 2048: 9 at a time 117 us, 11 with one workgroup 133), but less than room for more of them
  // (32 tokens, 2 of 8, d = 4096: 8 at a time 88 us, 14 80; 8 tokens, 2 of 8, inner = 2816: 3 28 us, 5 25).
  const int fit = (MLP_LDS - fixed) / row, want = 3 * pairs / (2 * a.experts) + 2;
  const double spare = fit - static_cast<double>(pairs) / a.experts;
  const bool enough = spare >= 0 && spare * spare * a.experts >= pairs;
  a.cap = std::min(most, enough ? fit : std::max(fit, std::min(want, (MLP_MOST_LDS - fixed) / row)));
  if (a.cap < 1) return GPTQ_ERR_UNSUPPORTED;
  const dim3 grid(static_cast<unsigned>(slots * ((tiles + GROUPS - 1) / GROUPS)));
  GPTQ_LAUNCH((mlp_kernel<UP, KS, KIND>), grid, dim3(MLP_NT), static_cast<size_t>(fixed) + a.cap * row, stream, a);
  return GPTQ_OK;
}
// Waves share a tile's inputs where there are fewer tiles than waves (4 workgroups of 4 for each CU), and
// where one tile's scales for each wave would take too much LDS: 4 where an expert has one token, else 2, whose
// tiles share the tokens' rows (16 tokens, 2 of 8 experts, 1408 x 2048: 28 us, 24 so; one token, 6 of 64: 17.5, 17).
int mlp_waves(bool up, int pairs, int experts, int d, int inner) {
  const int64_t tiles = static_cast<int64_t>(std::min(experts, pairs)) * (up ? inner / 16 : d / 32);
  const bool long_rows = (up ? d : inner) > 4096;
  if (long_rows || tiles <= (pairs <= experts ? 1024 : 384)) return 4;
  return tiles <= 1024 ? 2 : 1;
}
template <bool UP, int KIND>
gptq_status launch_half(const MlpArgs& a, hipStream_t stream) {
  const int waves = mlp_waves(UP, a.tokens * a.top_k, a.experts, a.d, a.inner);
  if (waves == 4) return launch_half<UP, 4, KIND>(a, stream);
  if (waves == 2) return launch_half<UP, 2, KIND>(a, stream);
  return launch_half<UP, 1, KIND>(a, stream);
}

template <int KIND>
gptq_status launch_mlp(const MlpArgs& a, hipStream_t stream) {
  const gptq_status st = launch_half<true, KIND>(a, stream);
  return st == GPTQ_OK ? launch_half<false, KIND>(a, stream) : st;
}

struct MlpLayout {
  size_t z, clean, done, total;
};
MlpLayout mlp_layout(int64_t pairs, int inner, int d) {
  MlpLayout l{};
  l.z = align_up(4 * static_cast<size_t>(pairs) * inner, 256);
  l.clean = l.z + align_up(4 * static_cast<size_t>(pairs) * d, 256);
  l.done = l.clean + align_up(4 * (static_cast<size_t>(pairs) + 1), 256);
  l.total = l.done + align_up(4 * APART * static_cast<size_t>(d / 16), 256);
  return l;
}

}  // namespace

size_t mx_mlp_workspace(int64_t pairs, int inner, int d) { return mlp_layout(pairs, inner, d).total; }

gptq_status mx_mlp_enqueue(const MxMlp& p, hipStream_t stream) {
  const int64_t pairs = static_cast<int64_t>(p.tokens) * p.top_k;
  const MlpLayout l = mlp_layout(pairs, p.inner, p.d);
  if (p.workspace == nullptr || p.workspace_bytes < l.total) return GPTQ_ERR_WORKSPACE;
  uint8_t* ws = static_cast<uint8_t*>(p.workspace);
  const MlpArgs a{p.tokens, p.top_k, p.experts, p.d, p.inner, p.d / MXB, p.inner / MXB,
                  static_cast<const uint8_t*>(p.X), 2 * p.ldx, p.ids, p.weights, p.W1, p.s1, p.W2, p.s2, p.activation,
                  reinterpret_cast<uint16_t*>(ws), reinterpret_cast<float*>(ws + l.z),
                  reinterpret_cast<int32_t*>(ws + l.clean), reinterpret_cast<int*>(ws + l.done), p.out, p.ldo, 0};
  return p.bf16 ? launch_mlp<kMxBf16>(a, stream) : launch_mlp<kMxF16>(a, stream);
}

}  // namespace gptq

// How many waves share a tile's inputs in the first (up) or second launch, for tests that cover every form; not
// part of the interface.
extern "C" int gptq_internal_mxfp4_mlp_waves(int up, int pairs, int experts, int d, int inner) {
  return gptq::mlp_waves(up != 0, pairs, experts, d, inner);
}
