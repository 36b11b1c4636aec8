// The expert layer of a mixture-of-experts block for few tokens on gfx950, in two launches:
//
//   out[t, :] = sum_j weights[t, j] W2[e] (act(G[e] x_t) * U[e] x_t),   e = ids[t, j]
//
// with W1[e] = [G[e]; U[e]] and W2[e] in the 4-bit microscaled form and 16-bit x.  Both kernels are
// bound by reading the weights of the experts that some token chose, each once; the weights become
// bf16 in registers, exactly, in front of v_mfma_f32_16x16x32_bf16, as the first operand, with
// tokens as the columns of the second.  The activations between the kernels carry the routing
// weight and are two bf16 planes (the value and the rest, 16 bits together): one plane would add
// an error like the output's own rounding, and the matrix cores are idle anyway.
#include <algorithm>
#include <cfloat>

#include "mx.h"

namespace gptq {
namespace {

constexpr int MLP_EXPERTS = 1024;   // most experts

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
  void* out;
  int64_t ldo;
};

enum MlpAct { kSilu = 0, kGeluTanh = 1 };
__device__ __forceinline__ float mlp_act(float g, int act) {
  // 0.5 g (1 + tanh z) = g / (1 + exp(-2 z)), z = sqrt(2 / pi) (g + 0.044715 g^3)
  const float z = act == kSilu ? g : 1.5957691216057308f * (g + 0.044715f * g * g * g);
  return g / (1.0f + expf(-z));
}

// The experts that a workgroup's choices name, as a bit each.  All threads call it, with a barrier
// before and after the counting.
struct Chosen {
  uint32_t words[MLP_EXPERTS / 32];
};
template <int NT>
__device__ __forceinline__ void mark_chosen(Chosen& c, int16_t* ids, const int32_t* from, int n, int experts) {
  for (int i = threadIdx.x; i < MLP_EXPERTS / 32; i += NT) c.words[i] = 0;
  __syncthreads();
  for (int i = threadIdx.x; i < n; i += NT) {
    const int e = from[i];
    const bool ok = e >= 0 && e < experts;
    ids[i] = static_cast<int16_t>(ok ? e : -1);
    if (ok) atomicOr(&c.words[e >> 5], 1u << (e & 31));
  }
  __syncthreads();
}
// The slot-th of them in ascending order, -1 behind the last (in every lane).
__device__ __forceinline__ int nth_chosen(const Chosen& c, int slot) {
  const int lane = threadIdx.x & 63;
  uint32_t w = lane < MLP_EXPERTS / 32 ? c.words[lane] : 0;
  const int own = __popc(w);
  int inc = own;
  for (int d = 1; d < 32; d <<= 1) {
    const int o = __shfl_up(inc, d);
    if (lane >= d) inc += o;
  }
  const uint64_t past = __ballot(lane < MLP_EXPERTS / 32 && inc > slot);
  if (past == 0) return -1;
  const int l = __builtin_ctzll(past);
  uint32_t v = static_cast<uint32_t>(__shfl(static_cast<int>(w), l));
  for (int skip = slot - __shfl(inc - own, l); skip > 0; --skip) v &= v - 1;
  return uniform(32 * l + __builtin_ctz(v));
}

// A token that names an expert twice takes it once, at its first choice, with both weights.
__device__ __forceinline__ bool first_choice(const int16_t* ids, int i, int top_k) {
  for (int k = i / top_k * top_k; k < i; ++k)
    if (ids[k] == ids[i]) return false;
  return true;
}

// Gate and up products: workgroup (slot, tile) makes 16 inner values of all tokens of the slot-th
// chosen expert.  Four waves take every fourth pair of chunks of 128 inputs straight from memory to
// registers, a block of 32 per lane, chunk and matrix, 4 chunks in flight; their sums meet in LDS.
constexpr int UP_NW = 4;
template <int KIND>
__global__ __launch_bounds__(UP_NW * 64) void mlp_up_kernel(MlpArgs a) {
  constexpr int U = 4, FM = 2;
  extern __shared__ int16_t mlp_ids[];   // [pairs] ids, then the expert's list of pairs [tokens]
  __shared__ Chosen chosen;
  __shared__ __attribute__((aligned(16))) float part[UP_NW][2][16 * FM][16];
  __shared__ int listed;
  const int tid = threadIdx.x, lane = tid & 63, wk = uniform(tid >> 6);
  const int tiles = a.inner / 16, pairs = a.tokens * a.top_k;
  const int slot = blockIdx.x / tiles, n0 = (blockIdx.x - slot * tiles) * 16;
  int16_t* const list = mlp_ids + pairs;
  mark_chosen<UP_NW * 64>(chosen, mlp_ids, a.ids, pairs, a.experts);
  const int e = nth_chosen(chosen, slot);
  if (e < 0) return;
  const int j = lane & 15, q = lane >> 4;
  const uint8_t* zeros = reinterpret_cast<const uint8_t*>(&zero16);
  const int64_t row0 = static_cast<int64_t>(e) * 2 * a.inner + n0 + j;
  const uint8_t* w[2];
  const uint8_t* ws[2];
#pragma unroll
  for (int g = 0; g < 2; ++g) {
    w[g] = a.W1 + (row0 + g * a.inner) * (a.d / 2);
    ws[g] = a.s1 + (row0 + g * a.inner) * a.kb1;
  }
  const int chunks = (a.kb1 + 3) / 4;
  auto chunk = [&](int g, int u) { return 2 * (wk + UP_NW * (g + u / 2)) + (u & 1); };
  i32x4 wv[U][2];
  uint32_t sw[U][2];
  auto load = [&](int u, int c) {
    const int b = 4 * c + q;
    const bool in = b < a.kb1;
#pragma unroll
    for (int g = 0; g < 2; ++g) {
      wv[u][g] = *reinterpret_cast<const i32x4*>(in ? w[g] + 16 * b : zeros);
      sw[u][g] = in ? ws[g][b] : 127u;
    }
  };
  auto begin = [&] {
#pragma unroll
    for (int u = 0; u < U; ++u)
      if (chunk(0, u) < chunks) load(u, chunk(0, u));
  };
  begin();
  // the expert's pairs, in order, while the first weights are on the way
  if (wk == 0) {
    int n = 0;
    for (int i0 = 0; i0 < pairs; i0 += 64) {
      const int i = i0 + lane;
      const bool mine = i < pairs && mlp_ids[i] == e && first_choice(mlp_ids, i, a.top_k);
      const uint64_t all = __ballot(mine);
      if (mine) list[n + __popcll(all & ((1ull << lane) - 1))] = static_cast<int16_t>(i);
      n += __popcll(all);
    }
    if (lane == 0) listed = n;
  }
  __syncthreads();
  const int count = listed;

  auto tokens = [&](int r0, auto kFm) {
    constexpr int F = kFm;
    const uint8_t* x[F];
    bool have[F];
#pragma unroll
    for (int i = 0; i < F; ++i) {
      const int r = r0 + 16 * i + j;
      have[i] = r < count;
      x[i] = a.X + static_cast<int64_t>(list[min(r, count - 1)] / a.top_k) * a.ldx;
    }
    f32x4 y[2][F];
#pragma unroll
    for (int g = 0; g < 2; ++g)
#pragma unroll
      for (int i = 0; i < F; ++i) y[g][i] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
    for (int g0 = 0; chunk(g0, 0) < chunks; g0 += U / 2) {
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int c = chunk(g0, u);
        if (c < chunks) {
          const int b = 4 * c + q;
          i32x4 xv[F][4];
#pragma unroll
          for (int i = 0; i < F; ++i)
#pragma unroll
            for (int p = 0; p < 4; ++p)
              __builtin_memcpy(&xv[i][p], have[i] && b < a.kb1 ? x[i] + 64 * b + 16 * p : zeros, 16);
#pragma unroll
          for (int p = 0; p < 4; ++p) {
            const bf16x8 gate = mx_bf16(static_cast<uint32_t>(wv[u][0][p]), sw[u][0]);
            const bf16x8 up = mx_bf16(static_cast<uint32_t>(wv[u][1][p]), sw[u][1]);
#pragma unroll
            for (int i = 0; i < F; ++i) {
              const XValues<KIND> v(xv[i][p]);
              y[0][i] = mx_mma16<KIND>(gate, v, y[0][i]);
              y[1][i] = mx_mma16<KIND>(up, v, y[1][i]);
            }
          }
          if (chunk(g0 + U / 2, u) < chunks) load(u, chunk(g0 + U / 2, u));
        }
      }
    }
    if (r0 > 0) __syncthreads();   // the tile before has been read
#pragma unroll
    for (int g = 0; g < 2; ++g)
#pragma unroll
      for (int i = 0; i < F; ++i) *reinterpret_cast<f32x4*>(&part[wk][g][16 * i + j][4 * q]) = y[g][i];
    __syncthreads();
    const int rows = min(16 * F, count - r0);
    for (int t = tid; t < rows * 4; t += UP_NW * 64) {
      const int c = t & 3, r = t >> 2, p = list[r0 + r];
      f32x4 v[2] = {{0.0f, 0.0f, 0.0f, 0.0f}, {0.0f, 0.0f, 0.0f, 0.0f}};
#pragma unroll
      for (int h = 0; h < UP_NW; ++h)
#pragma unroll
        for (int g = 0; g < 2; ++g) v[g] += *reinterpret_cast<const f32x4*>(&part[h][g][r][4 * c]);
      float weight = 0.0f;
      for (int k = p, end = (p / a.top_k + 1) * a.top_k; k < end; ++k)
        if (mlp_ids[k] == e) weight += a.weights[k];
      Vec<BF16, 4> hi, lo;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float h = weight * (mlp_act(v[0][i], a.act) * v[1][i]);
        hi.v[i] = from_f32<BF16>(h);
        const float near = bf16_to_f32(hi.v[i].bits);
        lo.v[i] = from_f32<BF16>(fabsf(near) <= FLT_MAX ? h - near : 0.0f);   // an infinity has no rest
      }
      uint16_t* to = a.H + static_cast<int64_t>(p) * a.inner + n0 + 4 * c;
      *reinterpret_cast<Vec<BF16, 4>*>(to) = hi;
      *reinterpret_cast<Vec<BF16, 4>*>(to + static_cast<int64_t>(pairs) * a.inner) = lo;
    }
  };
  for (int r0 = 0; r0 < count;) {
    if (r0 > 0) begin();
    if (count - r0 <= 16) {
      tokens(r0, std::integral_constant<int, 1>{});
      r0 += 16;
    } else {
      tokens(r0, std::integral_constant<int, FM>{});
      r0 += 16 * FM;
    }
  }
}

// Down products and the sum over a token's experts: workgroup (tile, group) makes 16 outputs of 16 TT
// tokens, over all experts that these chose.  A column of the second operand is a token, whichever
// expert is at hand, so that the sum over experts stays in the registers; where the token did
// not choose the expert its column is left out of the sum (not multiplied by 0: the expert's weights
// may hold a NaN).  Items of one expert's 256 inner values go to the NW waves in turn, two in
// flight per wave; the waves' sums meet in LDS and are added in wave order.
constexpr int DOWN_NW = 16;
template <typename T, int TT>
__global__ __launch_bounds__(DOWN_NW * 64) void mlp_down_kernel(MlpArgs a) {
  constexpr int NW = DOWN_NW, D = 2, TG = 16 * TT;
  extern __shared__ __attribute__((aligned(16))) uint8_t mlp_lds[];
  __shared__ Chosen chosen;
  __shared__ int before[MLP_EXPERTS / 32 + 1];   // chosen experts before a word
  const int tid = threadIdx.x, lane = tid & 63, wave = uniform(tid >> 6);
  const int n0 = blockIdx.x * 16, t0 = blockIdx.y * TG, mine = min(TG, a.tokens - t0);
  const int n = mine * a.top_k, first = t0 * a.top_k, pairs = a.tokens * a.top_k;
  // ids of the group, the chosen experts in order, their tokens' pairs + 1 [chosen][TG]; the sums
  // take the place of all of them
  int16_t* const ids = reinterpret_cast<int16_t*>(mlp_lds);
  const int most = min(a.experts, n);
  int16_t* const expert = ids + (n + 7) / 8 * 8;
  uint16_t* const table = reinterpret_cast<uint16_t*>(expert + (most + 7) / 8 * 8);
  mark_chosen<NW * 64>(chosen, ids, a.ids + first, n, a.experts);
  if (tid < 64) {
    const int own = lane < MLP_EXPERTS / 32 ? __popc(chosen.words[lane]) : 0;
    int inc = own;
    for (int d = 1; d < 64; d <<= 1) {
      const int o = __shfl_up(inc, d);
      if (lane >= d) inc += o;
    }
    if (lane <= MLP_EXPERTS / 32) before[lane] = inc - own;
  }
  __syncthreads();
  const int used = before[MLP_EXPERTS / 32];
  for (int i = tid; i < used * TG / 2; i += NW * 64) reinterpret_cast<uint32_t*>(table)[i] = 0;
  __syncthreads();
  for (int i = tid; i < n; i += NW * 64) {
    const int e = ids[i];
    if (e < 0 || !first_choice(ids, i, a.top_k)) continue;
    const int r = before[e >> 5] + __popc(chosen.words[e >> 5] & ((1u << (e & 31)) - 1));
    expert[r] = static_cast<int16_t>(e);
    table[r * TG + i / a.top_k] = static_cast<uint16_t>(first + i + 1);
  }
  __syncthreads();

  const int j = lane & 15, q = lane >> 4;
  const uint8_t* zeros = reinterpret_cast<const uint8_t*>(&zero16);
  const int per = (a.kb2 + 7) / 8, items = used * per;   // items of 8 blocks
  i32x4 wv[D][2];
  uint32_t sw[D][2];
  auto load = [&](int u, int item) {
    const int r = item / per;
    const int64_t row = static_cast<int64_t>(uniform(static_cast<int>(expert[r]))) * a.d + n0 + j;
    const uint8_t* w = a.W2 + row * (a.inner / 2);
    const uint8_t* ws = a.s2 + row * a.kb2;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int b = 8 * (item - r * per) + 4 * h + q;
      const bool in = b < a.kb2;
      wv[u][h] = *reinterpret_cast<const i32x4*>(in ? w + 16 * b : zeros);
      sw[u][h] = in ? ws[b] : 127u;
    }
  };
  f32x4 y[TT];
#pragma unroll
  for (int t = 0; t < TT; ++t) y[t] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
  auto multiply = [&](int u, int item) {
    const int r = item / per;
    bf16x8 wf[2][4];
#pragma unroll
    for (int h = 0; h < 2; ++h)
#pragma unroll
      for (int p = 0; p < 4; ++p) wf[h][p] = mx_bf16(static_cast<uint32_t>(wv[u][h][p]), sw[u][h]);
#pragma unroll
    for (int t = 0; t < TT; ++t) {
      const int pair = table[r * TG + 16 * t + j];
      if (__ballot(pair != 0) == 0) continue;
      const uint16_t* x = a.H + static_cast<int64_t>(max(pair - 1, 0)) * a.inner;
      f32x4 s = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const int b = 8 * (item - r * per) + 4 * h + q;
        const bool ok = pair != 0 && b < a.kb2;
        const uint8_t* hi = ok ? reinterpret_cast<const uint8_t*>(x + 32 * b) : zeros;
        const uint8_t* lo = ok ? reinterpret_cast<const uint8_t*>(x + static_cast<int64_t>(pairs) * a.inner + 32 * b) : zeros;
        const int step = ok ? 16 : 0;
        i32x4 xh[4], xl[4];
#pragma unroll
        for (int p = 0; p < 4; ++p) {
          xh[p] = *reinterpret_cast<const i32x4*>(hi + step * p);
          xl[p] = *reinterpret_cast<const i32x4*>(lo + step * p);
        }
#pragma unroll
        for (int p = 0; p < 4; ++p) {
          s = __builtin_amdgcn_mfma_f32_16x16x32_bf16(wf[h][p], __builtin_bit_cast(bf16x8, xl[p]), s, 0, 0, 0);
          s = __builtin_amdgcn_mfma_f32_16x16x32_bf16(wf[h][p], __builtin_bit_cast(bf16x8, xh[p]), s, 0, 0, 0);
        }
      }
#pragma unroll
      for (int i = 0; i < 4; ++i) y[t][i] += pair != 0 ? s[i] : 0.0f;
    }
  };
#pragma unroll
  for (int u = 0; u < D; ++u)
    if (wave + NW * u < items) load(u, wave + NW * u);
  for (int i = wave; i < items; i += NW * D) {
#pragma unroll
    for (int u = 0; u < D; ++u) {
      const int item = i + NW * u;
      if (item < items) {
        multiply(u, item);
        if (item + NW * D < items) load(u, item + NW * D);
      }
    }
  }
  __syncthreads();   // the table is done with
  float* const part = reinterpret_cast<float*>(mlp_lds);   // [NW][TG][16]
#pragma unroll
  for (int t = 0; t < TT; ++t) *reinterpret_cast<f32x4*>(&part[((wave * TG) + 16 * t + j) * 16 + 4 * q]) = y[t];
  __syncthreads();
  for (int g = tid; g < mine * 4; g += NW * 64) {
    const int c = g & 3, r = g >> 2;
    f32x4 v = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
    for (int h = 0; h < NW; ++h) v += *reinterpret_cast<const f32x4*>(&part[(h * TG + r) * 16 + 4 * c]);
    Vec<T, 4> o;
#pragma unroll
    for (int i = 0; i < 4; ++i) o.v[i] = from_f32<T>(v[i]);
    __builtin_memcpy(static_cast<T*>(a.out) + (t0 + r) * a.ldo + n0 + 4 * c, &o, sizeof(o));
  }
}

// LDS of the down kernel: its tables, then the waves' sums.
size_t down_lds(int tokens, int top_k, int experts, int tg) {
  const int n = std::min(tokens, tg) * top_k, most = std::min(experts, n);
  const size_t table = 2 * (static_cast<size_t>((n + 7) / 8 * 8) + (most + 7) / 8 * 8 + static_cast<size_t>(most) * tg);
  return std::max(table, static_cast<size_t>(DOWN_NW) * tg * 16 * sizeof(float));
}

template <typename T, int TT>
gptq_status launch_down(const MlpArgs& a, hipStream_t stream) {
  constexpr int TG = 16 * TT;
  GPTQ_LAUNCH((mlp_down_kernel<T, TT>), dim3(a.d / 16, (a.tokens + TG - 1) / TG), dim3(DOWN_NW * 64),
              down_lds(a.tokens, a.top_k, a.experts, TG), stream, a);
  return GPTQ_OK;
}

template <int KIND, typename T>
gptq_status launch_mlp(const MlpArgs& a, hipStream_t stream) {
  const int pairs = a.tokens * a.top_k, slots = std::min(a.experts, pairs);
  GPTQ_LAUNCH(mlp_up_kernel<KIND>, dim3(static_cast<unsigned>(slots) * (a.inner / 16)), dim3(UP_NW * 64),
              2 * static_cast<size_t>(pairs + a.tokens), stream, a);
  if (a.tokens <= 16) return launch_down<T, 1>(a, stream);
  if (a.tokens <= 32) return launch_down<T, 2>(a, stream);
  return launch_down<T, 4>(a, stream);
}

}  // namespace

size_t mx_mlp_workspace(int64_t pairs, int inner) {
  return 512 + align_up(4 * static_cast<size_t>(pairs) * inner, 256);   // above 256, which says that nothing is kept
}

gptq_status mx_mlp_enqueue(const MxMlp& p, hipStream_t stream) {
  const int64_t pairs = static_cast<int64_t>(p.tokens) * p.top_k;
  if (p.workspace == nullptr || p.workspace_bytes < mx_mlp_workspace(pairs, p.inner)) return GPTQ_ERR_WORKSPACE;
  if (std::min<int64_t>(p.experts, pairs) * (p.inner / 16) > INT32_MAX) return GPTQ_ERR_UNSUPPORTED;
  const MlpArgs a{p.tokens, p.top_k, p.experts, p.d, p.inner, p.d / MXB, p.inner / MXB,
                  static_cast<const uint8_t*>(p.X), 2 * p.ldx, p.ids, p.weights, p.W1, p.s1, p.W2, p.s2, p.activation,
                  static_cast<uint16_t*>(p.workspace), p.out, p.ldo};
  return p.bf16 ? launch_mlp<kMxBf16, BF16>(a, stream) : launch_mlp<kMxF16, F16>(a, stream);
}

}  // namespace gptq
