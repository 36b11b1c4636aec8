// Routing of tokens to experts, grouping of tokens by expert, and the sum of the experts'
// outputs (gfx950).
//
// "GPTQ Architecture, in depth", "Failure modes": each expert of a mixture-of-experts block
// sees only the tokens that the router sends it; the row ranges written here are those that the
// grouped Hessian and the grouped products take.
#include <algorithm>
#include <cmath>

#include "common.h"

namespace gptq {
namespace {

// ---------------------------------------------------------------------------- routing

struct RouteArgs {
  int64_t n_tokens;
  int E;
  const void* logits;
  int64_t ldl;
  const float* bias;
  int scoring, G, top_groups, group_score, k, renorm;
  float scale;
  int32_t* ids;
  float* weights;
};

// One wave per token, PER experts per lane (expert lane * PER + i), choice values in fp64:
// balance biases are multiples of a small step and 16-bit logits repeat, so that experts
// nearly equal in fp32 are common and their order would hang on the rounding of exp.
template <typename T, int PER>
__global__ __launch_bounds__(256) void route_kernel(RouteArgs a) {
  __shared__ double cs[4][64 * PER];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int64_t t = static_cast<int64_t>(blockIdx.x) * 4 + wave;
  if (t >= a.n_tokens) return;
  const T* row = static_cast<const T*>(a.logits) + t * a.ldl;
  const double ninf = -INFINITY;
  double l[PER], s[PER], c[PER];
  double m = ninf;
#pragma unroll
  for (int i = 0; i < PER; ++i) {
    const int e = lane * PER + i;
    const double v = e < a.E ? static_cast<double>(load_as_f32(row + e)) : ninf;
    l[i] = v == v ? v : ninf;
    m = fmax(m, l[i]);
  }
  for (int d = 32; d; d >>= 1) m = fmax(m, __shfl_xor(m, d));
  double sum = 0.0;
#pragma unroll
  for (int i = 0; i < PER; ++i) {
    if (a.scoring == 0) s[i] = l[i] == ninf ? 0.0 : l[i] == m ? 1.0 : exp(l[i] - m);
    else s[i] = l[i] == ninf ? 0.0 : 1.0 / (1.0 + exp(-l[i]));
    sum += s[i];
  }
  if (a.scoring == 0) {
    for (int d = 32; d; d >>= 1) sum += __shfl_xor(sum, d);
#pragma unroll
    for (int i = 0; i < PER; ++i) s[i] = sum > 0.0 ? s[i] / sum : 0.0;
  }
#pragma unroll
  for (int i = 0; i < PER; ++i) {
    const int e = lane * PER + i;
    c[i] = l[i];
    if (a.bias != nullptr && e < a.E && l[i] != ninf) {
      c[i] = s[i] + static_cast<double>(a.bias[e]);
      if (!(c[i] == c[i])) c[i] = ninf;
    }
  }
  if (a.top_groups < a.G) {
    const int per = a.E / a.G;
    const bool by_s = a.group_score == 1 && a.bias == nullptr;
#pragma unroll
    for (int i = 0; i < PER; ++i) cs[wave][lane * PER + i] = by_s ? (c[i] == ninf ? ninf : s[i]) : c[i];
    __builtin_amdgcn_wave_barrier();
    double rank = ninf;
    if (lane < a.G) {
      double b1 = ninf, b2 = ninf;
      for (int i = 0; i < per; ++i) {
        const double v = cs[wave][lane * per + i];
        if (v > b1) {
          b2 = b1;
          b1 = v;
        } else if (v > b2) {
          b2 = v;
        }
      }
      rank = a.group_score == 1 && b2 != ninf ? b1 + b2 : b1;
    }
    int better = 0;
    for (int g = 0; g < a.G; ++g) {
      const double o = __shfl(rank, g);
      better += o > rank || (o == rank && g < lane);
    }
    const uint64_t kept = __ballot(lane < a.G && better < a.top_groups);
#pragma unroll
    for (int i = 0; i < PER; ++i)
      if (!((kept >> min((lane * PER + i) / per, 63)) & 1)) c[i] = ninf;
  }
  // one choice after another
  double total = 0.0, mine = 0.0;
  int my_id = -1;
  for (int j = 0; j < a.k; ++j) {
    double best = ninf, bs = 0.0;
    int at = 1 << 20;
#pragma unroll
    for (int i = 0; i < PER; ++i)
      if (c[i] > best) {
        best = c[i];
        bs = s[i];
        at = lane * PER + i;
      }
    for (int d = 32; d; d >>= 1) {
      const double ob = __shfl_xor(best, d), os = __shfl_xor(bs, d);
      const int oa = __shfl_xor(at, d);
      if (ob > best || (ob == best && oa < at)) {
        best = ob;
        bs = os;
        at = oa;
      }
    }
    if (best == ninf) break;
#pragma unroll
    for (int i = 0; i < PER; ++i)
      if (lane * PER + i == at) c[i] = ninf;
    total += bs;
    if (lane == j) {
      mine = bs;
      my_id = at;
    }
  }
  if (lane < a.k) {
    double w = mine;
    if (a.renorm) w = total > 0.0 ? w / total : 0.0;
    a.ids[t * a.k + lane] = my_id;
    a.weights[t * a.k + lane] = static_cast<float>(w * static_cast<double>(a.scale));
  }
}

template <typename T>
gptq_status launch_route(const RouteArgs& a, hipStream_t stream) {
  const dim3 grid(static_cast<unsigned>((a.n_tokens + 3) / 4)), block(256);
  if (a.E <= 64) GPTQ_LAUNCH((route_kernel<T, 1>), grid, block, 0, stream, a);
  else if (a.E <= 256) GPTQ_LAUNCH((route_kernel<T, 4>), grid, block, 0, stream, a);
  else GPTQ_LAUNCH((route_kernel<T, 16>), grid, block, 0, stream, a);
  return GPTQ_OK;
}

// ---------------------------------------------------------------------------- grouping

constexpr int GR_WAVES = 8;
constexpr int GR_CHUNKS = 64;     // most chunks of slots
constexpr int GR_MIN = 1024;      // least slots per chunk

__global__ __launch_bounds__(512) void group_count_kernel(const int32_t* __restrict__ ids, int64_t slots, int chunk,
                                                          int E, int32_t* __restrict__ counts) {
  __shared__ int32_t h[1024];
  for (int e = threadIdx.x; e < E; e += 512) h[e] = 0;
  __syncthreads();
  const int64_t s0 = static_cast<int64_t>(blockIdx.x) * chunk;
  const int64_t s1 = min(slots, s0 + chunk);
  for (int64_t s = s0 + threadIdx.x; s < s1; s += 512) {
    const int id = ids[s];
    if (static_cast<unsigned>(id) < static_cast<unsigned>(E)) atomicAdd(&h[id], 1);
  }
  __syncthreads();
  for (int e = threadIdx.x; e < E; e += 512) counts[static_cast<int64_t>(blockIdx.x) * E + e] = h[e];
}

// One chunk of slots per workgroup, a contiguous eighth of it per wave.  A slot's position is
// the start of its expert + the expert's slots in earlier chunks + in earlier waves of this
// chunk + earlier in its wave (64 slots at a time: equal ids found by one ballot per bit).
__global__ __launch_bounds__(512) void group_place_kernel(const int32_t* __restrict__ ids, int64_t slots, int chunk,
                                                          int E, int k, const int32_t* __restrict__ counts,
                                                          int64_t* __restrict__ offsets,
                                                          int32_t* __restrict__ row_index,
                                                          int32_t* __restrict__ place) {
  __shared__ int32_t h[GR_WAVES][1024];
  __shared__ int32_t base[1024];
  __shared__ int32_t tot[1024];
  __shared__ int32_t wsum[GR_WAVES];
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int chunks = gridDim.x, me = blockIdx.x;
  const int64_t s0 = static_cast<int64_t>(me) * chunk;
  const int64_t s1 = min(slots, s0 + chunk);
  const int seg = chunk / GR_WAVES;   // a multiple of 64
  for (int i = tid; i < GR_WAVES * 1024; i += 512) (&h[0][0])[i] = 0;
  __syncthreads();
  const int64_t w0 = s0 + static_cast<int64_t>(wave) * seg, w1 = min(s1, w0 + seg);
  for (int64_t s = w0 + lane; s < w1; s += 64) {
    const int id = ids[s];
    if (static_cast<unsigned>(id) < static_cast<unsigned>(E)) atomicAdd(&h[wave][id], 1);
  }
  __syncthreads();
  for (int e = tid; e < 1024; e += 512) {
    int before = 0, all = 0;
    if (e < E) {
      if (chunks == 1) {
        for (int w = 0; w < GR_WAVES; ++w) all += h[w][e];
      } else {
        for (int c = 0; c < chunks; ++c) {
          const int n = counts[static_cast<int64_t>(c) * E + e];
          all += n;
          before += c < me ? n : 0;
        }
      }
    }
    base[e] = before;
    tot[e] = all;
  }
  __syncthreads();
  // exclusive sums of the totals: two neighbouring experts per thread
  const int x0 = tot[2 * tid], x1 = tot[2 * tid + 1];
  int inc = x0 + x1;
  for (int d = 1; d < 64; d <<= 1) {
    const int o = __shfl_up(inc, d);
    if (lane >= d) inc += o;
  }
  if (lane == 63) wsum[wave] = inc;
  __syncthreads();
  int lead = 0, total = 0;
  for (int w = 0; w < GR_WAVES; ++w) {
    lead += w < wave ? wsum[w] : 0;
    total += wsum[w];
  }
  const int start0 = lead + inc - x0 - x1, start1 = start0 + x0;
  base[2 * tid] += start0;
  base[2 * tid + 1] += start1;
  if (me == 0) {
    if (2 * tid < E) offsets[2 * tid] = start0;
    if (2 * tid + 1 < E) offsets[2 * tid + 1] = start1;
    if (tid == 0) offsets[E] = total;
  }
  __syncthreads();
  for (int e = tid; e < E; e += 512) {
    int run = base[e];
    for (int w = 0; w < GR_WAVES; ++w) {
      const int n = h[w][e];
      h[w][e] = run;
      run += n;
    }
  }
  __syncthreads();
  volatile int32_t* mine = h[wave];
  const int bits = 32 - __builtin_clz(E);
  for (int64_t b = w0; b < w1; b += 64) {
    const int64_t s = b + lane;
    const int id = s < w1 ? ids[s] : -1;
    const bool ok = static_cast<unsigned>(id) < static_cast<unsigned>(E);
    uint64_t same = __ballot(ok);
    for (int i = 0; i < bits; ++i) {
      const bool bit = (id >> i) & 1;
      const uint64_t with = __ballot(bit);
      same &= bit ? with : ~with;
    }
    if (ok) {
      const int rank = __popcll(same & ((1ull << lane) - 1));
      const int p = mine[id] + rank;
      row_index[p] = static_cast<int32_t>(s / k);
      place[s] = p;
      __builtin_amdgcn_wave_barrier();
      if (rank == 0) mine[id] = p + __popcll(same);
    } else if (s < w1) {
      place[s] = -1;
    }
    __builtin_amdgcn_wave_barrier();
  }
  for (int64_t s = s0 + tid; s < s1; s += 512)
    if (s >= total) row_index[s] = -1;
}

__global__ void group_none_kernel(int64_t* __restrict__ offsets, int n) {
  for (int i = threadIdx.x; i < n; i += 256) offsets[i] = 0;
}

int group_chunk(int64_t slots) {
  const int64_t c = std::max<int64_t>(GR_MIN, (slots + GR_CHUNKS - 1) / GR_CHUNKS);
  return static_cast<int>((c + 511) / 512 * 512);
}

// ---------------------------------------------------------------------------- combination

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

// One thread per V consecutive outputs of a token: V = 16 bytes where rows are aligned, else 1.
template <typename T, int V>
__global__ __launch_bounds__(256) void combine_kernel(int64_t n_tokens, int k, int64_t n_rows, int d, const T* Y,
                                                      int64_t ldy, const int32_t* place, const float* weights, T* out,
                                                      int64_t ldo) {
  const int per = (d + V - 1) / V;
  const int64_t i = static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x;
  const int64_t t = i / per;
  if (t >= n_tokens) return;
  const int64_t col = (i - t * per) * V;
  float acc[V];
#pragma unroll
  for (int v = 0; v < V; ++v) acc[v] = 0.0f;
  for (int j = 0; j < k; ++j) {
    const int p = place[t * k + j];
    if (p < 0 || p >= n_rows) continue;
    const float w = weights[t * k + j];
    const Vec<T, V> y = *reinterpret_cast<const Vec<T, V>*>(Y + p * ldy + col);
#pragma unroll
    for (int v = 0; v < V; ++v) acc[v] = fmaf(w, load_as_f32(&y.v[v]), acc[v]);
  }
  Vec<T, V> o;
#pragma unroll
  for (int v = 0; v < V; ++v) o.v[v] = from_f32<T>(acc[v]);
  *reinterpret_cast<Vec<T, V>*>(out + t * ldo + col) = o;
}

template <typename T>
gptq_status launch_combine(int64_t n_tokens, int k, int64_t n_rows, int d, const void* Y, int64_t ldy,
                           const int32_t* place, const float* weights, void* out, int64_t ldo, hipStream_t stream) {
  constexpr int V = 16 / sizeof(T);
  const bool wide = d % V == 0 && ldy % V == 0 && ldo % V == 0 && reinterpret_cast<uintptr_t>(Y) % 16 == 0 &&
                    reinterpret_cast<uintptr_t>(out) % 16 == 0;
  const int64_t n = n_tokens * (wide ? d / V : d);
  if ((n + 255) / 256 > INT32_MAX) return GPTQ_ERR_UNSUPPORTED;
  const dim3 grid(static_cast<unsigned>((n + 255) / 256)), block(256);
  if (wide)
    GPTQ_LAUNCH((combine_kernel<T, V>), grid, block, 0, stream, n_tokens, k, n_rows, d, static_cast<const T*>(Y), ldy,
                place, weights, static_cast<T*>(out), ldo);
  else
    GPTQ_LAUNCH((combine_kernel<T, 1>), grid, block, 0, stream, n_tokens, k, n_rows, d, static_cast<const T*>(Y), ldy,
                place, weights, static_cast<T*>(out), ldo);
  return GPTQ_OK;
}

}  // namespace

gptq_status route_enqueue(int64_t n_tokens, int n_experts, gptq_dtype l_dtype, const void* logits, int64_t ldl,
                          const float* bias, const gptq_route_params& p, int32_t* ids, float* weights,
                          hipStream_t stream) {
  RouteArgs a{};
  a.n_tokens = n_tokens; a.E = n_experts; a.logits = logits; a.ldl = ldl; a.bias = bias;
  a.scoring = p.scoring; a.G = p.n_groups; a.top_groups = p.top_groups; a.group_score = p.group_score;
  a.k = p.top_k; a.renorm = p.renormalize; a.scale = p.scale; a.ids = ids; a.weights = weights;
  if (l_dtype == GPTQ_F32) return launch_route<float>(a, stream);
  if (l_dtype == GPTQ_BF16) return launch_route<BF16>(a, stream);
  return launch_route<F16>(a, stream);
}

size_t group_workspace(int n_experts, int64_t slots) {
  const int chunk = group_chunk(slots);
  const int64_t chunks = (slots + chunk - 1) / chunk;
  return chunks > 1 ? static_cast<size_t>(chunks) * n_experts * sizeof(int32_t) : 256;
}

gptq_status group_enqueue(int64_t n_tokens, int top_k, int n_experts, const int32_t* ids, int64_t* token_offsets,
                          int32_t* row_index, int32_t* place, void* ws, size_t ws_bytes, hipStream_t stream) {
  const int64_t slots = n_tokens * top_k;
  if (slots == 0) {
    GPTQ_LAUNCH(group_none_kernel, dim3(1), dim3(256), 0, stream, token_offsets, n_experts + 1);
    return GPTQ_OK;
  }
  const int chunk = group_chunk(slots);
  const int chunks = static_cast<int>((slots + chunk - 1) / chunk);
  if (chunks > 1 && (ws == nullptr || ws_bytes < group_workspace(n_experts, slots))) return GPTQ_ERR_WORKSPACE;
  int32_t* counts = static_cast<int32_t*>(ws);
  if (chunks > 1)
    GPTQ_LAUNCH(group_count_kernel, dim3(chunks), dim3(512), 0, stream, ids, slots, chunk, n_experts, counts);
  GPTQ_LAUNCH(group_place_kernel, dim3(chunks), dim3(512), 0, stream, ids, slots, chunk, n_experts, top_k, counts,
              token_offsets, row_index, place);
  return GPTQ_OK;
}

gptq_status combine_enqueue(int64_t n_tokens, int top_k, int64_t n_rows, int d, gptq_dtype y_dtype, const void* Y,
                            int64_t ldy, const int32_t* place, const float* weights, void* out, int64_t ldo,
                            hipStream_t stream) {
  if (y_dtype == GPTQ_F32)
    return launch_combine<float>(n_tokens, top_k, n_rows, d, Y, ldy, place, weights, out, ldo, stream);
  if (y_dtype == GPTQ_BF16)
    return launch_combine<BF16>(n_tokens, top_k, n_rows, d, Y, ldy, place, weights, out, ldo, stream);
  return launch_combine<F16>(n_tokens, top_k, n_rows, d, Y, ldy, place, weights, out, ldo, stream);
}

}  // namespace gptq
