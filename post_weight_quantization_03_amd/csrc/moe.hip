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
  int batch;   // route_kernel: tokens per wave and turn, 1, 2 or 4
  int per, each, log_lanes;   // route_rows_kernel: experts per group and per lane, log2 of lanes per group
  bool exact;                 // and whether that is all experts, each once
};

// fp32 as integers in the same order (-0 as +0), which maxima over lanes take in one
// instruction each.
constexpr uint32_t kKeyNone = 0x007FFFFFu;   // of -inf
__device__ __forceinline__ uint32_t key_of(float v) {
  const int b = __float_as_int(v + 0.0f);
  return static_cast<uint32_t>(b) ^ (static_cast<uint32_t>(b >> 31) | 0x80000000u);
}
__device__ __forceinline__ float of_key(uint32_t k) {
  return __uint_as_float(k ^ (k >> 31 ? 0x80000000u : 0xFFFFFFFFu));
}
template <int CTRL>
__device__ __forceinline__ uint32_t moved(uint32_t v) {
  return static_cast<uint32_t>(__builtin_amdgcn_update_dpp(0, static_cast<int>(v), CTRL, 0xF, 0xF, false));
}
// The largest key of the wave, in a scalar register: row_shr 1, 2, 4, 8, then each row's last
// lane to the next row (0x142) and the first half's to the second (0x143); lane 63 has all.
__device__ __forceinline__ uint32_t wave_max(uint32_t v) {
  v = max(v, moved<0x111>(v));
  v = max(v, moved<0x112>(v));
  v = max(v, moved<0x114>(v));
  v = max(v, moved<0x118>(v));
  v = max(v, moved<0x142>(v));
  v = max(v, moved<0x143>(v));
  return static_cast<uint32_t>(__builtin_amdgcn_readlane(static_cast<int>(v), 63));
}
__device__ __forceinline__ double lane_value(double v, int lane) {
  const int64_t b = __double_as_longlong(v);
  const uint32_t lo = __builtin_amdgcn_readlane(static_cast<int>(b), lane);
  const uint32_t hi = __builtin_amdgcn_readlane(static_cast<int>(b >> 32), lane);
  return __longlong_as_double(static_cast<int64_t>(static_cast<uint64_t>(hi) << 32 | lo));
}
// Over the 16 lanes of a row, in all of them: rotations by 1, 2, 4 and 8.
__device__ __forceinline__ uint32_t row_max(uint32_t v) {
  v = max(v, moved<0x121>(v));
  v = max(v, moved<0x122>(v));
  v = max(v, moved<0x124>(v));
  return max(v, moved<0x128>(v));
}
template <int CTRL>
__device__ __forceinline__ double moved(double v) {
  const int64_t b = __double_as_longlong(v);
  const uint32_t lo = moved<CTRL>(static_cast<uint32_t>(b)), hi = moved<CTRL>(static_cast<uint32_t>(b >> 32));
  return __longlong_as_double(static_cast<int64_t>(static_cast<uint64_t>(hi) << 32 | lo));
}
__device__ __forceinline__ double row_sum(double v) {
  v += moved<0x121>(v);
  v += moved<0x122>(v);
  v += moved<0x124>(v);
  return v + moved<0x128>(v);
}
__device__ __forceinline__ double lanes_sum(double v, int lanes) {   // over runs of `lanes` lanes
  for (int d = lanes / 2; d; d >>= 1) v += __shfl_xor(v, d);
  return v;
}

// exp(x), x in [-150, 150]: 2^(x log2 e) with the product's error carried along, within 2 fp32
// roundings.
__device__ __forceinline__ float exp_f32(float x) {
  const float l2e = 0x1.715476p+0f, l2e_lo = 0x1.4ae0c0p-26f;   // log2 e and what fp32 leaves of it
  const float p = x * l2e;
  const float r = fmaf(x, l2e, -p) + x * l2e_lo;
  const float e = __builtin_amdgcn_exp2f(p);
  return isinf(e) ? e : fmaf(e, r * 0x1.62e43p-1f, e);
}

// One token by one wave in fp64 (expert lane * PER + i): the definition itself.
template <typename T, int PER>
__device__ __forceinline__ void route_exact(const RouteArgs& a, int64_t t, double* cs) {
  const int lane = threadIdx.x & 63;
  const T* row = static_cast<const T*>(a.logits) + t * a.ldl;
  const double ninf = -INFINITY;
  double l[PER], s[PER], c[PER];
#pragma unroll
  for (int i = 0; i < PER; ++i) {
    const int e = lane * PER + i;
    const double v = e < a.E ? static_cast<double>(load_as_f32(row + e)) : ninf;
    l[i] = v == v ? v : ninf;
  }
  if (a.scoring == 0) {
    uint32_t k = key_of(static_cast<float>(l[0]));   // logits are fp32 values
#pragma unroll
    for (int i = 1; i < PER; ++i) k = max(k, key_of(static_cast<float>(l[i])));
    const double m = static_cast<double>(of_key(wave_max(k)));
    double sum = 0.0;
#pragma unroll
    for (int i = 0; i < PER; ++i) {
      s[i] = exp(l[i] == ninf ? -800.0 : l[i] == m ? 0.0 : fmax(l[i] - m, -800.0));   // exp(-800) is 0
      sum += s[i];
    }
    sum = row_sum(sum);
    sum = lane_value(sum, 0) + lane_value(sum, 16) + (lane_value(sum, 32) + lane_value(sum, 48));
#pragma unroll
    for (int i = 0; i < PER; ++i) s[i] = sum > 0.0 ? s[i] / sum : 0.0;
  } else {
#pragma unroll
    for (int i = 0; i < PER; ++i) s[i] = 1.0 / (1.0 + exp(l[i] == ninf ? 800.0 : -l[i]));
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
    for (int i = 0; i < PER; ++i) cs[lane * PER + i] = by_s ? (c[i] == ninf ? ninf : s[i]) : c[i];
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    double rank = ninf;
    if (lane < a.G) {
      double b1 = ninf, b2 = ninf;
#pragma unroll 8
      for (int i = 0; i < per; ++i) {
        const double v = cs[lane * per + i];
        b2 = fmax(b2, fmin(b1, v));
        b1 = fmax(b1, v);
      }
      rank = a.group_score == 1 && b2 != ninf ? b1 + b2 : b1;
    }
    int better = 0;
    for (int g = 0; g < a.G; ++g) {
      const double o = lane_value(rank, g);
      better += o > rank || (o == rank && g < lane);
    }
    const uint64_t kept = __ballot(lane < a.G && better < a.top_groups);
#pragma unroll
    for (int i = 0; i < PER; ++i)
      if (!((kept >> min((lane * PER + i) / per, 63)) & 1)) c[i] = ninf;
  }
  // one choice after another: the largest high half of the keys, then the largest low half
  // of those; the lowest lane that has both holds the lowest index
  double total = 0.0, mine = 0.0;
  int my_id = -1;
  for (int j = 0; j < a.k; ++j) {
    double best = c[0], bs = s[0];
    int at = 0;
#pragma unroll
    for (int i = 1; i < PER; ++i)
      if (c[i] > best) {
        best = c[i];
        bs = s[i];
        at = i;
      }
    const uint64_t bits = static_cast<uint64_t>(__double_as_longlong(best + 0.0));
    const uint64_t key = bits ^ (static_cast<uint64_t>(static_cast<int64_t>(bits) >> 63) | 0x8000000000000000ull);
    const uint32_t hi = static_cast<uint32_t>(key >> 32), lo = static_cast<uint32_t>(key);
    const uint32_t mh = wave_max(hi), ml = wave_max(hi == mh ? lo : 0u);
    const int owner = __builtin_ctzll(__ballot(hi == mh && lo == ml));
    if (lane_value(best, owner) == ninf) break;
    const int e = __builtin_amdgcn_readlane(lane * PER + at, owner);
    const double se = lane_value(bs, owner);
#pragma unroll
    for (int i = 0; i < PER; ++i)
      if (lane * PER + i == e) c[i] = ninf;
    total += se;
    if (lane == j) {
      mine = se;
      my_id = e;
    }
  }
  if (lane < a.k) {
    double w = mine;
    if (a.renorm) w = total > 0.0 ? w / total : 0.0;
    a.ids[t * a.k + lane] = my_id;
    a.weights[t * a.k + lane] = static_cast<float>(w * static_cast<double>(a.scale));
  }
}

// One token at a time per wave, PER neighbouring experts per lane, sorted in the lane: a choice
// is one maximum over the lanes' first keys, and the lane it came from moves up its next.
// Choices are made on fp32 values whose error is bounded, and a token is done again in fp64
// (route_exact) where two values that its choice hangs on are nearer than that: balance biases
// are multiples of a small step and 16-bit logits repeat, so near values are common among many
// experts, and their order must not hang on the rounding of exp.  Scores are within 6 roundings
// of 2^-24, so two choice values within 2^-20 (relative to the larger, or to 1) of each other
// may be in either order; the check takes 2^-19, and 2^-18 for sums of two.  Experts with the
// same logit and bias are in index order in either form.  Without a bias the logits themselves
// are compared, which is exact.
// Weights are worked out in fp64 and rounded once, those of `batch` tokens together, one choice per
// lane.  The sum under a softmax is of fp32 exponentials, added in fp64: a weight that is not divided
// by the sum of the chosen ones was at most 1.3 * 2^-24 off (131072 of 64 to 384 experts; with fp64
// exponentials 1.0, and 16384 tokens of 256 experts took route_rows_kernel 12.3 us instead of 9.1).
// Bound by vector issue.
template <typename T, int PER>
__global__ __launch_bounds__(256) void route_kernel(RouteArgs a) {
  __shared__ double scratch[4][64 * PER];   // route_exact's, or choice values in fp32
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const float ninf = -INFINITY;
  const int per = a.E / a.G;
  const bool softmax = a.scoring == 0, biased = a.bias != nullptr, grouped = a.top_groups < a.G;
  const bool by_s = grouped && a.group_score == 1 && !biased;   // groups by scores, experts by logits
  const bool whole = per % PER == 0 && !by_s;                   // a lane's experts are of one group
  float* cs = reinterpret_cast<float*>(scratch[wave]);
  float bias[PER];
#pragma unroll
  for (int i = 0; i < PER; ++i) bias[i] = biased && lane * PER + i < a.E ? a.bias[lane * PER + i] : 0.0f;
  const int my_group = min(lane * PER / per, 63);
  const int seg = 64 / a.batch;   // lanes of one token's choices at the end

  for (int64_t t0 = (static_cast<int64_t>(blockIdx.x) * 4 + wave) * a.batch; t0 < a.n_tokens;
       t0 += static_cast<int64_t>(gridDim.x) * 4 * a.batch) {
    int my_id = -1;                  // choice lane % seg of token t0 + lane / seg
    float my_max = 0.0f;
    double my_total = 0.0;
    bool done = true;                // that token needs no weights here
    // the next token's logits are in flight while one is worked on
    T raw[PER];
    auto fetch = [&](int64_t t) {
      const T* row = static_cast<const T*>(a.logits) + t * a.ldl;
#pragma unroll
      for (int i = 0; i < PER; ++i)
        if (lane * PER + i < a.E) raw[i] = row[lane * PER + i];
    };
    fetch(t0);
    for (int tt = 0; tt < a.batch && t0 + tt < a.n_tokens; ++tt) {
      const T* row = static_cast<const T*>(a.logits) + (t0 + tt) * a.ldl;
      float l[PER], c[PER], m = ninf;
#pragma unroll
      for (int i = 0; i < PER; ++i) {
        const float v = lane * PER + i < a.E ? load_as_f32(&raw[i]) : ninf;
        l[i] = v == v ? v : ninf;
        c[i] = l[i];
      }
      if (tt + 1 < a.batch && t0 + tt + 1 < a.n_tokens) fetch(t0 + tt + 1);
      double total = 0.0;   // softmax: the sum of exp(l - m)
      if (softmax) {
        uint32_t k = key_of(l[0]);
#pragma unroll
        for (int i = 1; i < PER; ++i) k = max(k, key_of(l[i]));
        m = of_key(wave_max(k));
#pragma unroll
        for (int i = 0; i < PER; ++i) {
          c[i] = l[i] == ninf ? 0.0f : exp_f32(l[i] == m ? 0.0f : fmaxf(l[i] - m, -150.0f));
          total += static_cast<double>(c[i]);
        }
        total = row_sum(total);
        total = lane_value(total, 0) + lane_value(total, 16) + (lane_value(total, 32) + lane_value(total, 48));
      }
      if (biased || by_s) {
        const float r = softmax && total > 0.0 ? __builtin_amdgcn_rcpf(static_cast<float>(total)) : 0.0f;
#pragma unroll
        for (int i = 0; i < PER; ++i) {
          // sigmoid: the exponent's rounding moves s by s (1 - s) |l| 2^-24, under a third of a step
          const float s = softmax ? c[i] * r
                                  : __builtin_amdgcn_rcpf(1.0f + __builtin_amdgcn_exp2f(l[i] * -0x1.715476p+0f));
          const float v = s + bias[i];
          c[i] = l[i] == ninf || !(v == v) ? ninf : v;
        }
      } else {
#pragma unroll
        for (int i = 0; i < PER; ++i) c[i] = l[i];
      }

      bool near = false;
      uint64_t kept = ~0ull;
      uint32_t key[PER];
      int at[PER];   // expert of each key
      auto sort_lane = [&] {
#pragma unroll
        for (int i = 0; i < PER; ++i) at[i] = lane * PER + i;
        // neighbours only, strictly larger ones move up: equal keys stay in index order
#pragma unroll
        for (int n = PER - 1; n > 0; --n)
#pragma unroll
          for (int i = 0; i < n; ++i) {
            const bool up = key[i + 1] > key[i];
            const uint32_t hi = max(key[i], key[i + 1]), lo = min(key[i], key[i + 1]);
            const int ha = up ? at[i + 1] : at[i], la = up ? at[i] : at[i + 1];
            key[i] = hi;
            key[i + 1] = lo;
            at[i] = ha;
            at[i + 1] = la;
          }
      };
#pragma unroll
      for (int i = 0; i < PER; ++i) key[i] = key_of(c[i]);
      if (grouped) {
        float b1 = ninf, b2 = ninf;
        if (whole) {
          sort_lane();
          float2* pair = reinterpret_cast<float2*>(cs);
          pair[lane] = make_float2(of_key(key[0]), PER > 1 ? of_key(key[PER > 1]) : ninf);
          __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
          if (lane < a.G) {
            const int lanes = per / PER;
#pragma unroll 4
            for (int i = 0; i < lanes; ++i) {
              const float2 v = pair[lane * lanes + i];
              b2 = __builtin_amdgcn_fmed3f(b1, b2, v.x);   // b2 <= b1: the second of three
              b1 = fmaxf(b1, v.x);
              b2 = fmaxf(b2, v.y);
            }
          }
        } else {
#pragma unroll
          for (int i = 0; i < PER; ++i) cs[lane * PER + i] = c[i];
          __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
          if (lane < a.G) {
#pragma unroll 4
            for (int i = 0; i < per; ++i) {
              const float v = cs[lane * per + i];
              b2 = __builtin_amdgcn_fmed3f(b1, b2, v);
              b1 = fmaxf(b1, v);
            }
          }
        }
        __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
        const float rank = a.group_score == 1 && b2 != ninf ? b1 + b2 : b1;
        const uint32_t rk = lane < a.G ? key_of(rank) : 0u;
        int better = 0;
        for (int g = 0; g < a.G; ++g) {
          const uint32_t o = static_cast<uint32_t>(__builtin_amdgcn_readlane(static_cast<int>(rk), g));
          better += o > rk || (o == rk && g < lane);
        }
        kept = __ballot(lane < a.G && better < a.top_groups);
        if (biased || by_s) {
          const bool in = (kept >> lane) & 1;
          const float low = of_key(~wave_max(in ? ~rk : 0u)), high = of_key(max(wave_max(in ? 0u : rk), kKeyNone));
          near = high != ninf && !(low - high > 0x1p-18f * fmaxf(1.0f, fmaxf(fabsf(low), fabsf(high))));
        }
        if (whole) {
          const bool in = (kept >> my_group) & 1;
#pragma unroll
          for (int i = 0; i < PER; ++i) key[i] = in ? key[i] : kKeyNone;
        } else {
#pragma unroll
          for (int i = 0; i < PER; ++i) {
            const bool in = (kept >> min((lane * PER + i) / per, 63)) & 1;
            key[i] = in ? key_of(by_s ? l[i] : c[i]) : kKeyNone;
          }
          sort_lane();
        }
      } else {
        sort_lane();
      }
      // one choice after another, and with biases the best that is left behind
      const int first = tt * seg;
      uint32_t got = 0;
      int id = -1;
      if (!near) {
        for (int j = 0; j < a.k + (biased ? 1 : 0); ++j) {
          const uint32_t top = wave_max(key[0]);
          if (top <= kKeyNone) break;
          const int owner = __builtin_ctzll(__ballot(key[0] == top));
          const int e = __builtin_amdgcn_readlane(at[0], owner);
          got = lane == j ? top : got;
          id = lane == j ? e : id;
          if (lane == owner) {
#pragma unroll
            for (int i = 0; i + 1 < PER; ++i) {
              key[i] = key[i + 1];
              at[i] = at[i + 1];
            }
            key[PER - 1] = kKeyNone;
          }
        }
        if (biased) {
          const uint32_t next = static_cast<uint32_t>(__shfl_down(static_cast<int>(got), 1));
          const int next_id = __shfl_down(id, 1);
          auto close = [](float u, float v) { return !(u - v > 0x1p-19f * fmaxf(1.0f, fmaxf(fabsf(u), fabsf(v)))); };
          bool differ = false, twins = false;
          if (lane < a.k && next_id >= 0 && close(of_key(got), of_key(next))) {
            const bool same = load_as_f32(row + id) == load_as_f32(row + next_id) && a.bias[id] == a.bias[next_id];
            differ = !same;
            twins = same && lane == a.k - 1;
          }
          near = __ballot(differ) != 0;
          if (!near && __ballot(twins)) {
            const int last = __builtin_amdgcn_readlane(id, a.k - 1);
            const float u = of_key(__builtin_amdgcn_readlane(static_cast<int>(got), a.k - 1));
            const float l_last = load_as_f32(row + last), b_last = a.bias[last];
            bool other = false;
#pragma unroll
            for (int i = 0; i < PER; ++i)
              if (key[i] > kKeyNone && close(u, of_key(key[i])))
                other = other || !(load_as_f32(row + at[i]) == l_last && a.bias[at[i]] == b_last);
            near = __ballot(other) != 0;
          }
        }
      }
      if (near) {
        route_exact<T, PER>(a, t0 + tt, scratch[wave]);
      } else {
        const int src = __shfl(id, lane - first);   // choice j of this token moves to lane first + j
        if (lane >= first && lane < first + seg) {
          my_id = src;
          my_max = m;
          my_total = total;
          done = false;
        }
      }
    }
    const int j = lane & (seg - 1);
    const int64_t t = t0 + lane / seg;
    double w = 0.0;
    if (!done && j < a.k && my_id >= 0) {
      const double v = static_cast<double>(load_as_f32(static_cast<const T*>(a.logits) + t * a.ldl + my_id));
      const double top = static_cast<double>(my_max);
      w = softmax ? (v == top ? 1.0 : exp(v - top)) : 1.0 / (1.0 + exp(-v));
    }
    double norm = my_total;
    if (a.renorm) norm = lanes_sum(w, seg);
    if (a.renorm || softmax) w = norm > 0.0 ? w / norm : 0.0;
    if (!done && j < a.k) {
      a.ids[t * a.k + j] = my_id;
      a.weights[t * a.k + j] = static_cast<float>(w * static_cast<double>(a.scale));
    }
  }
}

// The same for up to 256 experts in 1, 2, 4, 8 or 16 groups and up to 15 choices: a token per
// row of 16 lanes, four at a time per wave, PER experts per lane.  A group is 16 / G lanes, each
// with `each` of its experts; everything between the lanes of a row is data-parallel moves, so
// that the four tokens' chains run side by side where the kernel above waits for each step
// (16384 tokens of 256 experts in 8 groups: 16.6 us, and 34 there).  Values and results are the same; the
// check of two choice values takes 2^-18, since keys give 4 bits to their number.
// Bound by vector issue: 1155 vector instructions a wave take 74% of the cycles in which a CU has waves.
// Where every token is done again in fp64, one after another, the time is several times that: 16384
// peaked softmaxes of 256 experts, whose groups rank by sums of two scores near 0 without a bias,
// 49 us, and 13.9 for logits of ordinary spread.
// Batcher's merging network, largest first.
template <int N>
__device__ __forceinline__ void sort_descending(uint32_t (&v)[N]) {
#pragma unroll
  for (int p = 1; p < N; p *= 2)
#pragma unroll
    for (int k = p; k >= 1; k /= 2)
#pragma unroll
      for (int j = k % p; j < N - k; j += 2 * k)
#pragma unroll
        for (int i = 0; i < k; ++i)
          if (i + j + k < N && (i + j) / (2 * p) == (i + j + k) / (2 * p)) {
            const uint32_t hi = max(v[i + j], v[i + j + k]), lo = min(v[i + j], v[i + j + k]);
            v[i + j] = hi;
            v[i + j + k] = lo;
          }
}

template <typename T, int PER>
__global__ __launch_bounds__(256) void route_rows_kernel(RouteArgs a) {
  __shared__ double scratch[4][256];   // route_exact's
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int l16 = lane & 15;
  const float ninf = -INFINITY;
  const int per = a.per, each = a.each, lanes = 1 << a.log_lanes;
  const int group = l16 >> a.log_lanes, from = (l16 & (lanes - 1)) * each;   // from .. from + each - 1 of the group
  const int e0 = group * per + from, mine = min(each, per - from);
  const bool softmax = a.scoring == 0, biased = a.bias != nullptr, grouped = a.top_groups < a.G;
  const bool by_s = grouped && a.group_score == 1 && !biased;
  const int64_t t0 = (static_cast<int64_t>(blockIdx.x) * 4 + wave) * 4;
  if (t0 >= a.n_tokens) return;
  const int64_t t = min(t0 + lane / 16, a.n_tokens - 1);
  const bool live = t0 + lane / 16 < a.n_tokens;
  const T* row = static_cast<const T*>(a.logits) + t * a.ldl;

  float l[PER], bias[PER], m = ninf;
  // Wide loads, which the chip takes at any address, where the lanes' experts end with the row or
  // run on into another row of these logits (what they hold of it is not used).
  if (a.exact || (a.E >= 64 && t0 + 4 < a.n_tokens)) {
    T w[PER];
    __builtin_memcpy(w, row + e0, sizeof(w));
#pragma unroll
    for (int i = 0; i < PER; ++i) l[i] = load_as_f32(&w[i]);
  } else {
#pragma unroll
    for (int i = 0; i < PER; ++i) l[i] = load_as_f32(row + min(max(e0 + min(i, mine - 1), 0), a.E - 1));
  }
#pragma unroll
  for (int i = 0; i < PER; ++i) bias[i] = 0.0f;
  if (biased && a.exact) {
    __builtin_memcpy(bias, a.bias + e0, sizeof(bias));
  } else if (biased) {
#pragma unroll
    for (int i = 0; i < PER; ++i) bias[i] = a.bias[min(max(e0 + min(i, mine - 1), 0), a.E - 1)];
  }
#pragma unroll
  for (int i = 0; i < PER; ++i) l[i] = i < mine && l[i] == l[i] ? l[i] : ninf;

  float c[PER];
  double total = 0.0;
  if (softmax) {
    uint32_t k = key_of(l[0]);
#pragma unroll
    for (int i = 1; i < PER; ++i) k = max(k, key_of(l[i]));
    m = of_key(row_max(k));
#pragma unroll
    for (int i = 0; i < PER; ++i) {   // 0 at -150, where masked logits go
      c[i] = exp_f32(l[i] == m ? 0.0f : fmaxf(l[i] - m, -150.0f));
      total += static_cast<double>(c[i]);
    }
    total = row_sum(total);
  }
  uint32_t key[PER];
  if (biased || by_s) {
    const float r = softmax && total > 0.0 ? __builtin_amdgcn_rcpf(static_cast<float>(total)) : 0.0f;
#pragma unroll
    for (int i = 0; i < PER; ++i) {
      // sigmoid: the exponent's rounding moves s by s (1 - s) |l| 2^-24, under a third of a step
      const float s = softmax ? c[i] * r
                              : __builtin_amdgcn_rcpf(1.0f + __builtin_amdgcn_exp2f(l[i] * -0x1.715476p+0f));
      const float v = s + bias[i];
      key[i] = l[i] == ninf || !(v == v) ? kKeyNone : key_of(v);
    }
  } else {
#pragma unroll
    for (int i = 0; i < PER; ++i) key[i] = key_of(l[i]);
  }

  bool near = false;
  if (grouped) {
    uint32_t b1 = kKeyNone, b2 = kKeyNone;
#pragma unroll
    for (int i = 0; i < PER; ++i) {
      b2 = max(b2, min(b1, key[i]));
      b1 = max(b1, key[i]);
    }
    auto join = [&](uint32_t o1, uint32_t o2) {
      b2 = max(max(b2, o2), min(b1, o1));
      b1 = max(b1, o1);
    };
    // a group's lanes by swaps inside pairs, quads, halves and the row
    if (lanes > 1) join(moved<0xB1>(b1), moved<0xB1>(b2));
    if (lanes > 2) join(moved<0x4E>(b1), moved<0x4E>(b2));
    if (lanes > 4) join(moved<0x141>(b1), moved<0x141>(b2));
    if (lanes > 8) join(moved<0x140>(b1), moved<0x140>(b2));
    const float rank = a.group_score == 1 && b2 != kKeyNone ? of_key(b1) + of_key(b2) : of_key(b1);
    const uint32_t rk = key_of(rank);
    int better = 0;
    for (int g = 1; g < a.G; ++g) {
      const uint32_t o = static_cast<uint32_t>(__shfl(static_cast<int>(rk), (lane & 48) | ((l16 + g * lanes) & 15)));
      better += (o > rk) | ((o == rk) & (group + g >= a.G));   // wrapped round: a lower group
    }
    const bool in = better < a.top_groups;
    if (biased || by_s) {
      const float low = of_key(~row_max(in ? ~rk : 0u)), high = of_key(max(row_max(in ? 0u : rk), kKeyNone));
      near = high != ninf && !(low - high > 0x1p-18f * fmaxf(1.0f, fmaxf(fabsf(low), fabsf(high))));
    }
    if (by_s) {
#pragma unroll
      for (int i = 0; i < PER; ++i) key[i] = key_of(l[i]);
    }
#pragma unroll
    for (int i = 0; i < PER; ++i) key[i] = in ? key[i] : kKeyNone;
  }
  // Keys carry their number in the lane in the low 4 bits (28 bits of value: all that 16-bit
  // logits have), so that sorting them is maxima and minima alone.
#pragma unroll
  for (int i = 0; i < PER; ++i) key[i] = (key[i] & ~15u) | static_cast<uint32_t>(15 - i);
  sort_descending<PER>(key);
  // one choice after another, and the best that is left behind where near values matter; lane j
  // keeps choice j
  const bool exact = !biased && sizeof(T) == 2;   // keys are logits in full
  uint32_t got = 0;
  int owner = -1;
  for (int j = 0; j < a.k + (exact ? 0 : 1); ++j) {
    const uint32_t value = row_max(key[0] & ~15u);
    // the lowest lane that holds it, and its number there
    const uint32_t at = row_max((key[0] & ~15u) == value ? (15u - l16) << 4 | (key[0] & 15u) : 0u);
    const uint32_t top = value | (at & 15u), first = 15u - (at >> 4);
    // that lane moves up its keys, by a bit mask (as selections the compiler turns this into
    // indexing, 400 instructions)
    uint32_t out = l16 == static_cast<int>(first) ? ~0u : 0u;
    asm("" : "+v"(out));
#pragma unroll
    for (int i = 0; i < PER; ++i) key[i] = ((i + 1 < PER ? key[i + 1 < PER ? i + 1 : 0] : kKeyNone) & out) | (key[i] & ~out);
    const bool here = l16 == j && top > kKeyNone;
    got = here ? top : got;
    owner = here ? static_cast<int>(first) : owner;
  }
  const int id = owner < 0 ? -1
                           : (owner >> a.log_lanes) * per + (owner & (lanes - 1)) * each + 15 - static_cast<int>(got & 15u);
  if (!exact) {
    const uint32_t next = moved<0x101>(got);                               // the lane after (row_shl 1)
    const int next_id = static_cast<int>(moved<0x101>(static_cast<uint32_t>(id + 1))) - 1;
    auto close = [&](uint32_t p, uint32_t q) {
      const float u = of_key(p & ~15u), v = of_key(q & ~15u);
      const float tol = biased ? 0x1p-18f * fmaxf(1.0f, fmaxf(fabsf(u), fabsf(v))) : 0.0f;
      return !(u - v > tol);
    };
    auto alike = [&](int p, int q) {
      return load_as_f32(row + p) == load_as_f32(row + q) && (!biased || a.bias[p] == a.bias[q]);
    };
    bool twins = false;
    if (l16 < a.k && next_id >= 0 && close(got, next)) {
      const bool same = alike(id, next_id);
      near = near || !same;
      twins = same && l16 == a.k - 1;
    }
    if (__ballot(twins)) {
      const int src = (lane & 48) | (a.k - 1);
      const uint32_t u = static_cast<uint32_t>(__shfl(static_cast<int>(got), src));
      const int last = __shfl(id, src);
      if (__shfl(static_cast<int>(twins), src)) {
#pragma unroll
        for (int i = 0; i < PER; ++i)
          if (key[i] > kKeyNone && close(u, key[i]))
            near = near || !alike(last, e0 + 15 - static_cast<int>(key[i] & 15u));
      }
    }
  }
  uint64_t again = __ballot(near && live);
  double w = 0.0;
  if (l16 < a.k && id >= 0) {
    const float v = load_as_f32(row + id);
    if (softmax) w = v == m ? 1.0 : exp(static_cast<double>(v) - static_cast<double>(m));
    else w = 1.0 / (1.0 + exp(-static_cast<double>(v)));
  }
  double norm = total;
  if (a.renorm) norm = row_sum(w);
  if (a.renorm || softmax) w = norm > 0.0 ? w / norm : 0.0;
  if (live && l16 < a.k && ((again >> (lane & 48)) & 0xFFFF) == 0) {
    a.ids[t * a.k + l16] = id;
    a.weights[t * a.k + l16] = static_cast<float>(w * static_cast<double>(a.scale));
  }
  while (again) {
    const int r = __builtin_ctzll(again) / 16;
    again &= ~(0xFFFFull << (16 * r));
    if (a.E <= 64) route_exact<T, 1>(a, t0 + r, scratch[wave]);
    else route_exact<T, 4>(a, t0 + r, scratch[wave]);
  }
}

template <typename T>
gptq_status launch_route(RouteArgs a, hipStream_t stream) {
  const dim3 block(256);
  if (a.E <= 256 && a.k <= 15 && a.G <= 16 && 16 % a.G == 0) {
    const int per = a.E / a.G, lanes = 16 / a.G, each = (per + lanes - 1) / lanes;
    const int slots = each <= 4 ? 4 : each <= 8 ? 8 : 16;
    a.exact = each == slots && per == lanes * each;
    a.per = per;
    a.each = each;
    a.log_lanes = __builtin_ctz(lanes);
    const int64_t blocks = (a.n_tokens + 15) / 16;
    if (blocks > (1 << 24) - 1) return GPTQ_ERR_UNSUPPORTED;
    const dim3 grid(static_cast<unsigned>(blocks));
    if (slots == 4) GPTQ_LAUNCH((route_rows_kernel<T, 4>), grid, block, 0, stream, a);
    else if (slots == 8) GPTQ_LAUNCH((route_rows_kernel<T, 8>), grid, block, 0, stream, a);
    else GPTQ_LAUNCH((route_rows_kernel<T, 16>), grid, block, 0, stream, a);
    return GPTQ_OK;
  }
  // a wave per token while there are few; then 4 tokens (2 where a token has over 16 choices)
  a.batch = a.n_tokens < 4096 ? 1 : a.k <= 16 ? 4 : 2;
  const int64_t per = 4 * a.batch;
  const dim3 grid(static_cast<unsigned>(std::min<int64_t>((a.n_tokens + per - 1) / per, 4096)));
  if (a.E <= 64) GPTQ_LAUNCH((route_kernel<T, 1>), grid, block, 0, stream, a);
  else if (a.E <= 256) GPTQ_LAUNCH((route_kernel<T, 4>), grid, block, 0, stream, a);
  else GPTQ_LAUNCH((route_kernel<T, 16>), grid, block, 0, stream, a);
  return GPTQ_OK;
}

// ---------------------------------------------------------------------------- grouping

constexpr int GR_WAVES = 16;
constexpr int GR_NT = GR_WAVES * 64;
constexpr int GR_CHUNKS = 64;     // most chunks of slots
constexpr int GR_ONE = 8192;      // up to this many slots: one chunk, one launch

__global__ __launch_bounds__(GR_NT) void group_count_kernel(const int32_t* __restrict__ ids, int64_t slots, int chunk,
                                                            int E, int32_t* __restrict__ counts) {
  __shared__ int32_t h[1024];
  for (int e = threadIdx.x; e < E; e += GR_NT) h[e] = 0;
  __syncthreads();
  const int64_t s0 = static_cast<int64_t>(blockIdx.x) * chunk;
  const int64_t s1 = min(slots, s0 + chunk);
  for (int64_t s = s0 + threadIdx.x; s < s1; s += GR_NT) {
    const int id = ids[s];
    if (static_cast<unsigned>(id) < static_cast<unsigned>(E)) atomicAdd(&h[id], 1);
  }
  __syncthreads();
  for (int e = threadIdx.x; e < E; e += GR_NT) counts[static_cast<int64_t>(blockIdx.x) * E + e] = h[e];
}

// One chunk of slots per workgroup, a contiguous sixteenth of it per wave.  A slot's position is
// the start of its expert + the expert's slots in earlier chunks + in earlier waves of this
// chunk + earlier in its wave (64 slots at a time: equal ids found by one ballot per bit).  Every
// workgroup adds up the counts of all chunks for itself (up to 64 numbers per expert), which
// saves a launch; no order of atomics reaches the result.  Bound by latency (131072 slots of 256
// experts: 2.9 us to count and 7.7 to place; 24 slots: 3.1).
// HOLD: a wave's ids, up to 512, stay in registers for the second pass, where their loads would come
// one after another (6126 slots of 160 experts: 8.6 us, 10.3 without; 24 slots: 3.5 and 3.1).
constexpr int GR_HELD = 8;
template <bool HOLD>
__global__ __launch_bounds__(GR_NT) void group_place_kernel(const int32_t* __restrict__ ids, int64_t slots, int chunk,
                                                            int E, int k, const int32_t* __restrict__ counts,
                                                            int64_t* __restrict__ offsets,
                                                            int32_t* __restrict__ row_index,
                                                            int32_t* __restrict__ place) {
  __shared__ int32_t h[GR_WAVES][1024];
  __shared__ int32_t base[1024];   // slots of this chunk's experts in earlier chunks, then their starts
  __shared__ int32_t tot[1024];
  __shared__ int32_t wsum[GR_WAVES];
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int chunks = gridDim.x, me = blockIdx.x;
  const int64_t s0 = static_cast<int64_t>(me) * chunk;
  const int64_t s1 = min(slots, s0 + chunk);
  const int seg = chunk / GR_WAVES;   // a multiple of 64
  const int64_t w0 = s0 + static_cast<int64_t>(wave) * seg, w1 = min(s1, w0 + seg);
  for (int e = lane; e < E; e += 64) h[wave][e] = 0;
  base[tid] = 0;
  tot[tid] = 0;
  __syncthreads();
  int held[HOLD ? GR_HELD : 1];
  if constexpr (HOLD) {
#pragma unroll
    for (int i = 0; i < GR_HELD; ++i)
      if (64 * i < seg) held[i] = w0 + 64 * i + lane < w1 ? ids[w0 + 64 * i + lane] : -1;
#pragma unroll
    for (int i = 0; i < GR_HELD; ++i)
      if (64 * i < seg && static_cast<unsigned>(held[i]) < static_cast<unsigned>(E)) atomicAdd(&h[wave][held[i]], 1);
  } else {
    for (int64_t s = w0 + lane; s < w1; s += 64) {
      const int id = ids[s];
      if (static_cast<unsigned>(id) < static_cast<unsigned>(E)) atomicAdd(&h[wave][id], 1);
    }
  }
  if (chunks > 1) {
    // several threads per expert, 16 loads in flight each
    const int parts = max(1, GR_NT / E), e = tid % E, part = tid / E;
    if (part < parts) {
      int before = 0, all = 0;
      for (int c0 = part; c0 < chunks; c0 += 16 * parts) {
        int n[16];
#pragma unroll
        for (int i = 0; i < 16; ++i) {
          const int c = c0 + i * parts;
          n[i] = c < chunks ? counts[static_cast<int64_t>(c) * E + e] : 0;
        }
#pragma unroll
        for (int i = 0; i < 16; ++i) {
          all += n[i];
          before += c0 + i * parts < me ? n[i] : 0;
        }
      }
      atomicAdd(&tot[e], all);
      atomicAdd(&base[e], before);
    }
    __syncthreads();
  } else {
    __syncthreads();
    if (tid < E) {
      int all = 0;
#pragma unroll
      for (int w = 0; w < GR_WAVES; ++w) all += h[w][tid];
      tot[tid] = all;
    }
  }
  // exclusive sums of the totals, one expert per thread
  const int x = chunks > 1 ? tot[tid] : (tid < E ? tot[tid] : 0);
  int inc = x;
  for (int d = 1; d < 64; d <<= 1) {
    const int o = __shfl_up(inc, d);
    if (lane >= d) inc += o;
  }
  if (lane == 63) wsum[wave] = inc;
  __syncthreads();
  int lead = 0, total = 0;
#pragma unroll
  for (int w = 0; w < GR_WAVES; ++w) {
    lead += w < wave ? wsum[w] : 0;
    total += wsum[w];
  }
  const int start = lead + inc - x;
  if (me == 0) {
    if (tid < E) offsets[tid] = start;
    if (tid == 0) offsets[E] = total;
  }
  if (tid < E) {
    int run = base[tid] + start;
#pragma unroll
    for (int w = 0; w < GR_WAVES; ++w) {
      const int n = h[w][tid];
      h[w][tid] = run;
      run += n;
    }
  }
  __syncthreads();
  volatile int32_t* mine = h[wave];
  const int bits = 32 - __builtin_clz(E);
  auto put = [&](int64_t b, int id) {
    const int64_t s = b + lane;
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
      row_index[p] = static_cast<int32_t>(static_cast<uint32_t>(s) / static_cast<uint32_t>(k));
      place[s] = p;
      __builtin_amdgcn_wave_barrier();
      if (rank == 0) mine[id] = p + __popcll(same);
    } else if (s < w1) {
      place[s] = -1;
    }
    __builtin_amdgcn_wave_barrier();
  };
  if constexpr (HOLD) {
#pragma unroll
    for (int i = 0; i < GR_HELD; ++i)
      if (w0 + 64 * i < w1) put(w0 + 64 * i, held[i]);
  } else {
    for (int64_t b = w0; b < w1; b += 64) put(b, b + lane < w1 ? ids[b + lane] : -1);
  }
  for (int64_t s = s0 + tid; s < s1; s += GR_NT)
    if (s >= total) row_index[s] = -1;
}

__global__ void group_none_kernel(int64_t* __restrict__ offsets, int n) {
  for (int i = threadIdx.x; i < n; i += 256) offsets[i] = 0;
}

int group_chunk(int64_t slots) {
  const int64_t c = slots <= GR_ONE ? std::max<int64_t>(slots, 1) : std::max<int64_t>(GR_ONE / 8, (slots + GR_CHUNKS - 1) / GR_CHUNKS);
  return static_cast<int>((c + GR_NT - 1) / GR_NT * GR_NT);
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

// V neighbouring outputs of one token.
template <typename T, int V>
__device__ __forceinline__ void combine_piece(int k, int64_t n_rows, const T* Y, int64_t ldy, const int32_t* place,
                                              const float* weights, T* out) {
  float acc[V];
#pragma unroll
  for (int v = 0; v < V; ++v) acc[v] = 0.0f;
  for (int j = 0; j < k; ++j) {
    const int p = place[j];
    if (p < 0 || p >= n_rows) continue;
    const float w = weights[j];
    T y[V];
    __builtin_memcpy(y, Y + p * ldy, sizeof(y));
#pragma unroll
    for (int v = 0; v < V; ++v) acc[v] = fmaf(w, load_as_f32(&y[v]), acc[v]);
  }
  T o[V];
#pragma unroll
  for (int v = 0; v < V; ++v) o[v] = from_f32<T>(acc[v]);
  __builtin_memcpy(out, o, sizeof(o));
}

// One thread per 16 bytes of a token's outputs; the chip loads and stores 16 bytes at any address,
// so rows may start at any element.  Bound by memory (16384 tokens of 6 x 2048 in bf16: 95 us, 4.95
// TB/s; of 6 x 2047: 101 us, 352 by single values).
template <typename T>
__global__ __launch_bounds__(256) void combine_kernel(int64_t n_tokens, int k, int64_t n_rows, int d, const T* Y,
                                                      int64_t ldy, const int32_t* place, const float* weights, T* out,
                                                      int64_t ldo) {
  constexpr int V = 16 / sizeof(T);
  const int per = (d + V - 1) / V;
  const int64_t i = (static_cast<int64_t>(blockIdx.y) * gridDim.x + blockIdx.x) * 256 + threadIdx.x;
  const int64_t t = i / per;
  if (t >= n_tokens) return;
  // a row's last piece ends with the row: outputs that it shares with the one before get equal values
  const int64_t col = max(min((i - t * per) * V, static_cast<int64_t>(d) - V), static_cast<int64_t>(0));
  if (d >= V) combine_piece<T, V>(k, n_rows, Y + col, ldy, place + t * k, weights + t * k, out + t * ldo + col);
  else
    for (int v = 0; v < d; ++v)
      combine_piece<T, 1>(k, n_rows, Y + v, ldy, place + t * k, weights + t * k, out + t * ldo + v);
}

template <typename T>
gptq_status launch_combine(int64_t n_tokens, int k, int64_t n_rows, int d, const void* Y, int64_t ldy,
                           const int32_t* place, const float* weights, void* out, int64_t ldo, hipStream_t stream) {
  constexpr int V = 16 / sizeof(T);
  // a launch's threads along x stay below 2^32
  const int64_t blocks = (n_tokens * ((d + V - 1) / V) + 255) / 256;
  const int64_t gx = std::min<int64_t>(blocks, 1 << 22), gy = (blocks + gx - 1) / gx;
  if (gy > 65535) return GPTQ_ERR_UNSUPPORTED;
  const dim3 grid(static_cast<unsigned>(gx), static_cast<unsigned>(gy)), block(256);
  GPTQ_LAUNCH((combine_kernel<T>), grid, block, 0, stream, n_tokens, k, n_rows, d, static_cast<const T*>(Y), ldy, place,
              weights, static_cast<T*>(out), ldo);
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

// 256 where nothing is kept in it, more where the counts are, however few experts there are: callers
// pass none for 256.
size_t group_workspace(int n_experts, int64_t slots) {
  const int chunk = group_chunk(slots);
  const int64_t chunks = (slots + chunk - 1) / chunk;
  return 256 + (chunks > 1 ? align_up(static_cast<size_t>(chunks) * n_experts * sizeof(int32_t), 256) : 0);
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
    GPTQ_LAUNCH(group_count_kernel, dim3(chunks), dim3(GR_NT), 0, stream, ids, slots, chunk, n_experts, counts);
  const int per_wave = chunk / GR_WAVES;
  if (per_wave > 64 && per_wave <= 64 * GR_HELD)
    GPTQ_LAUNCH(group_place_kernel<true>, dim3(chunks), dim3(GR_NT), 0, stream, ids, slots, chunk, n_experts, top_k,
                counts, token_offsets, row_index, place);
  else
    GPTQ_LAUNCH(group_place_kernel<false>, dim3(chunks), dim3(GR_NT), 0, stream, ids, slots, chunk, n_experts, top_k,
                counts, token_offsets, row_index, place);
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
