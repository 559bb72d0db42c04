// One token per row of logits, from a given uniform random number.
//
// With m the row's largest logit and t its temperature, token i weighs w_i = exp((x_i - m)/t).
// The kept tokens are a prefix of the order "larger logit first, lower index first among
// equals": the shortest of the prefixes that top-k, top-p (mass before the token below
// top_p times the mass of the top-k survivors) and min-p (w_i >= min_p) allow.  The sampled
// token is the first in vocabulary order whose cumulated kept weight exceeds u times the total.
// t = 0 keeps the largest logit alone.
//
// One CTA per row.  No sort: the two prefixes come from a radix descent over a monotone
// 32-bit key of the logit, by count for top-k and by mass for top-p.  Masses that meet in
// atomics are 64-bit integers (weight * 2^42), so their order does not matter; weights and
// the sums that pick the token are in 64 bits, since a token is decided by where u * total
// falls between two of up to a million borders.
#include <math_constants.h>

#include "serving.cuh"

namespace tv {
namespace {

constexpr int kThreads = 512;
constexpr int kWarps = kThreads / 32;
constexpr double kScale = 4398046511104.0;     // 2^42: a million weights stay below 2^62
constexpr uint32_t kKeyNegInf = 0x007FFFFFu;   // key of -inf

// Monotone key: larger float, larger key.  NaN counts as -inf, -0 as +0.
__device__ __forceinline__ uint32_t key_of(float x) {
  if (x != x) x = -CUDART_INF_F;
  const uint32_t b = __float_as_uint(x + 0.f);
  return b & 0x80000000u ? ~b : b | 0x80000000u;
}
__device__ __forceinline__ float value_of(uint32_t key) {
  return __uint_as_float(key & 0x80000000u ? key & 0x7FFFFFFFu : ~key);
}

struct SampleSmem {
  unsigned long long hist[256];
  unsigned long long part[kWarps];
  double above[kWarps];
  int ties[kWarps];
  uint32_t digit;
  unsigned long long before;
  int seg, seg_ties;
  double target, seg_before, total;
};

struct Weigher {
  float max;
  double t;
  __device__ __forceinline__ double operator()(uint32_t key) const {
    const float x = value_of(key);
    return x == max ? 1.0 : exp(((double)x - (double)max) / t);
  }
};

__device__ __forceinline__ unsigned long long fixed(double w) {
  return (unsigned long long)__double2ll_rn(w * kScale);
}

template <typename T>
__global__ void __launch_bounds__(kThreads) sample_kernel(SampleArgs a) {
  __shared__ SampleSmem sm;
  const int row = blockIdx.x, tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, V = a.V;
  const T *x = static_cast<const T *>(a.logits) + (long long)row * a.stride;
  const float u = a.uniform[row], t = a.temperature ? a.temperature[row] : 1.f;
  const float top_p = a.top_p ? a.top_p[row] : 1.f, min_p = a.min_p ? a.min_p[row] : 0.f;
  const int top_k = a.top_k ? a.top_k[row] : 0;
  if (!(u >= 0.f && u <= 1.f && t >= 0.f && t < CUDART_INF_F && top_p >= 0.f && top_p <= 1.f &&
        min_p >= 0.f && min_p <= 1.f)) {
    if (tid == 0) set_status(a.ws, TV_ERR_BAD_PARAM, row);
    return;
  }

  // ---- largest logit, lowest index of it -------------------------------------------------
  unsigned long long best = 0;
  for (int i = tid; i < V; i += kThreads) {
    const unsigned long long c = (unsigned long long)key_of(to_f32(x[i])) << 32 | (0xFFFFFFFFu - i);
    best = c > best ? c : best;
  }
#pragma unroll
  for (int o = 16; o; o >>= 1) {
    const unsigned long long c = __shfl_xor_sync(0xffffffffu, best, o);
    best = c > best ? c : best;
  }
  if (lane == 0) sm.part[warp] = best;
  __syncthreads();
  best = sm.part[0];
  for (int w = 1; w < kWarps; ++w) best = sm.part[w] > best ? sm.part[w] : best;
  const uint32_t max_key = best >> 32;
  if (max_key == kKeyNegInf || t == 0.f) {
    if (tid == 0) {
      const bool none = max_key == kKeyNegInf;
      a.token[row] = none ? -1 : (int)(0xFFFFFFFFu - (uint32_t)best);
      if (a.logprob) a.logprob[row] = none ? -CUDART_INF_F : 0.f;
    }
    return;
  }
  const Weigher weight{value_of(max_key), (double)t};

  // ---- kept: keys above `edge`, and the first `n_edge` equal to it ------------------------
  uint32_t edge = 0;
  int n_edge = V;
  if (top_k > 0 && top_k < V) {
    uint32_t prefix = 0, mask = 0;
    unsigned long long before = 0;
    for (int shift = 24; shift >= 0; shift -= 8) {
      if (tid < 256) sm.hist[tid] = 0;
      __syncthreads();
      for (int i = tid; i < V; i += kThreads) {
        const uint32_t key = key_of(to_f32(x[i]));
        if ((key & mask) == prefix) atomicAdd(&sm.hist[key >> shift & 255], 1ull);
      }
      __syncthreads();
      if (tid == 0) {
        int d = 255;
        unsigned long long c = before;
        for (; d > 0 && c + sm.hist[d] < (unsigned long long)top_k; --d) c += sm.hist[d];
        sm.digit = d;
        sm.before = c;
      }
      __syncthreads();
      before = sm.before;
      prefix |= sm.digit << shift;
      mask |= 255u << shift;
      __syncthreads();
    }
    edge = prefix;
    n_edge = top_k - (int)before;
  }
  if (top_p < 1.f) {
    // mass of the survivors of top-k
    unsigned long long mass = 0;
    for (int i = tid; i < V; i += kThreads) {
      const uint32_t key = key_of(to_f32(x[i]));
      if (key > edge) mass += fixed(weight(key));
    }
#pragma unroll
    for (int o = 16; o; o >>= 1) mass += __shfl_xor_sync(0xffffffffu, mass, o);
    if (lane == 0) sm.part[warp] = mass;
    __syncthreads();
    mass = edge ? n_edge * fixed(weight(edge)) : 0;
    for (int w = 0; w < kWarps; ++w) mass += sm.part[w];
    const double goal = (double)top_p * (double)mass;
    uint32_t prefix = 0, mask = 0;
    unsigned long long before = 0;
    for (int shift = 24; shift >= 0; shift -= 8) {
      __syncthreads();
      if (tid < 256) sm.hist[tid] = 0;
      __syncthreads();
      for (int i = tid; i < V; i += kThreads) {
        const uint32_t key = key_of(to_f32(x[i]));
        if (key >= edge && (key & mask) == prefix)
          atomicAdd(&sm.hist[key >> shift & 255], fixed(weight(key)));
      }
      __syncthreads();
      if (tid == 0) {
        // the last digit that holds mass and starts below the goal (the largest logit holds
        // the most, so there is one)
        unsigned long long c = before;
        int pick = -1;
        unsigned long long at = before;
        for (int d = 255; d >= 0; --d) {
          if (!sm.hist[d]) continue;
          if (pick >= 0 && !((double)c < goal)) break;
          pick = d;
          at = c;
          c += sm.hist[d];
        }
        sm.digit = pick;
        sm.before = at;
      }
      __syncthreads();
      before = sm.before;
      prefix |= sm.digit << shift;
      mask |= 255u << shift;
    }
    // equals at the border: kept while the mass before them is below the goal
    const unsigned long long w = fixed(weight(prefix));
    int most = prefix == edge ? n_edge : V, n = 1;
    if (w) {
      const double d = (goal - (double)before) / (double)w;
      n = d >= (double)most ? most : max(1, (int)ceil(d));
    }
    edge = prefix;
    n_edge = min(n, most);
  }

  // ---- kept weight by segments of the vocabulary, one warp each --------------------------
  const int seg = ((V + kWarps - 1) / kWarps + 31) / 32 * 32;
  const int s0 = min(V, warp * seg), s1 = min(V, s0 + seg);
  double above = 0.0;
  int ties = 0;
  for (int i = s0 + lane; i < s1; i += 32) {
    const uint32_t key = key_of(to_f32(x[i]));
    if (key > edge) {
      const double w = weight(key);
      if (w >= (double)min_p) above += w;
    } else if (key == edge) {
      ++ties;
    }
  }
#pragma unroll
  for (int o = 16; o; o >>= 1) {
    above += __shfl_xor_sync(0xffffffffu, above, o);
    ties += __shfl_xor_sync(0xffffffffu, ties, o);
  }
  if (lane == 0) {
    sm.above[warp] = above;
    sm.ties[warp] = ties;
  }
  const double w_raw = weight(edge), w_edge = w_raw >= (double)min_p ? w_raw : 0.0;
  __syncthreads();
  if (tid == 0) {
    double total = 0.0;
    int left = n_edge;
    for (int w = 0; w < kWarps; ++w) {
      const int k = min(left, sm.ties[w]);
      total += sm.above[w] + k * w_edge;
      left -= k;
    }
    const double target = (double)u * total;
    double c = 0.0;
    left = n_edge;
    sm.seg = -1;
    for (int w = 0; w < kWarps; ++w) {
      const int k = min(left, sm.ties[w]);
      const double m = sm.above[w] + k * w_edge;
      if (m > 0.0) {
        sm.seg = w;
        sm.seg_ties = left;
        sm.seg_before = c;
        if (c + m > target) break;
      }
      c += m;
      left -= k;
    }
    sm.total = total;
    sm.target = target;
  }
  __syncthreads();
  if (warp != sm.seg) return;

  // ---- the token, by the warp that owns its segment ----------------------------------------
  double c = sm.seg_before;
  int left = sm.seg_ties, token = -1;
  double w_token = 0.0;
  for (int i0 = s0; i0 < s1; i0 += 32) {
    const int i = i0 + lane;
    const uint32_t key = i < s1 ? key_of(to_f32(x[i])) : 0;
    const bool tie = i < s1 && key == edge;
    const unsigned tied = __ballot_sync(0xffffffffu, tie);
    const int rank = __popc(tied & ((1u << lane) - 1));
    double w = 0.0;
    if (i < s1 && (key > edge || (tie && rank < left))) {
      w = weight(key);
      if (w < (double)min_p) w = 0.0;
    }
    left -= min(left, __popc(tied));
    double sum = w;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const double y = __shfl_up_sync(0xffffffffu, sum, o);
      if (lane >= o) sum += y;
    }
    const unsigned live = __ballot_sync(0xffffffffu, w > 0.0);
    const unsigned hit = __ballot_sync(0xffffffffu, w > 0.0 && c + sum > sm.target);
    if (live) {                          // the last kept token so far, in case none is past
      const int src = hit ? __ffs(hit) - 1 : 31 - __clz(live);
      token = i0 + src;
      w_token = __shfl_sync(0xffffffffu, w, src);
    }
    if (hit) break;
    c += __shfl_sync(0xffffffffu, sum, 31);
  }
  if (lane == 0) {
    a.token[row] = token;
    if (a.logprob) a.logprob[row] = (float)log(w_token / sm.total);
  }
}

}  // namespace

cudaError_t launch_sample(const SampleArgs &a, int in_dtype, cudaStream_t st) {
  if (in_dtype == TV_F32) sample_kernel<float><<<a.R, kThreads, 0, st>>>(a);
  else sample_kernel<__nv_bfloat16><<<a.R, kThreads, 0, st>>>(a);
  return cudaGetLastError();
}

}  // namespace tv
